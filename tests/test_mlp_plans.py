"""CPU: the sizes of tests/mlp_plans.py reach the kernels they are meant to, and
together every variant of the products that begin with the rest's steps."""
import shutil

import pytest

from ffn_plans import Plans
from mlp_plans import BACKWARD_REST


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    return Plans(tmp_path_factory.mktemp("plan"))


def test_sizes_reach_their_kernels(plans):
    for key, want in BACKWARD_REST.items():
        assert plans.backward(*key, False, True) == want, key


def test_every_variant_is_reached():
    for product in (0, 1):
        got = {(p[product][0], p[product][1] > 1) for p in BACKWARD_REST.values() if p[product][2] > 2}
        assert got == {(bm, s) for bm in (64, 128, 256) for s in (False, True)}, product
    kinds = set()
    for (M, _, N), plan in BACKWARD_REST.items():
        for (_, splits, kper), C in zip(plan, ((N + 127) // 128 * 128, (M + 127) // 128 * 128)):
            for i in range(splits):
                first, end = i * kper, min((i + 1) * kper, C // 64 + C // 128)
                kinds.add("rest" if end <= C // 128 else "f16" if first >= C // 128 else "both")
    assert kinds == {"rest", "both", "f16"}
