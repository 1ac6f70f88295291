"""CPU: the sizes of tests/mlp_plans.py reach the kernels they are meant to, and
together every variant of layer norm and of the products that begin with the
rest's steps."""
import shutil

import pytest

from ffn_plans import Plans
from mlp_plans import BACKWARD_REST, LAYERNORM, LayerNormPlan


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


def test_layernorm_variants(plans, tmp_path):
    plan = LayerNormPlan(tmp_path)
    for key, want in LAYERNORM.items():
        assert plan(*key) == want, key
        assert key[0] > want[3], key                       # more rows than the grid takes at once
    # wave or workgroup, vectors, size of the workgroup, and rows of whole lines or not
    kind = lambda k, p: (p[0], p[1], p[2] > (256 if p[1] == 1 else 768), k[1] * (4 if k[2] == "f32" else 2) % 128 == 0)
    got = {kind(k, p) for k, p in LAYERNORM.items()}
    assert got == {(w, v, big, whole) for whole in (False, True)
                   for w, v, big in ((True, 1, False), (True, 2, False), (False, 1, False), (False, 1, True),
                                     (False, 2, False), (False, 2, True), (False, 4, big4(whole)))}
    assert plan(10, 3, "f32")[1] == 0 and plan(10, 7, "bf16")[1] == 0 and plan(10, 40000, "bf16")[1] == 0
    # never more vectors than its threads hold
    for nv in range(1, 4097):
        for rows in (1, 300):
            _, v, t, _ = plan(rows, nv * 8, "bf16")
            assert (v * (64 if plan(rows, nv * 8, "bf16")[0] else t)) >= nv, (rows, nv)


def big4(whole):
    """the two sizes of four vectors a thread: 1024 threads and 576"""
    return whole
