"""CPU: the sizes of tests/ffn_plans.py reach the kernels they are meant to, and
together every kernel variant, past the first steps of its pipeline or the first
row of its loop."""
import shutil

import pytest

from ffn_plans import BACKWARD, BACKWARD_REST, FORWARD, NORM, NORM_BACKWARD, NORM_ODD, Plans


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    return Plans(tmp_path_factory.mktemp("plan"))


def test_sizes_reach_their_kernels(plans):
    for key, want in FORWARD.items():
        assert plans.forward(*key) == want, key
    for key, want in BACKWARD.items():
        assert plans.backward(*key) == want, key
    for key, want in BACKWARD_REST.items():
        assert plans.backward(*key, True, True) == want, key
    for table in (NORM, NORM_ODD):
        for key, want in table.items():
            assert plans.norm(*key) == want, key
    for key, want in NORM_BACKWARD.items():
        assert plans.norm_backward(*key) == want, key


def test_every_variant_is_reached():
    """k_mm: heights x {whole, split} x {projection, pair} x kind of sum (binary32
    sums have no 256), each with a steady step; the cast of whole and of split
    products at both heights; k_mm16: heights x {whole, split} in both products of
    both backward passes, with more than two steps; the norms: more rows than the
    grid takes at once."""
    fwd = {(gated, exact, bm, s > 1) for (_, _, _, gated, exact), (bm, s, kper) in FORWARD.items()
           if kper > (2 if bm == 256 else 3)}
    assert fwd == {(g, e, bm, s) for g in (False, True) for e in (False, True) for bm in (64, 128, 256)
                   for s in (False, True) if not (e and bm == 256)}
    cast = {(bm, s > 1) for (_, _, F, gated, exact), (bm, s, _) in FORWARD.items() if gated and exact and F % 128 == 0}
    assert cast == {(bm, s) for bm in (64, 128) for s in (False, True)}
    for gated in (False, True):
        for product in (0, 1):
            got = {(p[product][0], p[product][1] > 1) for k, p in BACKWARD.items() if k[3] == gated and p[product][2] > 2}
            assert got == {(bm, s) for bm in (64, 128, 256) for s in (False, True)}, (gated, product)
    for product in (0, 1):
        got = {(p[product][0], p[product][1] > 1) for p in BACKWARD_REST.values() if p[product][2] > 2}
        assert got == {(bm, s) for bm in (64, 128, 256) for s in (False, True)}, product
    # splits of the rest's steps alone, of both kinds, and of f16 steps alone
    kinds = set()
    for (M, _, F), plan in BACKWARD_REST.items():
        for (_, splits, kper), C in zip(plan, (2 * ((F + 63) // 64 * 64), (M + 127) // 128 * 128)):
            for i in range(splits):
                first, end = i * kper, min((i + 1) * kper, C // 64 + C // 128)
                kinds.add("rest" if end <= C // 128 else "f16" if first >= C // 128 else "both")
    assert kinds == {"rest", "both", "f16"}
    for table in (NORM, NORM_ODD, NORM_BACKWARD):
        for (rows, _, _), (_, _, _, at_once) in table.items():
            assert rows > at_once
    kinds = lambda table: {(w, V, T > 512) for w, V, T, _ in table.values()}
    rows = {(True, 1, False), (True, 2, False), (False, 1, False), (False, 2, False), (False, 2, True), (False, 4, True)}
    assert kinds(NORM) == rows and kinds(NORM_ODD) == rows
    assert kinds(NORM_BACKWARD) == {(False, 1, False), (False, 2, False), (False, 2, True), (False, 0, True)}
