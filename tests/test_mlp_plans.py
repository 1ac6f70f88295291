"""CPU: the sizes of tests/mlp_plans.py reach the kernels they are meant to, and
together every variant of layer norm and of the products that begin with the
rest's steps."""
import heapq
import random
import shutil

import pytest

from ffn_plans import Plans
from mlp_plans import ACT, ALONE, ALONE_REST, BACKWARD, BACKWARD_REST, LAYERNORM, LAYERNORM_BACKWARD, MlpPlans


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    return Plans(tmp_path_factory.mktemp("plan"))


def test_backward_variants(plans, tmp_path):
    P = MlpPlans(tmp_path)
    for rest, table in ((False, BACKWARD), (True, BACKWARD_REST)):
        for key, want in table.items():
            assert P.backward(*key, rest) == want, key
        for product in (0, 1):
            got = {(p[product][0], p[product][1] > 1) for p in table.values() if p[product][2] > 2 and not p[2]}
            assert got == {(bm, s) for bm in (64, 128, 256) for s in (False, True)} | {(192, False)}, (rest, product)
        both = {p[0][0] for p in table.values() if p[2] and p[0][2] > 2 and p[1][2] > 2}
        assert both == {128, 192, 256}
    kinds = set()
    for (M, _, N), plan in BACKWARD_REST.items():
        for (_, splits, kper), C in zip(plan, ((N + 127) // 128 * 128, (M + 127) // 128 * 128)):
            for i in range(splits):
                first, end = i * kper, min((i + 1) * kper, C // 64 + C // 128)
                kinds.add("rest" if end <= C // 128 else "f16" if first >= C // 128 else "both")
    assert kinds == {"rest", "both", "f16"}


def test_layernorm_variants(plans, tmp_path):
    plan = MlpPlans(tmp_path).layernorm
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


def test_projection_tiles_cover_every_output_once(plans, tmp_path):
    """random sizes: the tiles of both widths cover the outputs, none begins past
    the end, and a split's blocks cover the contraction"""
    P = MlpPlans(tmp_path)
    rng = random.Random(5)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    seen = set()
    for _ in range(20000):
        M, N, K, ex = log(1, 20000), log(1, 40000), 128 * log(1, 200), rng.random() < 0.4
        bm, splits, kper, tm, tn, tn2, nt2 = P.act(M, K, N, ex)
        if M <= 16:
            assert bm == 0 and splits == 1
            continue
        key = (M, N, K, ex)
        assert bm in ((64, 128) if ex else (64, 128, 256)), key
        assert (tm - 1) * bm < M <= tm * bm, key
        last = 256 * tn if tn2 == 0 else 256 * tn + 64 * nt2 * (tn2 - 1)
        assert (last - 256 if tn2 == 0 else last) < N <= 256 * tn + 64 * nt2 * tn2, key
        assert splits == 1 or (tn2 == 0 and nt2 == 4), key
        assert (splits - 1) * kper < K // 128 <= splits * kper, key
        assert nt2 == 4 and tn2 == 0 or nt2 == 2 and bm == 64 and tn == 0 or nt2 == 3 and bm == 256 and not ex, key
        seen.add((bm, nt2, ex, splits > 1))
    assert {(bm, nt2, ex) for bm, nt2, ex, _ in seen} == {(64, 4, True), (128, 4, True), (64, 2, True), (64, 4, False),
                                                         (128, 4, False), (256, 4, False), (64, 2, False), (256, 3, False)}


def test_projection_variants(plans, tmp_path):
    P = MlpPlans(tmp_path)
    for key, want in ACT.items():
        bm, splits, kper, _, tn, tn2, nt2 = P.act(*key)
        assert (bm, splits, kper, tn, tn2, nt2) == want, key
        assert kper > (2 if bm == 256 else 3)
    whole = {(bm, nt2, key[3]) for key, (bm, splits, _, _, _, nt2) in ACT.items() if splits == 1}
    assert whole == {(64, 2, True), (64, 2, False), (64, 4, True), (64, 4, False), (128, 4, True), (128, 4, False),
                     (256, 4, False), (256, 3, False)}
    # casts of every kind with binary32 sums: whole groups
    assert {v[0] for k, v in ACT.items() if k[3] and k[2] % 128 == 0} == {64, 128}


def test_mixed_rounds(plans, tmp_path):
    """against workgroups that take the next tile as they end"""
    P = MlpPlans(tmp_path)
    rng = random.Random(6)
    for _ in range(300):
        whole, part, r = rng.randrange(0, 1500), rng.randrange(0, 1500), rng.uniform(0.6, 0.95)
        ends = [0.0] * 256
        for t in [1.0] * whole + [r] * part:
            heapq.heappush(ends, heapq.heappop(ends) + t)
        assert abs(P.mixed_rounds(whole, part, r) - max(ends)) < 1e-4 * (1 + max(ends)), (whole, part, r)


def test_one_gradient_without_the_other(plans, tmp_path):
    """Of a joint launch's products one alone takes the height of its own least
    time, which the joint one need not be, unsplit as there."""
    P = MlpPlans(tmp_path)
    for rest, table in ((False, ALONE), (True, ALONE_REST)):
        for key, want in table.items():
            assert P.backward(*key, rest)[2] and P.alone(*key, rest) == want, key
    assert {h for v in ALONE.values() for h in v} == {64, 128, 192, 256}
    rng = random.Random(8)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    both = slower = 0
    for _ in range(4000):
        M, K, N, rest = log(32, 5000), 128 * log(1, 60), log(32, 6000), rng.random() < 0.5
        dx, dw, joint = P.backward(M, K, N, rest)
        if not joint:
            continue
        both += 1
        for (bm, splits, steps), h, rows in zip((dx, dw), P.alone(M, K, N, rest), (M, N)):
            assert splits == 1
            best = min(P.time16(rows, K, steps, b) for b in (64, 128, 192, 256))
            assert P.time16(rows, K, steps, h) == best
            slower += P.time16(rows, K, steps, bm) > 1.2 * best
    assert both > 100 and slower > 50                       # what the joint height would cost


def test_layernorm_backward_variants(plans, tmp_path):
    """the sizes that run on the GPU reach every instance, with more rows than workgroups"""
    plan = MlpPlans(tmp_path).layernorm_backward
    for key, want in LAYERNORM_BACKWARD.items():
        assert plan(*key) == want and key[0] > want[2], key
    # type, vectors a thread, and the size of the workgroup that its launch bounds name
    got = {(k[2] == "f32", v, t > 512) for k, (v, t, _) in LAYERNORM_BACKWARD.items()}
    assert got == {(f, v, big) for f in (False, True) for v, big in ((1, False), (2, False), (2, True), (0, True))}
    # 16-bit rows of the most threads ask for 128 KB of LDS
    assert max(2 * v * 8 * t * 4 for (_, _, dt), (v, t, _) in LAYERNORM_BACKWARD.items() if dt != "f32") == 128 << 10
