"""GPU: projections with bias, activation and residual in their epilogue, and
with the group cast (include/fp8q_mlp.h), against their definitions in binary64
on the CPU: one row to many, every tiling and split, odd widths, views, each
activation at its tails, in place, graphs and streams; their backward pass also
against differences.  Tolerances as in test_gpu_ffn.py: the sums' bound
(sum_err), the slope of the activation, one rounding of each output."""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
from ffn_plans import FORWARD
from mlp_plans import ACT, BACKWARD, BACKWARD_REST
from gpu_util import G, TORCH_HP
from test_gpu_ffn import BWD, D, FP8, act64, bwd_err, cast_close, codes, gen_of, near, out_tol, rand, sum_err, up, w64, x64

pytestmark = pytest.mark.gpu

ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def unary64(name, z):
    """(the activation, its derivative)"""
    if name is None:
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if name == "gelu":                                      # erfc keeps the tail that 1 + erf cancels
        p = 0.5 * torch.erfc(-z / 2 ** 0.5)
        return z * p, p + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    return act64(name, z)


def value_err(act, z, y, ez):
    """error of act(z) from that of z: slopes are at most 1.13, and the
    activation itself is within a few binary32 roundings of |y|, or of what
    vanishes times |z|"""
    if act is None:
        return ez
    if act == "relu":
        return ez
    return 1.13 * ez + (y.abs() + z.abs() * 2.0 ** -2) * 2.0 ** -20


def operands(g, M, K, N, xf="e4m3fn", wf="e4m3fn"):
    xq, xs = codes(g, M, K, xf, M)
    wq, ws = codes(g, N, K, wf, (N + 127) // 128)
    xs = xs * (0.3 / max(K, 1) ** 0.5)
    return xq, xs, wq, ws


def product(g, M, K, N, bias, xf="e4m3fn", wf="e4m3fn", exact=True, bt=torch.float32):
    xq, xs, wq, ws = operands(g, M, K, N, xf, wf)
    X, W = x64(xq, xs), w64(wq, ws)
    b = rand(g, N).to(bt) if bias else None
    z = X @ W.t() + (0 if b is None else b.to(D))
    ez = sum_err(X.abs(), W.abs(), K, exact) + z.abs() * 2.0 ** -24
    return (up(xq), up(xs), up(wq), up(ws)), b, z, ez


def linear_case(M, K, N, dt, act, bias, res, keep, xf="e4m3fn", wf="e4m3fn", bt=None):
    g = gen_of(M, K, N, dt, act)
    T = TORCH_HP[dt]
    exact = dt == "f32" or keep == "f32" or M <= 16        # else sums on the fp8 instruction
    args, b, z, ez = product(g, M, K, N, bias, xf, wf, exact, bt or T)
    r = rand(g, M, N).to(T) if res else None
    y = unary64(act, z)[0]
    ey = value_err(act, z, y, ez)
    want = y if r is None else y + r.to(D)
    zo = G.empty((M, N), dtype=TORCH_HP[keep]) if keep else None
    yo, zo = fq.linear_act_fp8(*args, None if b is None else up(b), act, None if r is None else up(r),
                               out=(G.empty((M, N), dtype=T), zo))
    near(yo, want, out_tol(want, dt, ey + want.abs() * 2.0 ** -24), "y")
    if keep:
        near(zo, z, out_tol(z, keep, ez), "z")
    if res:                                                 # y over the residual: the same bits
        rd = up(r)
        assert torch.equal(fq.linear_act_fp8(*args, None if b is None else up(b), act, rd, out=(rd, None))[0],
                           fq.linear_act_fp8(*args, None if b is None else up(b), act, up(r),
                                             out=(torch.empty_like(rd), None))[0])


SIZES = [(1, 128, 1), (1, 7168, 33), (15, 1152, 130), (17, 256, 16), (33, 1152, 257), (64, 2176, 100), (65, 256, 129),
         (70, 4096, 128), (200, 4224, 300), (1000, 512, 3001), (1700, 384, 4104), (4200, 128, 4096), (5, 384, 9001),
         (13, 1280, 8500), (8, 128, 40), (9, 2048, 4100), (300, 0, 70), (3, 0, 20)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dt,act,bias,res,keep,xf,wf", [
    ("bf16", None, True, True, None, "e4m3fn", "e4m3fn"), ("f16", "gelu", True, False, "f16", "e5m2", "e4m3fn"),
    ("f32", "gelu_tanh", True, True, "f32", "e4m3fn", "e5m2"), ("bf16", "silu", False, True, "bf16", "e5m2", "e5m2"),
    ("f16", "relu", True, True, None, "e4m3fn", "e4m3fn"), ("bf16", None, False, False, "f32", "e4m3fn", "e4m3fn")])
def test_linear_act(M, K, N, dt, act, bias, res, keep, xf, wf):
    linear_case(M, K, N, dt, act, bias, res, keep, xf, wf)


@pytest.mark.parametrize("M,K,N", [k[:3] for k in FORWARD if not k[3]])
@pytest.mark.parametrize("act", [None, "gelu"])
def test_every_tiling(M, K, N, act):
    """every tile height, whole and split, of both kinds of sum, past its first steps"""
    exact = {k[:3]: k[4] for k in FORWARD if not k[3]}[(M, K, N)]
    linear_case(M, K, N, "f32" if exact else "bf16", act, True, True, None)


@pytest.mark.parametrize("M,K,N,exact", list(ACT))
@pytest.mark.parametrize("act,res,keep", [(None, True, False), ("gelu", False, True), ("silu", True, True)])
def test_every_epilogue(M, K, N, exact, act, res, keep):
    """each kind of tile, with and without a residual and kept pre-activations"""
    dt = "f32" if exact else "f16"
    linear_case(M, K, N, dt, act, True, res, dt if keep else None)


@pytest.mark.parametrize("bt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_bias_types(M, bt):
    for dt in ("bf16", "f32"):
        linear_case(M, 256, 200, dt, "silu", True, False, None, bt=TORCH_HP[bt])


@pytest.mark.parametrize("M,K,N", [(1, 128, 128), (1, 7168, 256), (16, 1152, 384), (17, 640, 128), (17, 3584, 256),
                                   (50, 1152, 1280), (65, 256, 256), (200, 512, 8320), (1000, 640, 4224), (1030, 7168, 128),
                                   (4100, 3584, 128), (300, 128, 640), (5, 0, 128), (90, 0, 256), (9, 7168, 15360),
                                   (3, 256, 36992), (16, 384, 36864), (1, 1024, 4224)])
@pytest.mark.parametrize("act,fmt,keep", [("gelu", "e4m3fn", "bf16"), (None, "e5m2", None), ("relu", "e4m3fn", "f32"),
                                          ("silu", "e5m2", "f16")])
def test_linear_act_cast(M, K, N, act, fmt, keep):
    g = gen_of(M, K, N, act, fmt)
    args, b, z, ez = product(g, M, K, N, True, bt=torch.bfloat16)
    y = unary64(act, z)[0]
    q, s = G.empty((M, N), dtype=FP8[fmt]), G.empty((M, N // 128), dtype=torch.float32)
    zo = G.empty((M, N), dtype=TORCH_HP[keep]) if keep else None
    fq.linear_act_fp8_cast(*args, up(b), act, fmt, out=(q, s, zo))
    cast_close(q, s, y, value_err(act, z, y, ez), fmt, "cast")
    if keep:
        near(zo, z, out_tol(z, keep, ez), "z")


@pytest.mark.parametrize("M", [1, 12, 40, 130, 600])
@pytest.mark.parametrize("N,K", [(256, 512), (251, 512), (256, 7168)])
def test_views(M, N, K):
    """outputs, bias and residual one element into their buffers: the same bits"""
    g = gen_of("views", M, N)
    xq, xs, wq, ws = operands(g, M, K, N)
    args = (up(xq), up(xs), up(wq), up(ws))

    def view(t):
        return G.empty(t.numel() + 1, dtype=t.dtype)[1:].copy_(t.reshape(-1)).view(t.shape)

    for dt in ("bf16", "f32"):
        T = TORCH_HP[dt]
        b, r = rand(g, N).to(T), rand(g, M, N).to(T)
        new = lambda: torch.zeros(M, N).to(T)
        y0, z0 = fq.linear_act_fp8(*args, up(b), "gelu", up(r), out=(up(new()), up(new())))
        y1, z1 = fq.linear_act_fp8(*args, view(b), "gelu", view(r), out=(view(new()), view(new())))
        assert torch.equal(y0, y1) and torch.equal(z0, z1)
    if N % 128 == 0:
        out = lambda o: (G.empty(M * N + 1, dtype=torch.uint8)[o:][: M * N].view(M, N), G.empty((M, 2), dtype=torch.float32), None)
        a, c = (fq.linear_act_fp8_cast(*args, up(b), "gelu", out=out(o)) for o in (0, 1))
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@pytest.mark.parametrize("M", [2, 40, 100])
@pytest.mark.parametrize("act", ACTS)
def test_nan_and_infinity(M, act):
    """an infinite or NaN bias and residual reach their own outputs alone"""
    g = gen_of("nan", M)
    N = 256
    args = [up(t) for t in operands(g, M, 256, N)]
    b, r = rand(g, N), rand(g, M, N)
    clean, _ = fq.linear_act_fp8(*args, up(b), act, up(r), ret_type=torch.float32)
    b2, r2 = b.clone(), r.clone()
    b2[7], b2[9], b2[11] = float("nan"), float("inf"), float("-inf")
    r2[1, 20], r2[1, 21] = float("nan"), float("-inf")
    y, _ = fq.linear_act_fp8(*args, up(b2), act, up(r2), ret_type=torch.float32)
    y, clean = y.cpu(), clean.cpu()
    assert torch.isnan(y[:, 7]).all() and torch.isnan(y[1, 20]) and y[1, 21] == float("-inf")
    assert (y[:, 9] == float("inf")).all()
    if act == "relu":
        assert torch.equal(y[:, 11], r[:, 11])
    keep = torch.ones(N, dtype=torch.bool)
    keep[[7, 9, 11, 20, 21]] = False
    assert torch.equal(y[:, keep], clean[:, keep])


def test_offsets_past_32_bits():
    """outputs, residual and z of more than 2^31 elements: rows at the far end
    are right"""
    M, K, N = (1 << 20) + 77, 128, 2184
    g = gen_of("far")
    x = torch.empty(M, K, dtype=torch.uint8, device="cuda").fill_(0x30)
    xs = torch.full((M, 1), 0.5, device="cuda")
    wq, ws = codes(g, N, K, "e4m3fn", 18)
    b = rand(g, N)
    y = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 255, 983039, 983040, M - 78, M - 77, M - 1])
    xq, xr = codes(g, len(rows), K, "e4m3fn", len(rows))
    x[rows.cuda()] = xq.view(torch.uint8).cuda()
    xs[rows.cuda()] = xr.cuda()
    fq.linear_act_fp8(x.view(torch.float8_e4m3fn), xs, up(wq), up(ws), up(b), "gelu", y, out=(y, None))
    X, W = x64(xq, xr), w64(wq, ws)
    z = X @ W.t() + b.to(D)
    v = unary64("gelu", z)[0]
    err = value_err("gelu", z, v, sum_err(X.abs(), W.abs(), K, False) + z.abs() * 2.0 ** -24)
    near(y[rows.cuda()], v + 1, out_tol(v + 1, "bf16", err + 2.0 ** -23), "far rows")


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------

def backward_case(M, K, N, dt, gdt, act, xf="e4m3fn", wf="e4m3fn", only=True):
    g = gen_of(M, K, N, act, "b")
    T, GT = TORCH_HP[dt], TORCH_HP[gdt]
    xq, xs, wq, ws = operands(g, M, K, N, xf, wf)
    X, W = x64(xq, xs), w64(wq, ws)
    dy = (0.05 * rand(g, M, N)).to(T)
    z = None if act is None else (2 * rand(g, M, N)).to(T)
    slope = torch.ones(1, dtype=D) if act is None else unary64(act, z.to(D))[1]
    dz = dy.to(D) * slope
    # the slope's own binary32 evaluation: a few roundings of max(1, |z|) terms
    ez = torch.zeros(1, dtype=D) if act in (None, "relu") else dy.to(D).abs() * 2.0 ** -19 * (1 + z.to(D).abs())
    args = (up(dy), None if z is None else up(z), up(xq), up(xs), up(wq), up(ws))
    out = (G.empty((M, K), dtype=T), G.empty((N, K), dtype=GT), G.empty(N, dtype=GT))
    dx, dw, db = fq.linear_act_fp8_backward(*args, act, out=out)
    a = dz.abs() + ez
    near(dx, dz @ W, out_tol(dz @ W, dt, bwd_err(a, W.abs(), N + 128) + (ez + 0 * dz) @ W.abs()), "dx")
    near(dw, dz.t() @ X, out_tol(dz.t() @ X, gdt, bwd_err(a.t(), X.abs(), M + 128) + (ez + 0 * dz).t() @ X.abs()), "dw")
    # 16 rows and 4 waves of a tile, then M / 64 tiles over 32 lanes
    depth = 8 + M // 2048 + 6
    near(db, dz.sum(0), out_tol(dz.sum(0), gdt, a.sum(0) * depth * 2.0 ** -24 + (ez + 0 * dz).sum(0)), "dbias")
    if not only:
        return
    # each alone, with a workspace of just its size between guards: the same bits
    ws_ = G.empty(fq.fp8q_linear_act_backward_workspace_bytes(M, N, K), dtype=torch.uint8)
    for i in range(3):
        o = [torch.empty_like(t) if j == i else None for j, t in enumerate(out)]
        fq.fp8q_linear_act_backward(*args, *o, act, ws_)
        assert torch.equal(o[i], out[i]), i


@pytest.mark.parametrize("M,K,N", BWD)
@pytest.mark.parametrize("dt,gdt,act,xf,wf", [("bf16", "bf16", "gelu", "e4m3fn", "e4m3fn"), ("f16", "f16", "silu", "e5m2", "e4m3fn"),
                                              ("f16", "f32", None, "e4m3fn", "e5m2"), ("bf16", "f32", "relu", "e5m2", "e5m2"),
                                              ("bf16", "bf16", None, "e4m3fn", "e4m3fn"), ("f16", "f16", "gelu_tanh", "e4m3fn", "e4m3fn")])
def test_backward(M, K, N, dt, gdt, act, xf, wf):
    backward_case(M, K, N, dt, gdt, act, xf, wf)


@pytest.mark.parametrize("M,K,N", list(BACKWARD))
def test_backward_every_tiling(M, K, N):
    backward_case(M, K, N, "bf16", "f32", "gelu", only=M * K * N < 5e8)


@pytest.mark.parametrize("M,K,N", list(BACKWARD_REST))
def test_backward_every_tiling_with_a_rest(M, K, N):
    """f16 gradients through an activation: the contraction begins with the
    rest's steps, whole and split"""
    backward_case(M, K, N, "f16", "f16", "gelu", only=M * K * N < 5e8)


def test_f16_gradients_keep_their_bits():
    """The rest of dz that f16 leaves goes through the product: in root mean
    square within 1.5 times the outputs' own rounding (a quarter of 2^-11 over
    sqrt(3) of f16's smallest step to largest, 2.1e-4)."""
    g = gen_of("bits")
    M, K, N = 500, 640, 700
    xq, xs, wq, ws = operands(g, M, K, N)
    dy, z = (0.05 * rand(g, M, N)).half(), (2 * rand(g, M, N)).half()
    X, W = x64(xq, xs), w64(wq, ws)
    dz = dy.to(D) * unary64("gelu", z.to(D))[1]
    dx, dw, _ = fq.linear_act_fp8_backward(up(dy), up(z), up(xq), up(xs), up(wq), up(ws), "gelu")
    for got, want in ((dx, dz @ W), (dw, dz.t() @ X)):
        assert float((got.cpu().to(D) - want).norm() / want.norm()) < 3.2e-4


def test_gradients_against_differences():
    """sum(dy * act(X W^T + b)) along each gradient, in binary64, by central
    differences: bf16 gradients, within 2^-8 of their value an element, less in
    norm; z as the forward pass keeps it."""
    g = gen_of("lad")
    M, K, N = 70, 256, 200
    xq, xs, wq, ws = operands(g, M, K, N)
    X, W, b = x64(xq, xs), w64(wq, ws), rand(g, N).bfloat16()
    dy = rand(g, M, N).bfloat16()
    for act in ("silu", "gelu", "gelu_tanh", None):
        f = lambda X, W, b: (dy.to(D) * unary64(act, X @ W.t() + b)[0]).sum()
        _, z = fq.linear_act_fp8(up(xq), up(xs), up(wq), up(ws), up(b), act, keep=torch.bfloat16)
        grads = fq.linear_act_fp8_backward(up(dy), z, up(xq), up(xs), up(wq), up(ws), act)
        for i, grad in enumerate(grads):
            d = grad.cpu().to(D)
            step = 1e-5 * d / d.norm()
            at = lambda t: f(*[v.to(D) + (t if j == i else 0) for j, v in enumerate((X, W, b))])
            slope = (at(step) - at(-step)) / 2e-5
            assert abs(slope - d.norm()) <= 2.0 ** -6 * d.norm(), (act, i, float(slope), float(d.norm()))


@pytest.mark.parametrize("act", [None, "gelu"])
def test_backward_empty(act):
    E = torch.float8_e4m3fn
    e = lambda r, c: torch.zeros(r, c, device="cuda").to(E)
    f = lambda r, c: torch.zeros(r, c, device="cuda")
    b = lambda r, c: torch.zeros(r, c, device="cuda", dtype=torch.bfloat16)
    for gd in (torch.bfloat16, torch.float32):
        dw, db = G.full((70, 128), 5.0, dtype=gd), G.full((70,), 5.0, dtype=gd)
        fq.fp8q_linear_act_backward(b(0, 70), b(0, 70), e(0, 128), f(0, 1), e(70, 128), f(1, 1), b(0, 128), dw, db, act)
        assert (dw == 0).all() and (db == 0).all()
    dx = G.full((9, 128), 5.0, dtype=torch.bfloat16)
    fq.fp8q_linear_act_backward(b(9, 0), b(9, 0), e(9, 128), f(9, 1), e(0, 128), f(0, 1), dx, b(0, 128), None, act)
    assert (dx == 0).all()
    # no contraction: dbias is still the sum of dz
    dy, z = rand(gen_of("k0"), 70, 200).bfloat16(), rand(gen_of("k1"), 70, 200).bfloat16()
    db = G.empty(200, dtype=torch.float32)
    ws = G.empty(fq.fp8q_linear_act_backward_workspace_bytes(70, 200, 0), dtype=torch.uint8)
    fq.fp8q_linear_act_backward(up(dy), up(z), e(70, 0), f(70, 0), e(200, 0), f(2, 0), None, None, db, act, ws)
    dz = dy.to(D) * (1 if act is None else unary64(act, z.to(D))[1])
    near(db, dz.sum(0), dy.to(D).abs().sum(0) * (2.0 ** -19 * 4 + 2.0 ** -20), "dbias")


def test_backward_nan_stays_in_its_row_and_column():
    g = gen_of("bn")
    M, K, N = 70, 256, 96
    args = [up(t) for t in operands(g, M, K, N)]
    dy, z = (1e-6 * rand(g, M, N)).bfloat16(), rand(g, M, N).bfloat16()
    for act in (None, "gelu"):
        keep = dy.clone()
        keep[5] = 0.0
        want = fq.linear_act_fp8_backward(up(keep), up(z), *args, act)
        for bad in (float("nan"), float("inf")):
            d = keep.clone()
            d[5, 7] = bad
            dx, dw, db = fq.linear_act_fp8_backward(up(d), up(z), *args, act)
            rows, cols = torch.arange(M) != 5, torch.arange(N) != 7
            assert not torch.isfinite(dx[5]).any() and torch.equal(dx.cpu()[rows], want[0].cpu()[rows])
            assert not torch.isfinite(dw[7]).all() and torch.equal(dw.cpu()[cols], want[1].cpu()[cols])
            assert not torch.isfinite(db[7]) and torch.equal(db.cpu()[cols], want[2].cpu()[cols])


# ---------------------------------------------------------------------------
# together, on streams and in graphs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 40, 200])
def test_block_on_streams_in_graphs_and_two_at_once(M):
    """The whole block twice, two at once on two streams, and replayed from a
    graph with eager calls between: the same bits every time."""
    g = gen_of("lasg", M)
    K, N = 512, 384
    x, r = up(rand(g, M, K).bfloat16()), up(rand(g, M, K).bfloat16())
    nw, nb, b1, b2 = (up(t.bfloat16()) for t in (1 + 0.1 * rand(g, K), rand(g, K), rand(g, N), rand(g, K)))
    w1, w2 = [up(t) for t in operands(g, 1, K, N)[2:]], [up(t) for t in operands(g, 1, N, K)[2:]]
    w1[1] *= 0.05
    w2[1] *= 0.05

    def step():
        q, s, h, mean, rstd = fq.layernorm_cast(x, nw, nb, r)
        p, ps, z = fq.linear_act_fp8_cast(q, s, *w1, b1, "gelu", keep=torch.bfloat16)
        y, _ = fq.linear_act_fp8(p, ps, *w2, b2, residual=h)
        dp, dw2, db2 = fq.linear_act_fp8_backward(y, None, p, ps, *w2)
        dn, dw1, db1 = fq.linear_act_fp8_backward(dp, z, q, s, *w1, "gelu")
        dx, dnw, dnb = fq.layernorm_backward(dn, h, nw, mean, rstd, y)
        return q, s, h, mean, rstd, p, ps, z, y, dp, dw2, db2, dn, dw1, db1, dx, dnw, dnb

    want = [t.clone() for t in step()]
    same = lambda out: all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(out, want))
    assert all(torch.isfinite(t.float()).all() for t in want)
    assert same(step())
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(step())
    torch.cuda.synchronize()
    assert all(same(o) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = step()
    for _ in range(3):
        for t in out:
            t.view(torch.uint8).fill_(0x55)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out)
        assert same(step())


def test_example_block_runs():
    """examples/mlp_block.py: the operators together, as a training step and a
    decode step.  Casts to e4m3fn (2^-4 at most, about 2^-5 in root mean square,
    an element) leave the block's own part of the output within a tenth of its
    norm."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(fq.__file__), "examples", "mlp_block.py")
    spec = importlib.util.spec_from_file_location("mlp_block_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    err, same = mod.main(200, 512, 640)
    assert err < 0.1 and same
