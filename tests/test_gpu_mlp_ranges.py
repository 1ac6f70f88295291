"""GPU: layer norm and projections with an epilogue over whole ranges of values
and sizes: the activations and their slopes at every finite 16-bit argument, gradients that
binary orders divide, tensors of more than 2^31 elements, one tensor as both
operands, codes without a type, workspaces of just their size.

Tolerances of the activations count roundings, u = 2^-24 each.  GELU: exp's
argument z^2 / 2 is off by z^2 u at most, and R, exp, the reciprocal and the
products by 16 u.  SiLU and the tanh form are s z with s = 1 / (1 + t), t = e^-w: w
has 6 roundings (none for SiLU), t is off by (6 |w| + 4) u of itself and s by
1 - s of that and 3 u; 1 - s, where the slope takes it, is off by what s is and
one rounding (or, where t is under 2^-26, by t).  TINY: two of binary32's
smallest steps."""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
from gpu_util import G, TORCH_HP
from test_gpu_ffn import D, codes, gen_of, near, out_tol, rand, up, w64, x64
from test_gpu_layernorm import U, layernorm64
from test_gpu_linear_act import ACTS, operands, unary64

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -148


def every_finite(dt):
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TORCH_HP[dt])
    return v[torch.isfinite(v.float())]


def logistic(act, z):
    """(w', |w|, s, 1 - s, the roundings of w) of SiLU's and the tanh form's s = 1 / (1 + e^-w)"""
    if act == "silu":
        return torch.ones_like(z), z.abs(), torch.sigmoid(z), torch.sigmoid(-z), 0
    h, k = z.clamp(-64, 64), 2 * (2 / torch.pi) ** 0.5
    w = k * (h + 0.044715 * h ** 3)
    return k * (1 + 0.134145 * h * h), w.abs(), torch.sigmoid(w), torch.sigmoid(-w), 6


def gelu_parts(z):
    """z^2 (where exp is not 0), Phi(-|z|) and |z| phi(z)"""
    x = z.abs().clamp_max(60.0)
    return x * x, 0.5 * torch.erfc(x / 2 ** 0.5), x * torch.exp(-x * x / 2) / (2 * torch.pi) ** 0.5


def value_tol(act, z, y):
    if act in (None, "relu"):
        return 0 * z
    if act == "gelu":
        x2, tail, _ = gelu_parts(z)
        return (x2 + 16) * U * x2.sqrt() * tail + 2 * U * y.abs() + TINY
    _, w, s, s1, c = logistic(act, z)
    return ((c * w + 4) * s1 + 6) * U * y.abs() + TINY


def slope64(act, z):
    if act == "silu":
        s, s1 = torch.sigmoid(z), torch.sigmoid(-z)
        return s * (1 + z * s1)
    if act == "gelu_tanh":
        w1, _, s, s1, _ = logistic(act, z)
        return s * (1 + z.clamp(-64, 64) * s1 * w1)
    return unary64(act, z)[1]


def slope_tol(act, z, d):
    if act in (None, "relu"):
        return 0 * z
    if act == "gelu":
        x2, tail, dens = gelu_parts(z)
        return (x2 + 16) * U * (tail + dens) + 2 * U * d.abs()
    w1, w, s, s1, c = logistic(act, z)
    h = z.abs().clamp_max(64.0)
    rs = ((c * w + 4) * s1 + 3) * U                         # of s, relative
    one = torch.minimum(torch.full_like(s, 2 * U), 4 * s1)  # of 1 - s, besides
    return s * (rs * (1 + h * w1 * s1) + h * w1 * (s * rs + one + 4 * U * s1)) + 4 * U * d.abs()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 40])
def test_values_at_every_argument(act, dt, M):
    """without a contraction z is the bias itself"""
    b = every_finite(dt)
    E, N = torch.float8_e4m3fn, b.numel()
    x, w, none = (torch.empty(r, 0, dtype=t, device="cuda") for r, t in ((M, E), (N, E), (0, torch.float32)))
    y, z = fq.linear_act_fp8(x, none, w, none, up(b), act, out=tuple(G.empty((M, N), dtype=torch.float32) for _ in range(2)))
    z64 = b.to(D)
    assert torch.equal(z.cpu(), b.float().expand(M, N))
    if act == "gelu_tanh":                                  # far arguments: the cube leaves no range
        want = z64 * logistic(act, z64)[2]
    else:
        want = unary64(act, z64)[0]
    near(y, want.expand(M, N), value_tol(act, z64, want).expand(M, N), "y")
    far = torch.tensor([float("-inf"), float("inf"), float("nan")])
    y, _ = fq.linear_act_fp8(x, none, w[:3], none, up(far), act, ret_type=torch.float32)
    y = y.cpu()
    assert (y[:, 0] == (0 if act else float("-inf"))).all() and (y[:, 1] == float("inf")).all() and torch.isnan(y[:, 2]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("top", [1.0, 2.0 ** 100])
def test_slopes_at_every_argument(act, dt, top):
    """one row: dbias is dy times the slope, which a large dy shows far down"""
    if dt == "f16" and top > 1:
        top = 2.0 ** 15
    b = every_finite(dt)
    z64, N = b.to(D), b.numel()
    dy = torch.full((1, N), top).to(b.dtype)
    db = G.empty(N, dtype=torch.float32)
    E = torch.float8_e4m3fn
    none = torch.empty(0, device="cuda")
    ws = G.empty(fq.fp8q_linear_act_backward_workspace_bytes(1, N, 0), dtype=torch.uint8)
    fq.fp8q_linear_act_backward(up(dy), up(b.view(1, N)), torch.empty(1, 0, dtype=E, device="cuda"), none,
                                torch.empty(N, 0, dtype=E, device="cuda"), none, None, None, db, act, ws)
    d = slope64(act, z64)
    near(db, top * d, top * slope_tol(act, z64, d) + TINY, "dbias")
    if act:
        far = torch.tensor([[float("-inf"), float("inf")]]).to(b.dtype)
        fq.fp8q_linear_act_backward(up(dy[:, :2]), up(far), torch.empty(1, 0, dtype=E, device="cuda"), none,
                                    torch.empty(2, 0, dtype=E, device="cuda"), none, None, None, db[:2], act, ws)
        assert db[:2].tolist() == [0.0, top]


FAR = {"silu": -100.0, "gelu": -13.0, "gelu_tanh": -9.0}


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gradients_that_binary_orders_divide(act, dt):
    """Rows (for dx) and columns (for dw) of dz 2^100 apart, by dy and by slopes
    far down, keep the bits that each has by itself."""
    g = gen_of("orders", act, dt)
    M, K, N = 70, 256, 200
    T = TORCH_HP[dt]
    xq, xs, wq, ws = operands(g, M, K, N)
    X, W = x64(xq, xs), w64(wq, ws)
    low, high = (-60, 60) if dt == "bf16" else (-8, 8)
    for axis in (0, 1):
        n = (M, N)[axis]
        order = torch.randint(low, high + 1, (n,), generator=g).to(D)
        far = torch.rand(n, generator=g) < 0.3
        if act != "relu":
            order[far] = 120.0 if dt == "bf16" else 14.0
        shape = (M, 1) if axis == 0 else (1, N)
        dy = ((0.5 + torch.rand(M, N, generator=g, dtype=D)) * 2.0 ** order.view(shape)).to(T)
        z = rand(g, M, N)
        if act != "relu":
            z = torch.where(far.view(shape), torch.full_like(z, FAR[act] if dt == "bf16" else -4.0), z)
        z = z.to(T)
        z64 = z.to(D)
        d = slope64(act, z64)
        dz, ez = dy.to(D) * d, dy.to(D).abs() * slope_tol(act, z64, d)
        a = dz.abs() + ez
        grads = fq.linear_act_fp8_backward(up(dy), up(z), up(xq), up(xs), up(wq), up(ws), act, grad_type=torch.float32)
        A, B, got = (a, W.abs(), grads[0]) if axis == 0 else (a.t(), X.abs(), grads[1])
        want = dz @ W if axis == 0 else dz.t() @ X
        # each operand's rounding to f16, the additions, f16's smallest step below each row's exponent
        err = (A @ B) * (2.0 ** -10 + 2.0 ** -20 + (A.shape[1] + 128) * 2.0 ** -23)
        err = err + 2.0 ** -33 * (A.amax(1, keepdim=True) * B.sum(0, keepdim=True) + B.max() * A.sum(1, keepdim=True))
        err = err + (ez if axis == 0 else ez.t()) @ B
        near(got, want, out_tol(want, dt if axis == 0 else "f32", err), ("dx", "dw")[axis])
        assert dt == "f16" or float(want.abs().max()) > 2.0 ** 50


def test_infinite_and_nan_arguments_reach_their_row_and_column():
    """z of the activations where the forward pass left infinities and NaN"""
    g = gen_of("zinf")
    M, K, N = 40, 128, 96
    args = [up(t) for t in operands(g, M, K, N)]
    dy, z = rand(g, M, N).bfloat16(), rand(g, M, N).bfloat16()
    dy[5] = 0.0
    for act in ACTS[1:]:
        want = fq.linear_act_fp8_backward(up(dy), up(z), *args, act)
        for bad in (float("nan"), float("inf"), float("-inf")):
            zb = z.clone()
            zb[5, 7] = bad
            got = fq.linear_act_fp8_backward(up(dy), up(zb), *args, act)
            rows, cols = torch.arange(M) != 5, torch.arange(N) != 7
            assert torch.equal(got[0].cpu()[rows], want[0].cpu()[rows])
            assert torch.equal(got[1].cpu()[cols], want[1].cpu()[cols])
            assert torch.equal(got[2].cpu()[cols], want[2].cpu()[cols])
            if bad == bad:                                  # slopes there are 0 and 1
                for a, c in zip(got, want):
                    assert torch.equal(a, c)


@pytest.mark.parametrize("M", [5, 70])
@pytest.mark.parametrize("xf,wf", [("e4m3fn", "e5m2"), ("e5m2", "e4m3fn")])
def test_codes_without_a_type_and_workspaces_of_their_size(M, xf, wf):
    g = gen_of("u8", M)
    K, N = 7168, 256
    xq, xs, wq, ws = (up(t) for t in operands(g, M, K, N, xf, wf))
    b, r = up(rand(g, N)), up(rand(g, M, N).bfloat16())
    bits = [t.view(torch.uint8) for t in (xq, wq)]
    u8 = lambda f, *a, **k: f(bits[0], xs, bits[1], ws, *a, x_fmt=xf, w_fmt=wf, **k)
    size = lambda n: G.empty(n, dtype=torch.uint8)
    y, z = fq.linear_act_fp8(xq, xs, wq, ws, b, "silu", r, keep=torch.float16)
    y2, z2 = torch.empty_like(y), torch.empty_like(z)
    u8(fq.fp8q_linear_act, b, y2, r, z2, "silu", size(fq.fp8q_linear_act_workspace_bytes(M, N, K, False)))
    assert torch.equal(y, y2) and torch.equal(z, z2)
    q, s, z = fq.linear_act_fp8_cast(xq, xs, wq, ws, b, "gelu", keep=torch.float16)
    q2, s2 = torch.empty_like(q).view(torch.uint8), torch.empty_like(s)
    u8(fq.fp8q_linear_act_cast, b, q2, s2, z2, "gelu", "e4m3fn", size(fq.fp8q_linear_act_workspace_bytes(M, N, K, True)))
    assert torch.equal(q.view(torch.uint8), q2) and torch.equal(s, s2) and torch.equal(z, z2)
    dy = up(rand(g, M, N).half())
    want = fq.linear_act_fp8_backward(dy, z, xq, xs, wq, ws, "gelu")
    got = fq.linear_act_fp8_backward(dy, z, bits[0], xs, bits[1], ws, "gelu", x_fmt=xf, w_fmt=wf)
    assert all(torch.equal(a, c) for a, c in zip(want, got))


@pytest.mark.parametrize("rows,cols", [(5, 7168), (300, 200), (3, 1003), (2, 33333)])
def test_one_tensor_as_x_and_residual(rows, cols):
    g = gen_of("twice", cols)
    x, w, b = rand(g, rows, cols).bfloat16(), (1 + rand(g, cols)).bfloat16(), rand(g, cols).bfloat16()
    want = fq.layernorm(up(x), up(w), up(b), up(x))
    xd = up(x)
    new = lambda: G.empty(rows, dtype=torch.float32)
    y = G.empty((rows, cols), dtype=torch.bfloat16)
    got = fq.layernorm(xd, up(w), up(b), xd, out=(y, xd, new(), new()))
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    assert torch.equal(xd.cpu(), (x.float() * 2).bfloat16())


@pytest.mark.parametrize("cols", [7168, 7171])
def test_layernorm_offsets_past_32_bits(cols):
    """rows at the far end are what a call on them alone gives; dweight and dbias
    are the sums over all"""
    rows = 2 ** 31 // cols + 300
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w, b = up((1 + rand(gen_of("w"), cols)).bfloat16()), up(rand(gen_of("b"), cols).bfloat16())
    at = torch.tensor([0, 511, rows // 2, rows - 301, rows - 300, rows - 299, rows - 1], device="cuda")
    some = x[at].clone()
    y, _, mean, rstd = fq.layernorm(x, w, b)
    y1, _, m1, r1 = fq.layernorm(some, w, b)
    assert torch.equal(y[at], y1) and torch.equal(mean[at], m1) and torch.equal(rstd[at], r1)
    # dy = y, over which dx is written
    n = 64
    part = lambda t: t[:, :n].contiguous().double()
    dyn, nn = part(y), (part(x) - mean.double()[:, None]) * rstd.double()[:, None]
    want, size = ((dyn * nn).sum(0), dyn.sum(0)), ((dyn * nn).abs().sum(0), dyn.abs().sum(0))
    del dyn, nn
    dx1, _, _ = fq.layernorm_backward(y1, some, w, m1, r1)
    wf = w.float()
    dx, dw, db = fq.layernorm_backward(y, x, wf, mean, rstd, out=(y, torch.empty_like(wf), torch.empty_like(wf)))
    assert torch.equal(dx[at], dx1)
    depth = 1.01 * (rows // 512 + 1 + 16 + 6 + 3) * U
    for got, c, a in zip((dw, db), want, size):
        near(got[:n], c.cpu(), a.cpu() * depth + TINY, "sums over the rows")


def test_backward_offsets_past_32_bits():
    """dy, z and the operands made of them hold more than 2^31 elements; few rows
    have a gradient"""
    M, K, N = (1 << 20) + 77, 128, 2184
    g = gen_of("farb")
    rows = torch.tensor([0, 255, 983039, 983040, M - 78, M - 77, M - 1])
    n = len(rows)
    xq, xr = codes(g, n, K, "e4m3fn", n)
    wq, ws = codes(g, N, K, "e4m3fn", 18)
    d1, z1 = rand(g, n, N).bfloat16(), rand(g, n, N).bfloat16()
    x = torch.full((M, K), 0x30, dtype=torch.uint8, device="cuda")
    xs = torch.full((M, 1), 0.5, device="cuda")
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    z = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    at = rows.cuda()
    x[at], xs[at], dy[at], z[at] = xq.view(torch.uint8).cuda(), xr.cuda(), d1.cuda(), z1.cuda()
    dx, dw, db = fq.linear_act_fp8_backward(dy, z, x.view(torch.float8_e4m3fn), xs, up(wq), up(ws), "gelu",
                                            grad_type=torch.float32)
    X, W, z64 = x64(xq, xr), w64(wq, ws), z1.to(D)
    s = slope64("gelu", z64)
    dz, ez = d1.to(D) * s, d1.to(D).abs() * slope_tol("gelu", z64, s)
    a = dz.abs() + ez
    eps = 2.0 ** -10 + 2.0 ** -20
    floor = lambda A, B: 2.0 ** -33 * (A.amax(1, keepdim=True) * B.sum(0, keepdim=True) + B.max() * A.sum(1, keepdim=True))
    ex = a @ W.abs() * (eps + (N + 128) * 2.0 ** -23) + floor(a, W.abs()) + ez @ W.abs()
    near(dx[at], dz @ W, out_tol(dz @ W, "bf16", ex), "dx")
    # X' is below 2^15 with the scales of all rows
    big = X.abs().clamp_min(0.5 * 1.0)
    ew = a.t() @ X.abs() * (eps + (n + 128) * 2.0 ** -23) + floor(a.t(), big) + ez.t() @ X.abs()
    near(dw, dz.t() @ X, out_tol(dz.t() @ X, "f32", ew), "dw")
    near(db, dz.sum(0), a.sum(0) * 40 * U + ez.sum(0) + TINY, "dbias")
    dx[at] = 0
    assert not dx.any()


def test_h_without_a_residual_is_a_copy():
    g = gen_of("copy")
    for cols in (200, 1003, 33333):
        x, w = up(rand(g, 5, cols).bfloat16()), up(rand(g, cols).bfloat16())
        h = G.full((5, cols), 7.0, dtype=torch.bfloat16)
        new = lambda: G.empty(5, dtype=torch.float32)
        y, h2, _, _ = fq.layernorm(x, w, out=(torch.empty_like(x), h, new(), new()))
        assert h2 is h and torch.equal(h, x) and torch.equal(y, fq.layernorm(x, w)[0])


def test_batches_of_more_dimensions():
    """[2, 3, K] is the six rows of [6, K]"""
    g = gen_of("3d")
    K, N = 256, 384
    x, r = up(rand(g, 6, K).bfloat16()), up(rand(g, 6, N).bfloat16())
    nw, b = up(rand(g, K).bfloat16()), up(rand(g, N).bfloat16())
    w = [up(t) for t in operands(g, 1, K, N)[2:]]

    def run(x, r):
        q, s, h, mean, rstd = fq.layernorm_cast(x, nw, None, x)
        y, _ = fq.linear_act_fp8(q, s, *w, b, None, r)
        p, ps, z = fq.linear_act_fp8_cast(q, s, *w, b, "silu", keep=torch.bfloat16)
        dn, dw, db = fq.linear_act_fp8_backward(r, z, q, s, *w, "silu")
        return (q, s, h, y, p, ps, z, dn, dw, db, *fq.layernorm_backward(dn, h, nw, mean, rstd, x))

    flat, deep = run(x, r), run(x.view(2, 3, K), r.view(2, 3, N))
    for a, c in zip(flat, deep):
        assert torch.equal(a.view(torch.uint8).flatten(), c.view(torch.uint8).flatten())
    for i, last in ((0, K), (2, K), (3, N), (4, N), (6, N), (7, K), (10, K)):
        assert deep[i].shape == (2, 3, last)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1, 7, 128, 130, 384, 1000, 5001, 7168, 20001, 40001])
def test_constant_rows_leave_nothing(cols, dt):
    """every element is its row's mean: y is the bias itself, and without one a
    cast per row is zeros with the scale of zeros, whose amax counts as 1"""
    g = gen_of("constant", cols)
    x = (0.5 * rand(g, 300, 1)).to(TORCH_HP[dt]).expand(300, cols).contiguous()
    w, b = (1 + 0.2 * rand(g, cols)).to(x.dtype), (0.2 * rand(g, cols)).to(x.dtype)
    y, _, _, _ = fq.layernorm(up(x), up(w), up(b))
    assert torch.equal(y.cpu(), b.expand(300, cols))
    q, s, _, _, _ = fq.layernorm_cast(up(x), up(w), per_channel_scale=True)
    assert not q.float().any()
    assert torch.equal(s.cpu(), torch.ones(300) / 448.0)
