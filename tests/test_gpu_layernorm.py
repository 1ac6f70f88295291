"""GPU: layer norm (include/fp8q_mlp.h) against its definition in binary64 on
the CPU, at the widths where it can go wrong: one element, less than a vector,
vectors that end inside the last one, rows held by a wave, a workgroup or in
passes; rows far from zero, constant rows, NaN and infinity; in place, views,
graphs and streams; gradients also against differences.

Tolerances are derived, per element, from how the results are computed, with
u = 2^-24 (one binary32 rounding): a sum of n terms in the kernels' order has at
most `depth(n)` additions on its longest path, so it is within depth(n) u of the
sum of the terms' magnitudes (1.01 covers the second order).
"""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
from gpu_util import G, TORCH_HP
from mlp_plans import LAYERNORM
from test_gpu_ffn import D, FP8, HALF_ULP, TINY, cast_close, gen_of, near, out_tol, rand, up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def depth(cols):
    """additions on the longest path of a sum over a row: a lane's own elements
    (32 in registers, or every 1024th vector), 6 lane steps, 16 waves"""
    return max(32, cols // 1024 + 8) + 6 + 16


def layernorm64(x, r, w, b, eps):
    h = x.to(D) + (0 if r is None else r.to(D))
    mean = h.mean(1)
    rstd = 1 / torch.sqrt((h - mean[:, None]).square().mean(1) + eps)
    return h, mean, rstd, (h - mean[:, None]) * rstd[:, None] * w.to(D) + (0 if b is None else b.to(D))


def bounds(h, mean, rstd, y, w, b, eps, summed):
    """errors of the computed mean, rstd and y.  The mean is m0 + m1: m0 is off
    the mean by off0, which the differences d = h - m0 carry without loss, and
    m1 is their mean; h itself has one rounding where it is a sum."""
    gam = 1.01 * depth(h.shape[1]) * U
    row = lambda t: t.mean(1)
    eh = h.abs() * (U if summed else 0.0)
    off0 = gam * row(h.abs()) + row(eh) + 2 * U * mean.abs()
    dev = (h - mean[:, None]).abs()
    d = dev + off0[:, None]
    ed = eh + U * d                                             # d's own error
    em1 = (gam + 2 * U) * row(d) + row(ed)
    emean = em1 + U * mean.abs() + U * off0
    edev = ed + em1[:, None] + U * dev
    evar = (gam + 4 * U) * row(d * d) + 2 * row(d * ed) + 2 * off0 * em1 + 2 * U * off0 ** 2
    var = dev.square().mean(1)
    lo, hi = (var - evar).clamp_min(0.0) + eps, var + evar + eps
    erstd = torch.maximum(1 / torch.sqrt(lo) - rstd, rstd - 1 / torch.sqrt(hi)) + 4 * U / torch.sqrt(lo)
    n = dev * rstd[:, None]
    en = edev * (rstd + erstd)[:, None] + dev * erstd[:, None] + 2 * U * n
    ey = en * w.abs() + 2 * U * (n * w.abs() + (0 if b is None else b.abs())) + U * y.abs()
    return emean, erstd, ey


def forward_case(rows, cols, dt, res, bias, to, fmt="e4m3fn", wf32=False, eps=1e-5, x=None):
    g = gen_of(rows, cols, dt, to)
    T = TORCH_HP[dt]
    if x is None:
        x = 3 * rand(g, rows, cols) + rand(g, rows, 1)
        if rows > 2:
            x[1] = 0.0
        if rows > 3:
            x[2] += 50.0
    x = x.to(T)
    r = rand(g, rows, cols).to(T) if res else None
    wt = torch.float32 if wf32 else T
    w, b = (1 + rand(g, cols)).to(wt), rand(g, cols).to(wt) if bias else None
    h, mean, rstd, y = layernorm64(x, r, w, b, eps)
    emean, erstd, ey = bounds(h, mean, rstd, y, w.to(D), None if b is None else b.to(D), eps, res)
    xd, wd, bd, rd = up(x), up(w), None if b is None else up(b), up(r) if res else None
    ho = G.empty((rows, cols), dtype=T) if res else xd
    mo, so = G.empty(rows, dtype=torch.float32), G.empty(rows, dtype=torch.float32)
    if to == "plain":
        yo = G.empty((rows, cols), dtype=T)
        fq.layernorm(xd, wd, bd, rd, eps, out=(yo, ho, mo, so))
        near(yo, y, out_tol(y, dt, ey), "y")
    else:
        q = G.empty((rows, cols), dtype=FP8[fmt])
        s = G.empty((rows, cols // 128) if to == "group" else (rows,), dtype=torch.float32)
        got = fq.layernorm_cast(xd, wd, bd, rd, eps, fmt, per_channel_scale=to == "row", out=(q, s, ho, mo, so))
        assert got[0] is q
        cast_close(q, s, y, ey, fmt, "cast", groups=to == "group")
    near(mo, mean, emean, "mean")
    near(so, rstd, erstd, "rstd")
    if res:
        near(ho, h, out_tol(h, dt, h.abs() * U), "h")


WHOLE = [(1, 128, "bf16", True), (1, 7168, "bf16", True), (5, 7168, "f32", False), (3, 256, "f16", True),
         (300, 1024, "bf16", True), (260, 512, "f32", True), (700, 640, "f16", False), (2, 16384, "bf16", True),
         (3, 32768, "f16", True), (2, 40960, "bf16", True), (2, 20480, "f32", False), (9, 3200, "f32", True),
         (3, 12288, "f32", True)]
ODD = [(1, 1, "bf16", True), (4, 7, "f32", False), (5, 3, "f32", True), (9, 7, "bf16", True), (3, 8, "f16", False),
       (300, 5, "f16", True), (300, 333, "f16", True), (260, 129, "bf16", False), (5, 5001, "f32", True),
       (3, 8195, "bf16", True), (2, 40001, "f16", True), (2, 33333, "f32", False), (1000, 64, "bf16", True),
       (7, 1501, "bf16", False), (4, 12001, "f32", True), (300, 9, "bf16", True), (300, 517, "f32", True)]


@pytest.mark.parametrize("rows,cols,dt,res", WHOLE)
@pytest.mark.parametrize("fmt,wf32,bias", [("e4m3fn", False, True), ("e5m2", True, False)])
def test_cast_per_group(rows, cols, dt, res, fmt, wf32, bias):
    forward_case(rows, cols, dt, res, bias, "group", fmt, wf32)


@pytest.mark.parametrize("rows,cols,dt,res", ODD + WHOLE[:4])
@pytest.mark.parametrize("fmt,wf32,bias", [("e4m3fn", True, True), ("e5m2", False, False)])
def test_cast_per_row(rows, cols, dt, res, fmt, wf32, bias):
    forward_case(rows, cols, dt, res, bias, "row", fmt, wf32)


@pytest.mark.parametrize("rows,cols,dt,res", ODD + WHOLE)
@pytest.mark.parametrize("wf32,bias", [(True, True), (False, True), (False, False)])
def test_plain(rows, cols, dt, res, wf32, bias):
    forward_case(rows, cols, dt, res, bias, "plain", "e4m3fn", wf32)


@pytest.mark.parametrize("rows,cols,dt", list(LAYERNORM))
@pytest.mark.parametrize("wf32", [False, True])
def test_every_variant(rows, cols, dt, wf32):
    """each kernel past the rows its grid takes at once"""
    for to in ("plain", "row") + (("group",) if cols % 128 == 0 else ()):
        forward_case(rows, cols, dt, rows % 200 == 0, True, to, "e5m2", wf32)


@pytest.mark.parametrize("cols", [200, 4099, 20000, 33333])
def test_rows_far_from_zero(cols):
    """deviations of 1 on rows at 1e6 (16 units in the last place of h), and of
    2^-20 on rows at 1: what the rounded mean alone would lose"""
    g = gen_of("far", cols)
    x = torch.cat([rand(g, 4, cols) + 1e6, rand(g, 4, cols) * 2.0 ** -20 + 1.0, rand(g, 4, cols) - 3e4])
    forward_case(12, cols, "f32", False, True, "plain", eps=1e-13, x=x)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1, 7, 128, 1000, 7168, 20001, 40001])
def test_constant_rows(cols, dt):
    """every value alike: the differences from the mean are exactly zero, and y is the bias"""
    T = TORCH_HP[dt]
    x = torch.tensor([[0.0], [1000.0], [-0.3], [60000.0]]).expand(4, cols).contiguous().to(T)
    b = rand(gen_of("c", cols), cols).to(T)
    y, _, mean, rstd = fq.layernorm(up(x), up(torch.ones(cols, dtype=T)), up(b))
    tol = 2 * U * (x.abs().amax(1).to(D) * 2 * U) * 1e5      # m0 + m1 leaves a difference's rounding, times rstd
    assert ((y.cpu().to(D) - b.to(D)).abs() <= tol[:, None] + b.to(D).abs() * HALF_ULP[dt] + TINY[dt]).all()
    assert ((mean.cpu().to(D) - x[:, 0].to(D)).abs() <= 2 * U * x[:, 0].to(D).abs()).all()
    assert ((rstd.cpu().to(D) * 1e-5 ** 0.5 - 1).abs() <= 8 * U).all()


def test_nan_infinity_and_eps_zero():
    x = rand(gen_of("n"), 6, 256)
    x[1, 3] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 2.0
    x[4, 5] = 2e19                                          # its square passes binary32: rstd 0
    w, b = torch.ones(256), torch.full((256,), 0.25)
    y, _, mean, rstd = fq.layernorm(up(x), up(w), up(b), eps=0.0)
    y, mean, rstd = y.cpu(), mean.cpu(), rstd.cpu()
    for r in (1, 2):
        assert torch.isnan(y[r]).all() and torch.isnan(rstd[r])
    assert torch.isnan(y[3]).all() and torch.isinf(rstd[3]) and mean[3] == 2.0       # 0 * inf
    assert (y[4] == 0.25).all() and rstd[4] == 0.0
    clean = x[[0, 5]]
    h, m, s, want = layernorm64(clean, None, w, b, 0.0)
    near(y[[0, 5]], want, bounds(h, m, s, want, w.to(D), b.to(D), 0.0, False)[2] + want.abs() * U, "clean rows")
    q, s, _, _, _ = fq.layernorm_cast(up(x), up(w), up(b), eps=0.0)
    assert torch.isnan(q.cpu().float()[1]).all() and torch.isnan(s.cpu()[1]).all()
    assert torch.isfinite(q.cpu().float()[[0, 5]]).all()
    _, s, _, _, _ = fq.layernorm_cast(up(x), up(w), up(b), eps=0.0, per_channel_scale=True)
    assert s.cpu()[1] == torch.tensor(1.0) / 448            # the per-row rule: a NaN amax stands for 1


def test_empty():
    for shape in ((0, 256), (4, 0)):
        x, w = up(torch.zeros(shape)), up(torch.ones(shape[1]))
        _, s, _, _, _ = fq.layernorm_cast(x, w, w, per_channel_scale=True)
        assert (s.cpu() == 1).all()
        fq.layernorm_cast(x, w, w)
        y, _, _, _ = fq.layernorm(x, w)
        assert y.shape == shape


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(37, 1152), (290, 1003), (3, 8194), (2, 33333), (5, 6)])
def test_views_and_in_place(rows, cols, dt):
    """Views one element into their buffers; h over x or over the residual, and
    y over the other one: the same bits."""
    g = gen_of("views", cols)
    T = TORCH_HP[dt]
    x, r, w, b = rand(g, rows, cols).to(T), rand(g, rows, cols).to(T), (1 + rand(g, cols)).to(T), rand(g, cols).to(T)

    def view(t):
        return G.empty(t.numel() + 1, dtype=t.dtype)[1:].copy_(t.reshape(-1)).view(t.shape)

    new = lambda: (G.empty(rows, dtype=torch.float32), G.empty(rows, dtype=torch.float32))
    y0, h0, (m0, s0) = G.empty((rows, cols), dtype=T), G.empty((rows, cols), dtype=T), new()
    fq.fp8q_layernorm(up(x), up(w), up(b), y0, up(r), h0, m0, s0)
    for h_over, y_over in (("x", None), ("r", None), ("x", "r"), ("r", "x"), (None, "x"), (None, "r")):
        t = {"x": view(x), "r": view(r), None: view(torch.zeros(rows, cols, dtype=T))}
        h = t[h_over] if h_over else G.empty((rows, cols), dtype=T)
        y, (m, s) = t[y_over], new()
        fq.fp8q_layernorm(t["x"], view(w), view(b), y, t["r"], h, m, s)
        for a, c in ((y0, y), (h0, h), (m0, m), (s0, s)):
            assert torch.equal(a, c), (h_over, y_over)
    qs = []
    for v in (up, view):
        xv = v(x)
        q = G.empty(rows * cols + 1, dtype=torch.uint8)[1 if v is view else 0:][: rows * cols].view(rows, cols)
        s = G.empty(rows, dtype=torch.float32)
        fq.fp8q_layernorm_cast_per_channel(xv, v(w), v(b), q, s, v(r), xv)
        assert torch.equal(xv, h0)
        qs.append((q, s))
    assert torch.equal(qs[0][0], qs[1][0]) and torch.equal(qs[0][1], qs[1][1])


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------

def backward64(dy, h, w, mean, rstd, dh):
    n = (h.to(D) - mean.to(D)[:, None]) * rstd.to(D)[:, None]
    dn = dy.to(D) * w.to(D)
    dx = (dn - dn.mean(1, keepdim=True) - n * (dn * n).mean(1, keepdim=True)) * rstd.to(D)[:, None]
    return dx + (0 if dh is None else dh.to(D)), (dy.to(D) * n).sum(0), dy.to(D).sum(0), n, dn


BWD = [(1, 1, "f32", True, False), (1, 7168, "bf16", True, False), (9, 130, "f16", False, True),
       (700, 2048, "bf16", True, True), (33, 5001, "f32", True, False), (513, 72, "f32", False, False),
       (5, 20000, "bf16", True, False), (600, 8193, "f32", True, False), (3, 33001, "f16", False, False),
       (11, 3, "f32", True, False), (40, 5, "bf16", True, True), (530, 7168, "bf16", True, False),
       (520, 1501, "f16", True, True), (515, 4100, "bf16", False, False)]


@pytest.mark.parametrize("rows,cols,dt,dh,wf32", BWD)
def test_backward(rows, cols, dt, dh, wf32):
    g = gen_of(rows, cols, "lb")
    T = TORCH_HP[dt]
    h, dy = (rand(g, rows, cols) + rand(g, rows, 1)).to(T), rand(g, rows, cols).to(T)
    dhv = rand(g, rows, cols).to(T) if dh else None
    w = (1 + 0.3 * rand(g, cols)).to(torch.float32 if wf32 else T)
    _, mean, rstd, _ = layernorm64(h, None, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    want, wantw, wantb, n, dn = backward64(dy, h, w, mean, rstd, dhv)
    dx, dw, db = G.empty((rows, cols), dtype=T), G.empty(cols, dtype=w.dtype), G.empty(cols, dtype=w.dtype)
    args = (up(h), up(w), up(mean), up(rstd))
    fq.layernorm_backward(up(dy), *args, up(dhv) if dh else None, out=(dx, dw, db))
    gam = 1.01 * (depth(cols) + 4) * U
    m1, m2 = dn.abs().mean(1, keepdim=True), (dn * n).abs().mean(1, keepdim=True)
    err = rstd.to(D)[:, None] * (4 * U * (dn.abs() + m1 + n.abs() * m2) + gam * m1 + n.abs() * m2 * (gam + 4 * U))
    err = err + 2 * U * want.abs() + (dhv.to(D).abs() * 2 * U if dh else 0)
    near(dx, want, out_tol(want, dt, err), "dx")
    wdt = "f32" if wf32 else dt
    rowsum = 1.01 * (rows // 512 + 1 + 16 + 6) * U           # a workgroup's rows, then 512 partial rows over 32 lanes
    near(dw, wantw, out_tol(wantw, wdt, (dy.to(D) * n).abs().sum(0) * (rowsum + 3 * U)), "dweight")
    near(db, wantb, out_tol(wantb, wdt, dy.to(D).abs().sum(0) * rowsum), "dbias")
    # in place over dh or dy, each of the column sums alone or neither: the same bits
    if dh:
        dhd = up(dhv)
        fq.fp8q_layernorm_backward(up(dy), *args, dhd, None, None, dhd)
        assert torch.equal(dhd, dx)
    need = fq.fp8q_layernorm_backward_workspace_bytes(rows, cols)
    for which in (0, 1):
        dyd, o, ws = up(dy), G.empty(cols, dtype=w.dtype), G.empty(need, dtype=torch.uint8)
        fq.fp8q_layernorm_backward(dyd, *args, dyd, *((o, None) if which == 0 else (None, o)), up(dhv) if dh else None, ws)
        assert torch.equal(dyd, dx) and torch.equal(o, (dw, db)[which])


def test_backward_no_rows_and_no_bias():
    for wd in (torch.float32, torch.bfloat16):
        dw, db = G.full((96,), 7.0, dtype=wd), G.full((96,), 7.0, dtype=wd)
        e, z = torch.zeros(0, 96, dtype=wd, device="cuda"), torch.zeros(0, device="cuda")
        fq.fp8q_layernorm_backward(e, e, up(torch.ones(96, dtype=wd)), z, z, e, dw, db)
        assert (dw == 0).all() and (db == 0).all()
    x = up(rand(gen_of("nb"), 5, 96))
    o = up(torch.ones(96))
    _, h, mean, rstd = fq.layernorm(x, o)
    a, b = fq.layernorm_backward(x, h, o, mean, rstd), fq.layernorm_backward(x, h, o, mean, rstd, with_bias=False)
    assert b[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_against_differences():
    """sum(dy * y) along each gradient, in binary64, by central differences:
    binary32 gradients (1e-6 in norm), and step^2 ~ 1e-8"""
    g = gen_of("lnd")
    x, w, b, dy = rand(g, 6, 203) + 0.7, 1 + 0.3 * rand(g, 203), rand(g, 203), rand(g, 6, 203)
    f = lambda x, w, b: (dy.to(D) * layernorm64(x, None, w, b, 1e-5)[3]).sum()
    _, h, mean, rstd = fq.layernorm(up(x), up(w), up(b))
    for i, grad in enumerate(fq.layernorm_backward(up(dy), h, up(w), mean, rstd)):
        d = grad.cpu().to(D)
        step = 1e-4 * d / d.norm()
        at = lambda t: f(*[v.to(D) + (t if j == i else 0) for j, v in enumerate((x, w, b))])
        slope = (at(step) - at(-step)) / 2e-4
        assert abs(slope - d.norm()) <= 1e-5 * d.norm(), i


def test_nan_row_stays_in_its_row():
    """A NaN in one row of dy, and a row whose statistics are NaN: their rows of
    dx and the column sums have it, the other rows are as without."""
    g = gen_of("nr")
    x, dy, w = rand(g, 7, 300), rand(g, 7, 300), up(1 + rand(g, 300))
    _, h, mean, rstd = fq.layernorm(up(x), w)
    want = fq.layernorm_backward(up(dy), h, w, mean, rstd)[0]
    bad = dy.clone()
    bad[3, 7] = float("nan")
    rs = rstd.clone()
    rs[5] = float("inf")
    dx, dw, db = fq.layernorm_backward(up(bad), h, w, mean, rs)
    ok = [0, 1, 2, 4, 6]
    assert torch.equal(dx[ok], want[ok]) and torch.isnan(dx[3]).all() and not torch.isfinite(dx[5]).any()
    assert torch.isnan(db[7]) and torch.isfinite(db[torch.arange(300) != 7]).all()


@pytest.mark.parametrize("rows", [1, 700])
def test_streams_graphs_and_two_at_once(rows):
    """Twice, on a side stream, two calls at once on two streams, and replayed
    from a graph with eager calls between: the same bits every time."""
    g = gen_of("lnsg", rows)
    K = 1152
    x, r, dy = (up(rand(g, rows, K).bfloat16()) for _ in range(3))
    w, b = up((1 + 0.1 * rand(g, K)).bfloat16()), up(rand(g, K).bfloat16())

    def step():
        q, s, h, mean, rstd = fq.layernorm_cast(x, w, b, r)
        y, _, _, _ = fq.layernorm(x, w, b, r)
        return (q, s, h, mean, rstd, y, *fq.layernorm_backward(dy, h, w, mean, rstd, x))

    want = [t.clone() for t in step()]
    bits = lambda t: t.view(torch.uint8) if t.dtype != torch.float32 else t.view(torch.int32)
    same = lambda out: all(torch.equal(bits(a), bits(c)) for a, c in zip(out, want))
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
            bits(t).fill_(0x55)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out)
        assert same(step())
