"""GPU: the backward products over the whole range of the values they meet.
A row of dx depends on its own row of the gradient, a row of dW on its own
column of it, and a row of X (or a block row of W) whose gradient is zero on
neither, whatever magnitudes the others have.

Tolerances, per element, from how the operands are rounded.  With 2^ex[m] and
2^ew[n/128] the powers of two of the largest scale of a row of X and of a block
row of W, dx = (dz 2^ew)(W 2^-ew) and dW = (dz 2^ex)^T (X 2^-ex), and each
operand is rounded to f16 below a power of two of its own (per row of the
first, per 128 columns of the second):

(a gated pair's take the scale itself, which is within a factor of two)

* a value is within 2^-11 of itself, or within half an f16 subnormal's unit,
  2^-25 of the scaled value: the largest of a row lies in [2^14, 2^15), so
  2^-39 of it; the codes' bound is 2^q times twice the largest scale's power of
  two, so 2^(q - 39) of the largest scale;
* the products are summed in binary32 (n 2^-23 of the sum of magnitudes), and
  the result is rounded once.
"""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
from gpu_util import G, TORCH_HP
from test_gpu_ffn import D, act64, codes, gen_of, near, out_tol, rand, up, w64, x64

pytestmark = pytest.mark.gpu

QBITS = {torch.float8_e4m3fn: 9, torch.float8_e5m2: 16}


def power(s):
    """2^floor(log2(largest of a row)), 1 for a row of zeros"""
    m = s.to(D).amax(1)
    return torch.where(m > 0, 2.0 ** torch.floor(torch.log2(m.clamp_min(1e-300))), torch.ones_like(m))


def product_err(a, b, scales, q, n):
    """bound on the error of a [M, n] times b [n, K] as the module's docstring
    says; scales [rows, K / 128] are b's, as folded"""
    a0 = a.abs().amax(1, keepdim=True) * 2.0 ** -39
    b0 = (scales.amax(0) * 2.0 ** (q - 39)).repeat_interleave(128)[None]
    A, B = a.abs(), b.abs()
    return (A @ B) * (2 * 2.0 ** -11 + 2.0 ** -20 + n * 2.0 ** -23) + a0 * (B.sum(0, keepdim=True) + n * b0) + \
        b0 * A.sum(1, keepdim=True)


def dx_err(dzs, ws, n):
    """dzs, ws: gradients with (codes, scales) of each projection"""
    fold = [power(s).repeat_interleave(128)[: q.shape[0]] for q, s in ws]
    a = torch.cat([dz * f for dz, f in zip(dzs, fold)], 1)
    b = torch.cat([w64(q, s) / f[:, None] for (q, s), f in zip(ws, fold)])
    sc = torch.cat([s.to(D) / power(s)[:, None] for _, s in ws])
    return product_err(a, b, sc, QBITS[ws[0][0].dtype], n)


def dw_err(dz, xq, xs, n):
    f = power(xs)
    return product_err((dz * f[:, None]).t(), x64(xq, xs) / f[:, None], xs.to(D) / f[:, None], QBITS[xq.dtype], n)


# powers of two that the rows and columns of the gradient, the masked rows of X
# and the masked block rows of W reach; f16 gradients hold 2^-24 to 2^15
SPREAD = {"bf16": (80, 100), "f16": (5, 100)}


def gradient(g, M, N, dt):
    """rows and columns of widely spread magnitudes; row 5 and the columns of
    the second block row of W are zero"""
    e, _ = SPREAD[dt]
    r = torch.tensor([2.0 ** ((m * 37) % (e + 1) - e // 2) for m in range(M)])
    c = torch.tensor([2.0 ** ((n * 11) % (e // 2 + 1) - e // 4) for n in range(N)])
    dy = rand(g, M, N) * r[:, None] * c[None]
    dy[5] = 0.0
    dy[:, 128:256] = 0.0
    return dy


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,xf", [(70, 256, 300, "e4m3fn"), (130, 384, 576, "e5m2")])
def test_linear_backward_spread(M, K, N, xf, dt):
    g = gen_of(M, K, N, dt, "spread")
    _, big = SPREAD[dt]
    xq, xs = codes(g, M, K, xf, M)
    wq, ws = codes(g, N, K, "e4m3fn", (N + 127) // 128)
    xs[5] *= 2.0 ** big                                     # meets a zero row of the gradient
    ws[1] *= 2.0 ** big                                     # and zero columns
    dy = gradient(g, M, N, dt).to(TORCH_HP[dt])
    X, W, d = x64(xq, xs), w64(wq, ws), dy.to(D)
    dx, dw = fq.linear_fp8_backward(up(dy), up(xq), up(xs), up(wq), up(ws), torch.float32)
    near(dx, d @ W, out_tol(d @ W, dt, dx_err([d], [(wq, ws)], N + 64)), "dx")
    near(dw, d.t() @ X, out_tol(d.t() @ X, "f32", dw_err(d, xq, xs, M + 64)), "dw")
    assert (dx[5] == 0).all() and (dw[128:256] == 0).all()


def test_a_row_of_dx_does_not_see_the_others():
    """The same bits for a row alone and beside rows 2^60 larger and smaller."""
    g = gen_of("alone")
    M, K, N = 70, 384, 200
    xq, xs = codes(g, M, K, "e4m3fn", M)
    wq, ws = codes(g, N, K, "e4m3fn", 2)
    dy = rand(g, M, N)
    for dt in ("bf16", "f16"):
        big = 60 if dt == "bf16" else 12
        base = dy.to(TORCH_HP[dt])
        want, _ = fq.linear_fp8_backward(up(base), up(xq), up(xs), up(wq), up(ws))
        other = base.clone()
        other[::2] *= 2.0 ** big
        other[1::4] *= 2.0 ** -big
        got, _ = fq.linear_fp8_backward(up(other), up(xq), up(xs), up(wq), up(ws))
        keep = torch.arange(M) % 4 == 3
        assert torch.equal(got.cpu()[keep], want.cpu()[keep]), dt
        assert torch.isfinite(got.cpu()[keep]).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,F", [(70, 256, 300), (130, 384, 576)])
def test_gated_backward_spread(M, K, F, act, dt):
    """Also pre-activations that are huge where dp is zero, and large up
    projections beside gates whose slope is zero."""
    g = gen_of(M, K, F, act, dt, "spread")
    e, big = SPREAD[dt]
    T = TORCH_HP[dt]
    xq, xs = codes(g, M, K, "e4m3fn", M)
    gq, gs = codes(g, F, K, "e4m3fn", (F + 127) // 128)
    uq, us = codes(g, F, K, "e4m3fn", (F + 127) // 128)
    xs[5] *= 2.0 ** big
    gs[1] *= 2.0 ** big
    us[1] *= 2.0 ** -big
    dp = (gradient(g, M, F, dt) * (1.0 if dt == "bf16" else 2.0 ** -4)).to(T)
    z = rand(g, M, 2 * F)
    z[5] *= 2.0 ** (12 if dt == "bf16" else 8)              # dp is zero there
    z[9, :F] = -60.0                                        # no slope, no activation
    z[9, F:] *= 2.0 ** 12
    z[9, 0] = 1.0
    z = z.to(T)
    zg, zu, d = z[:, :F].to(D), z[:, F:].to(D), dp.to(D)
    a, da = act64(act, zg)
    dg, du = d * zu * da, d * a
    X, Wg, Wu = x64(xq, xs), w64(gq, gs), w64(uq, us)
    dx, dwg, dwu = fq.gated_linear_fp8_backward(up(dp), up(z), up(xq), up(xs), up(gq), up(gs), up(uq), up(us), act,
                                                torch.float32)
    # the binary32 evaluation of the activation: a few ulps of max(1, |g|) terms
    ea = 2.0 ** -19 * (1 + zg.abs())
    eg, eu = (d * zu).abs() * ea, d.abs() * ea
    want = dg @ Wg + du @ Wu
    err = dx_err([dg.abs() + eg, du.abs() + eu], [(gq, gs), (uq, us)], 2 * F + 128) + eg @ Wg.abs() + eu @ Wu.abs()
    near(dx, want, out_tol(want, dt, err), "dx")
    for got, v, ev, what in ((dwg, dg, eg, "dw_gate"), (dwu, du, eu, "dw_up")):
        near(got, v.t() @ X, out_tol(v.t() @ X, "f32", dw_err(v.abs() + ev, xq, xs, M + 64) + ev.t() @ X.abs()), what)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gated_nan_and_infinity_stay_in_their_row(dt):
    """A NaN or infinity in one row of dp (or of z) reaches that row of dx and no
    other, and of the weight gradients the rows of its column."""
    g = gen_of("gnan", dt)
    M, K, F = 140, 256, 200
    T = TORCH_HP[dt]
    xq, xs = codes(g, M, K, "e4m3fn", M)
    w = [up(t) for p in (codes(g, F, K, "e4m3fn", 2) for _ in range(2)) for t in p]
    dp, z = (0.01 * rand(g, M, F)).to(T), rand(g, M, 2 * F).to(T)
    dp[5] = 0.0
    call = lambda dp, z: fq.gated_linear_fp8_backward(up(dp), up(z), up(xq), up(xs), *w)
    clean = call(dp, z)
    assert all(torch.isfinite(t).all() for t in clean) and (clean[0][5] == 0).all()
    rest = torch.arange(M) != 5
    for where, bad in (("dp", float("nan")), ("dp", float("inf")), ("z", float("nan"))):
        d, y = dp.clone(), z.clone()
        (d if where == "dp" else y)[5, 7] = bad
        dx, dg, du = call(d, y)
        assert not torch.isfinite(dx[5]).any()
        assert torch.equal(dx.cpu()[rest], clean[0].cpu()[rest])
        cols = torch.arange(F) != 7
        for got, want in ((dg, clean[1]), (du, clean[2])):
            assert not torch.isfinite(got[7]).all()
            assert torch.equal(got.cpu()[cols], want.cpu()[cols])
