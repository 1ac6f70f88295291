"""GPU: bits that layer norm and projections with an epilogue have to keep
(include/fp8q_mlp.h): the mean of rows around zero, rows whose squares pass
binary32, constant rows of 10^6 columns; the sums of projections of 17 to 64
rows and of more; gradients asked for alone, and f16 ones; and every instance of
the layer norm's backward pass over more rows than it has workgroups."""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
import test_gpu_layernorm as L
from gpu_util import G, TORCH_HP
from mlp_plans import ALONE, ALONE_REST, LAYERNORM_BACKWARD
from test_gpu_ffn import D, FP8, codes, gen_of, rand, up, w64, x64
from test_gpu_layernorm import U

pytestmark = pytest.mark.gpu


# rows of a wave (1 and 2 vectors), of a workgroup (1, 2 and 4), in passes, shorter than a vector
WIDTHS = [(300, 256, "bf16"), (300, 1001, "f16"), (300, 500, "f32"), (70, 7168, "bf16"), (40, 5001, "f32"),
          (20, 12001, "bf16"), (10, 32768, "f16"), (10, 40001, "bf16"), (10, 20000, "f32"), (50, 5, "bf16"), (50, 3, "f32")]


@pytest.mark.parametrize("rows,cols,dt", WIDTHS)
@pytest.mark.parametrize("res", [False, True])
def test_mean_of_rows_around_zero(rows, cols, dt, res):
    """x and residual are multiples of 2^-6 under 2, so that a row's sum has at most
    24 bits in any order: the mean has the rounding of a quotient alone, two
    where it is a product by the rounded 1 / n.  (Differences from it, each
    rounded, would add 2^-24 of the deviation to a mean 100 times smaller.)"""
    g = gen_of("mean", rows, cols, dt, res)
    units = lambda: torch.randint(-127, 128, (rows, cols), generator=g).float()
    a, r = units(), units()
    for t in (a, r):                                        # the last row sums to zero: its mean is zero
        n = cols // 2
        t[-1, n:2 * n] = -t[-1, :n]
        t[-1, 2 * n:] = 0.0
    T = TORCH_HP[dt]
    x, r = (a * 2.0 ** -6).to(T), (r * 2.0 ** -6).to(T)
    h = x.to(D) + (r.to(D) if res else 0)
    mean, var = h.mean(1), h.var(1, correction=0)
    _, _, m, _ = fq.layernorm(up(x), up(torch.ones(cols, dtype=T)), None, up(r) if res else None)
    err = (m.cpu().to(D) - mean).abs()
    inside = 16 * mean.square() < 0.99 * var                # further out the mean is held to the row's bound
    size = cols * a.new_empty(0, dtype=T).element_size()
    inside |= not 16 <= size <= 65536                       # (rows in passes: a binary64 sum's)
    assert inside.sum() > rows // 2
    assert (err <= 2.01 * U * mean.abs())[inside].all(), float((err / mean.abs().clamp_min(1e-30))[inside].max() / U)
    assert float(m[-1]) == 0.0


@pytest.mark.parametrize("cols", [3, 256, 701, 5001, 7168, 16384, 20000, 33333])
@pytest.mark.parametrize("rows", [6, 300])
def test_rows_whose_squares_pass_binary32(rows, cols):
    """One element, or every one, of 1e27 to 1e35: the mean square of the
    differences is infinite, so that rstd is 0 and y the bias.  A constant row of
    1e30 has no differences, or infinite squares of its mean's roundings: y is
    the bias too, and the mean is its value."""
    g = gen_of("squares", rows, cols)
    x = 256 * rand(g, rows, cols)
    at = cols // 3
    x[0, at], x[1, at], x[2, at] = 1e30, -1e35, 1e27
    x[3], x[4] = 1e30 * rand(g, cols), 1e35 * rand(g, cols)
    x[5] = 1e30
    w, b = 1 + rand(g, cols), rand(g, cols)
    y, _, mean, rstd = fq.layernorm(up(x), up(w), up(b))
    assert (rstd[:5] == 0).all() and torch.isfinite(mean).all()
    assert torch.equal(y[:6].cpu(), b.expand(6, cols))
    assert abs(float(mean[5].cpu().to(D) / x[5, 0].to(D)) - 1) <= 2 * U
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("cols,dt", [(500001, "f32"), (1000003, "f32"), (1 << 20, "f32"), (1000003, "bf16")])
def test_constant_rows_of_a_million(cols, dt):
    """every value alike: the differences from the mean are exactly zero at any
    width, so that y is the bias and a cast without one has nothing to scale"""
    T = TORCH_HP[dt]
    g = gen_of("million", cols)
    v = (rand(g, 20, 1) * 10 ** (2 * rand(g, 20, 1))).to(T)
    x = v.cuda().expand(20, cols).contiguous()
    w, b = torch.ones(cols, dtype=T, device="cuda"), torch.linspace(-1, 1, cols, device="cuda").to(T)
    y, _, mean, _ = fq.layernorm(x, w, b)
    assert torch.equal(y, b.expand(20, cols))
    assert torch.equal(mean.cpu(), v[:, 0].float())
    q, s, _, _, _ = fq.layernorm_cast(x, w, None, per_channel_scale=True)
    assert (q.float() == 0).all() and (s == torch.tensor(1.0) / 448).all()


@pytest.mark.parametrize("M", [17, 33, 48, 64])
@pytest.mark.parametrize("K,N", [(128, 72), (1152, 200), (7168, 61), (2048, 4104)])
@pytest.mark.parametrize("dt,xf,wf,res", [("bf16", "e4m3fn", "e4m3fn", False), ("f16", "e5m2", "e4m3fn", True)])
def test_sums_up_to_64_rows_are_binary32(M, K, N, dt, xf, wf, res):
    """In every 128-block two products of 448^2 cancel beside 126 of 1/2, at
    places that differ from block to block, and scales are powers of two: all
    partial sums are multiples of a half, or of scales times it, of at most 24
    bits, so binary32 sums have no rounding in any order.  (Sums that keep 16
    bits below a block's largest product lose the halves.)"""
    g = gen_of("binary32", M, K, N)
    KB = K // 128
    x, w = torch.ones(M, K), torch.full((N, K), 0.5)
    for kb in range(KB):
        i, j = (kb * 128 + torch.randperm(128, generator=g)[:2]).tolist()
        x[:, i], x[:, j], w[:, i], w[:, j] = 448.0, 448.0, 448.0, -448.0
    xq, wq = x.to(FP8[xf]), w.to(FP8[wf])
    xs = 2.0 ** torch.randint(-2, 1, (M, KB), generator=g).float()
    ws = 2.0 ** torch.randint(-2, 1, ((N + 127) // 128, KB), generator=g).float()
    z = x64(xq, xs) @ w64(wq, ws).t()
    assert torch.equal(z, 63 * xs.to(D) @ ws.to(D).repeat_interleave(128, dim=0)[:N].t())
    T = TORCH_HP[dt]
    r = torch.randint(-64, 65, (M, N), generator=g).to(T) if res else None
    y, kept = fq.linear_act_fp8(up(xq), up(xs), up(wq), up(ws), None, None, None if r is None else up(r), T, keep=T)
    assert torch.equal(kept.cpu(), z.to(T)) and torch.equal(y.cpu(), (z + (0 if r is None else r.to(D))).to(T))
    if not res:                                             # and as a bare projection has them
        assert torch.equal(y, fq.linear_fp8(up(xq), up(xs), up(wq), up(ws), out=torch.empty_like(y)))


@pytest.mark.parametrize("M,K,N", [(65, 640, 72), (100, 4096, 264), (300, 7168, 300), (1003, 2048, 200), (1000, 512, 4101)])
@pytest.mark.parametrize("keep", [False, True])
def test_fp8_sums_keep_their_bits(M, K, N, keep):
    """16-bit outputs of more than 64 rows: 16 bits are kept below the largest
    product of 128, so a product is off by 2^-16 / sqrt 3 of it in root mean
    square and a block's sum by sqrt(128) times that: 2^-13.1 of the root of the
    sum of squared products, r, of which the largest is a part.  So f16 outputs
    are within 2^-13 r, in root mean square, of their own rounding, and none is
    further off than 2^-10 r and half a unit in its last place."""
    g = gen_of("act bits", M, K, N)
    xq, xs = codes(g, M, K, "e4m3fn", M)
    wq, ws = codes(g, N, K, "e4m3fn", (N + 127) // 128)
    X, W = x64(xq, xs) * 2.0 ** -4, w64(wq, ws)             # no f16 overflow
    want = X @ W.t()
    assert float(want.abs().max()) < 65504
    H = torch.float16
    y, z = fq.linear_act_fp8(up(xq), up(xs * 2.0 ** -4), up(wq), up(ws), ret_type=H, keep=H if keep else None)
    r = torch.sqrt((X * X) @ (W * W).t())
    live = r > 2.0 ** -8                                     # f16's subnormals are no matter here; zero rows
    rms = lambda v: float(v.square().mean().sqrt())
    for got in (y, z) if keep else (y,):
        got = got.cpu().to(D)
        e, rounding = ((got - want) / r)[live], ((want.half().to(D) - want) / r)[live]
        assert rms(e) <= rms(rounding) + 2.0 ** -13
        assert ((got - want).abs() <= r * 2.0 ** -10 + want.abs() * 2.0 ** -11 + 2.0 ** -25).all()


@pytest.mark.parametrize("M,K,N,dt,act", [(*s, *t) for s in ALONE for t in (("bf16", "gelu"), ("f16", None))] +
                         [(*s, "f16", "silu") for s in ALONE_REST])
def test_one_gradient_alone(M, K, N, dt, act):
    """dx without dw and dw without dx run in tiles of their own: the same bits"""
    g = gen_of("alone", M, K, N)
    xq, xs = codes(g, M, K, "e4m3fn", M)
    wq, ws = codes(g, N, K, "e4m3fn", (N + 127) // 128)
    dy, z = (0.05 * rand(g, M, N)).to(TORCH_HP[dt]), (2 * rand(g, M, N)).to(TORCH_HP[dt])
    args = (up(dy), None if act is None else up(z), up(xq), up(xs), up(wq), up(ws))
    out = fq.linear_act_fp8_backward(*args, act)
    scratch = G.empty(fq.fp8q_linear_act_backward_workspace_bytes(M, N, K), dtype=torch.uint8)
    for i in range(3):
        o = [torch.empty_like(t) if j == i else None for j, t in enumerate(out)]
        fq.fp8q_linear_act_backward(*args, *o, act, scratch)
        assert torch.equal(o[i], out[i]), i


@pytest.mark.parametrize("M,K,N", [(500, 640, 700), (300, 1024, 1000), (1500, 256, 90)])
def test_f16_gradients_of_a_bare_product(M, K, N):
    """Without an activation dy is exact in f16 and one operand of a product has one
    f16 rounding: of independent signs, in the sum the share of its norm that the
    outputs' own rounding is of theirs.  So sqrt 2 times that in all; a tenth more for
    the sample."""
    g = gen_of("bare", M, K, N)
    xq, xs = codes(g, M, K, "e4m3fn", M)
    wq, ws = codes(g, N, K, "e4m3fn", (N + 127) // 128)
    dy = (0.01 * rand(g, M, N)).half()
    dx, dw, _ = fq.linear_act_fp8_backward(up(dy), None, up(xq), up(xs), up(wq), up(ws))
    for got, want in ((dx, dy.to(D) @ w64(wq, ws)), (dw, dy.to(D).t() @ x64(xq, xs))):
        assert float(want.abs().max()) < 65504
        own = (want.half().to(D) - want).norm()
        assert (got.cpu().to(D) - want).norm() <= 1.1 * 2 ** 0.5 * own


@pytest.mark.parametrize("rows,cols,dt", list(LAYERNORM_BACKWARD))
@pytest.mark.parametrize("dh,wf32", [(False, False), (True, True)])
def test_every_instance_of_the_norms_backward(rows, cols, dt, dh, wf32):
    """more rows than workgroups: the next row's loads, the sums over rows, and
    dx over dy and over dh"""
    L.test_backward(rows, cols, dt, dh, wf32)
