"""GPU: the activations of the gated pair and their slopes in the tails, where
the function is a small part of what it is computed from, and at arguments whose
powers leave binary32.

Each pre-activation is set exactly: a row of X is one code with the row's scale,
a row of W one code, so that g is their product.  Tolerances, relative to the
activation itself: the arguments of exp and erfc carry a few binary32 roundings,
which grow by the argument's size (2 x^2 + 2 = g^2 + 2 for erfc(g / sqrt 2), 2 |y|
for exp(2 y)), and 16 units in the last place cover the functions themselves.
"""
import math

import pytest
import torch

import dequantize_amax_reduce_amd as fq
from gpu_util import TORCH_HP
from test_gpu_ffn import D, HALF_ULP, TINY, up

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn
ULP = 2.0 ** -23
TAIL = [-0.25, -1.0, -2.0, -3.0, -4.0, -4.5, -5.0, -5.5, -6.0, -7.0, -8.0, -9.0, -10.0, -12.0]


def act_mp(name, g):
    """(act, act', relative error of act, absolute error of act') in binary64,
    from forms that do not cancel"""
    if name == "silu":
        s, r = torch.sigmoid(g), torch.sigmoid(-g)
        d = s * (1 + g * r)
        return g * s, d, 20 * ULP + 0 * g, s * (1 + g.abs() * r) * 20 * ULP + s * g.abs() * ULP
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        p = g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        rel = (g * g + 20) * ULP
        return g * c, c + p, rel, (c + p.abs()) * rel
    h = g.clamp(-1e3, 1e3)                                  # the logistic is 0 or 1 beyond
    y2 = 2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)
    s, r = torch.sigmoid(y2), torch.sigmoid(-y2)
    t = h * s * r * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * h * h)
    rel = (4 * y2.abs() + 20) * ULP
    slope = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * h.clamp(-64, 64) ** 2)
    return g * s, s + t, rel, (s + t.abs()) * rel + s * h.abs().clamp(max=64) * slope * ULP


def one_hot(rows, cols, at, value=1.0):
    q = torch.zeros(rows, cols)
    q[torch.arange(rows), at] = value
    return q.to(E4)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [14, 200])                    # the few-row kernel, tiles
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_forward_tail(act, M, dt):
    K, F = 128, 40
    g = torch.tensor([TAIL[i % len(TAIL)] * (1 + (i // len(TAIL)) / 64) for i in range(M)], dtype=torch.float32)
    x = torch.zeros(M, K)
    x[:, 0] = 1.0
    w = one_hot(F, K, 0, -1.0)
    w1 = one_hot(F, K, 0, 0.5)
    xs, one = -g[:, None].clone(), torch.ones(1, 1)         # X[m, 0] = -g: gate g, up -g / 2
    h, z = fq.gated_linear_fp8(up(x.to(E4)), up(xs), up(w), up(one), up(w1), up(one), act, TORCH_HP[dt],
                               keep=torch.float32)
    gd = g.to(D)[:, None].expand(M, F)
    assert torch.equal(z.cpu()[:, :F].to(D), gd) and torch.equal(z.cpu()[:, F:].to(D), -gd / 2)
    a, _, rel, _ = act_mp(act, gd)
    want = a * -gd / 2
    err = (h.cpu().to(D) - want).abs()
    assert (err <= want.abs() * (rel + 2 * ULP + HALF_ULP[dt]) + TINY[dt]).all(), float((err / want.abs()).max())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_backward_tail(act):
    """dW of one-hot rows of X is dz itself: one column of dz has one
    pre-activation, so that its f16 scale is its own."""
    M, K, F = 128, 128, len(TAIL) + 6
    gv = torch.tensor(TAIL + [0.5, 1.0, 2.0, 4.0, 8.0, 16.0])
    z = torch.cat([gv.expand(M, F), torch.full((M, F), 1.5)], 1).bfloat16()
    gen = torch.Generator().manual_seed(5)
    dp = (1 + torch.rand(M, F, generator=gen)).bfloat16()
    x = one_hot(M, K, torch.arange(M))
    w = one_hot(F, K, torch.arange(F))
    one, xs = torch.ones(1, 1), torch.ones(M, 1)
    _, dwg, dwu = fq.gated_linear_fp8_backward(up(dp), up(z), up(x), up(xs), up(w), up(one), up(w), up(one), act,
                                               torch.float32)
    a, da, rel, eda = act_mp(act, z[:, :F].to(D))
    for got, want, err in ((dwg, dp.to(D) * da * 1.5, dp.to(D) * 1.5 * eda), (dwu, dp.to(D) * a, (dp.to(D) * a).abs() * rel)):
        want, err = want.t(), err.t()
        tol = err + want.abs() * (2.0 ** -11 + 4 * ULP) + TINY["f32"]
        assert ((got.cpu().to(D)[:, :M] - want).abs() <= tol).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_backward_far_arguments(act):
    """Finite gradients where g^2, g^3 or dp * u leave binary32."""
    M, K, F = 128, 128, 8
    gv = torch.tensor([-3e38, -1e30, -2e19, -1e4, 1e4, 2e19, 1e30, 3e38])
    z = torch.cat([gv.expand(M, F), torch.where(gv < 0, 1e30, 1.0).expand(M, F)], 1).bfloat16()
    dp = torch.where(gv < 0, 1e30, 1e-6).expand(M, F).contiguous().bfloat16()
    x = one_hot(M, K, torch.arange(M))
    w = one_hot(F, K, torch.arange(F))
    one, xs = torch.ones(1, 1), torch.ones(M, 1)
    dx, dwg, dwu = fq.gated_linear_fp8_backward(up(dp), up(z), up(x), up(xs), up(w), up(one), up(w), up(one), act,
                                                torch.float32)
    a, da, _, _ = act_mp(act, z[:, :F].to(D))
    zu, d = z[:, F:].to(D), dp.to(D)
    for got, want in ((dwg, d * da * zu), (dwu, d * a)):
        got, want = got.cpu().to(D), want.t()
        assert torch.isfinite(got).all()
        assert ((got[:, :M] - want).abs() <= want.abs() * (2.0 ** -11 + 64 * ULP)).all()
    assert torch.isfinite(dx).all()
