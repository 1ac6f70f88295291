"""uint8 codes of either format in the feed-forward operators: x_fmt and w_fmt
name it, and may not contradict a float8 tensor's own."""
import pytest
import torch

import dequantize_amax_reduce_amd as fq

E4, E5, U8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.uint8


def operands(gen, M, K, N, xt, wt, device):
    c = lambda r, t: (torch.randn(r, K, generator=gen) * 4).to(t).to(device)
    return (c(M, xt), torch.rand(M, K // 128, generator=gen).to(device) + 0.5), \
        [(c(N, wt), torch.rand((N + 127) // 128, K // 128, generator=gen).to(device) + 0.5) for _ in range(2)]


def calls(x, w, dy, z, **k):
    """every operator that reads codes"""
    (xq, xs), ((gq, gs), (uq, us)) = x, w
    yield fq.linear_fp8, (xq, xs, gq, gs), k
    yield fq.linear_fp8_backward, (dy, xq, xs, gq, gs), k
    yield fq.gated_linear_fp8, (xq, xs, gq, gs, uq, us), k
    yield fq.gated_linear_fp8_cast, (xq, xs, gq, gs, uq, us), k
    yield fq.gated_linear_fp8_backward, (dy, z, xq, xs, gq, gs, uq, us), k


def test_formats_that_contradict_the_codes():
    gen = torch.Generator().manual_seed(1)
    x, w = operands(gen, 4, 128, 128, E4, E5, "cpu")
    dy, z = torch.zeros(4, 128).bfloat16(), torch.zeros(4, 256).bfloat16()
    for bad in (dict(x_fmt="e5m2"), dict(w_fmt="e4m3fn"), dict(x_fmt="e3m4")):
        for f, a, k in calls(x, w, dy, z, **bad):
            with pytest.raises(TypeError):
                f(*a, **k)


@pytest.mark.gpu
@pytest.mark.parametrize("xt,wt", [(E4, E5), (E5, E4), (E5, E5)])
def test_uint8_codes(xt, wt):
    gen = torch.Generator().manual_seed(2)
    M, K, N = 70, 256, 256
    x, w = operands(gen, M, K, N, xt, wt, "cuda")
    dy, z = torch.randn(M, N).bfloat16().cuda(), torch.randn(M, 2 * N).bfloat16().cuda()
    u8 = lambda c: (c[0].view(U8), c[1])
    for (f, a, _), (_, b, k) in zip(calls(x, w, dy, z), calls(u8(x), [u8(c) for c in w], dy, z, x_fmt=xt, w_fmt=wt)):
        want, got = f(*a), f(*b, **k)
        for p, q in zip(want if isinstance(want, tuple) else (want,), got if isinstance(got, tuple) else (got,)):
            assert (p is None and q is None) or torch.equal(p.view(U8), q.view(U8)), f.__name__
