"""GPU: bits that layer norm and projections with an epilogue have to keep
(include/fp8q_mlp.h): constant rows of 10^6 columns."""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
from gpu_util import TORCH_HP
from test_gpu_ffn import gen_of, rand

pytestmark = pytest.mark.gpu


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
