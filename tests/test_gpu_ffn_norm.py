"""GPU: the norm's launch shapes and outputs beyond tests/test_gpu_ffn.py."""
import pytest
import torch

import dequantize_amax_reduce_amd as fq
from gpu_util import G, TORCH_HP
from test_gpu_ffn import FP8, gen_of, rand, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,per_row", [(3, 256, False), (40, 333, True), (2, 40960, False)])
def test_h_is_written_without_a_residual(rows, cols, per_row):
    """`out` with an h of its own: x's values, whatever it held before; x itself
    in its place stays as it is."""
    g = gen_of(rows, cols, "h")
    for dt in ("bf16", "f32"):
        T = TORCH_HP[dt]
        x, w = rand(g, rows, cols).to(T), (1 + rand(g, cols)).to(T)
        xd = up(x)
        out = lambda h: (G.empty((rows, cols), dtype=FP8["e4m3fn"]),
                         G.empty((rows,) if per_row else (rows, cols // 128), dtype=torch.float32), h,
                         G.empty(rows, dtype=torch.float32))
        h = G.full((rows, cols), 7.0, dtype=T)
        a = fq.rmsnorm_cast(xd, up(w), per_channel_scale=per_row, out=out(h))
        assert a[2] is h and torch.equal(h.cpu(), x)
        b = fq.rmsnorm_cast(xd, up(w), per_channel_scale=per_row, out=out(xd))
        assert b[2] is xd and torch.equal(xd.cpu(), x)
        for i in (0, 1, 3):
            assert torch.equal(a[i].view(torch.uint8), b[i].view(torch.uint8))


def test_backward_of_a_very_long_row():
    """2^27 + 5 columns: more column tiles of dweight than one grid holds.  One
    row of equal values: n = 1, so dweight = dy, and dx = dy - mean(dy)."""
    cols = (1 << 27) + 5
    h = torch.ones(1, cols, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    dy[0, ::2] = 0.5
    dy[0, -1] = 3.0
    w, rstd = torch.ones(cols, dtype=torch.bfloat16, device="cuda"), torch.ones(1, device="cuda")
    dw = torch.full((cols,), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full_like(dy, 7.0)
    fq.rmsnorm_cast_backward(dy, h, w, rstd, out=(dx, dw))
    assert torch.equal(dw, dy[0])
    mean = 0.25                                             # to 2^-25; dy - mean is exact in bf16
    assert torch.equal(dx, dy - mean)
