"""A feed-forward block on fp8 operands, as a training step and as a decode
step: residual + norm -> fp8 -> gate/up/activation -> fp8 -> down projection,
and the gradients of all of it.

    python dequantize_amax_reduce_amd/examples/ffn_block.py [tokens] [hidden] [width]

(run from the repository's root; needs an MI355X).  Activations pass between
the operators as codes with scales; the only 16-bit tensors are the residual
stream, the pre-activations kept for the backward pass, and the gradients.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__)))))
import dequantize_amax_reduce_amd as fq  # noqa: E402


def quantize_weight(w):
    """One scale per 128x128 block: what a checkpoint in this format holds."""
    n, k = w.shape
    b = torch.nn.functional.pad(w.float(), (0, 0, 0, -n % 128)).view(-1, 128, k // 128, 128)
    s = b.abs().amax(dim=(1, 3)).clamp_min(1e-8) / 448.0
    q = (b / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1, k)[:n].contiguous()
    return q, s


class Block:
    def __init__(self, hidden, width, device="cuda", activation="silu"):
        r = lambda n, k: torch.randn(n, k, device=device) * k ** -0.5
        self.norm = torch.ones(hidden, device=device, dtype=torch.bfloat16)
        self.gate, self.up, self.down = (quantize_weight(r(*s)) for s in ((width, hidden), (width, hidden),
                                                                          (hidden, width)))
        self.activation = activation

    def forward(self, x, residual, keep=False):
        """(the block's output, the new residual stream, what backward reads)"""
        q, s, h, rstd = fq.rmsnorm_cast(x, self.norm, residual)
        p, ps, z = fq.gated_linear_fp8_cast(q, s, *self.gate, *self.up, self.activation,
                                            keep=torch.bfloat16 if keep else None)
        y = fq.linear_fp8(p, ps, *self.down)
        return y, h, (q, s, h, rstd, p, ps, z)

    def backward(self, dy, dh, kept):
        """Gradients of x (and of the residual alike) and of the weights, from
        those of the output and of the residual stream."""
        q, s, h, rstd, p, ps, z = kept
        dp, d_down = fq.linear_fp8_backward(dy, p, ps, *self.down)
        dn, d_gate, d_up = fq.gated_linear_fp8_backward(dp, z, q, s, *self.gate, *self.up, self.activation)
        dx, d_norm = fq.rmsnorm_cast_backward(dn, h, self.norm, rstd, dh)
        return dx, (d_norm, d_gate, d_up, d_down)


def main(tokens=2048, hidden=2048, width=5632):
    torch.manual_seed(0)
    block = Block(hidden, width)
    bf = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16)

    # a training step
    x, residual = bf(tokens, hidden), bf(tokens, hidden)
    y, h, kept = block.forward(x, residual, keep=True)
    dx, grads = block.backward(bf(tokens, hidden) * 0.01, bf(tokens, hidden) * 0.01, kept)

    # the same block in plain 32-bit torch, from the weights' own values
    deq = lambda q, s: fq.weight_dequant(q, s, ret_type=torch.float32)
    hf = x.float() + residual.float()
    n = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + 1e-6)
    ref = (torch.nn.functional.silu(n @ deq(*block.gate).t()) * (n @ deq(*block.up).t())) @ deq(*block.down).t()
    err = float((y.float() - ref).norm() / ref.norm())
    print(f"training step: {tokens} tokens, output {tuple(y.shape)}, dx {tuple(dx.shape)}, "
          f"{len(grads)} weight gradients; against 32-bit activations the fp8 ones cost {err:.3f} of the output's norm")

    # a decode step: one token, captured once and replayed
    x1, r1 = bf(1, hidden), bf(1, hidden)
    first = block.forward(x1, r1)[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1, _, _ = block.forward(x1, r1)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(first, y1)
    print(f"decode step: one token, three replays of a graph, the same bits as the eager call: {same}")
    return err, same


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:4]))
