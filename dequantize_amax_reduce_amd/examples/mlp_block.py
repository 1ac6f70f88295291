"""A block with layer norm and biased projections on fp8 operands, as a
training step and as a decode step: residual + layer norm -> fp8 -> first
projection, bias, GELU -> fp8 -> second projection, bias, residual, and the
gradients of all of it.

    python dequantize_amax_reduce_amd/examples/mlp_block.py [tokens] [hidden] [width]

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
    def __init__(self, hidden, width, device="cuda", activation="gelu"):
        r = lambda *s: torch.randn(*s, device=device)
        bf = lambda t: t.to(torch.bfloat16)
        self.norm = bf(1 + 0.1 * r(hidden)), bf(0.1 * r(hidden))
        self.up, self.down = (quantize_weight(r(n, k) * k ** -0.5) for n, k in ((width, hidden), (hidden, width)))
        self.up_bias, self.down_bias = bf(0.1 * r(width)), bf(0.1 * r(hidden))
        self.activation = activation

    def forward(self, x, residual, keep=False):
        """(the new residual stream, what backward reads)"""
        q, s, h, mean, rstd = fq.layernorm_cast(x, *self.norm, residual)
        p, ps, z = fq.linear_act_fp8_cast(q, s, *self.up, self.up_bias, self.activation,
                                          keep=torch.bfloat16 if keep else None)
        y, _ = fq.linear_act_fp8(p, ps, *self.down, self.down_bias, residual=h)
        return y, (q, s, h, mean, rstd, p, ps, z)

    def backward(self, dy, kept):
        """Gradients of x (and of the residual alike) and of the parameters,
        from that of the new residual stream."""
        q, s, h, mean, rstd, p, ps, z = kept
        dp, d_down, d_down_bias = fq.linear_act_fp8_backward(dy, None, p, ps, *self.down)
        dn, d_up, d_up_bias = fq.linear_act_fp8_backward(dp, z, q, s, *self.up, self.activation)
        dx, d_norm, d_norm_bias = fq.layernorm_backward(dn, h, self.norm[0], mean, rstd, dy)
        return dx, (d_norm, d_norm_bias, d_up, d_up_bias, d_down, d_down_bias)


def main(tokens=2048, hidden=2048, width=8192):
    torch.manual_seed(0)
    block = Block(hidden, width)
    bf = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16)

    # a training step
    x, residual = bf(tokens, hidden), bf(tokens, hidden)
    y, kept = block.forward(x, residual, keep=True)
    dx, grads = block.backward(bf(tokens, hidden) * 0.01, kept)

    # the same block in plain 32-bit torch, from the weights' own values
    deq = lambda q, s: fq.weight_dequant(q, s, ret_type=torch.float32)
    hf = x.float() + residual.float()
    n = (hf - hf.mean(1, keepdim=True)) * torch.rsqrt(hf.var(1, correction=0, keepdim=True) + 1e-5)
    n = n * block.norm[0].float() + block.norm[1].float()
    ref = torch.nn.functional.gelu(n @ deq(*block.up).t() + block.up_bias.float()) @ deq(*block.down).t()
    ref = ref + block.down_bias.float()
    err = float((y.float() - hf - ref).norm() / ref.norm())
    print(f"training step: {tokens} tokens, output {tuple(y.shape)}, dx {tuple(dx.shape)}, "
          f"{len(grads)} parameter gradients; against 32-bit activations the fp8 ones cost {err:.3f} of the norm of "
          "what the block adds")

    # a decode step: one token, captured once and replayed
    x1, r1 = bf(1, hidden), bf(1, hidden)
    first = block.forward(x1, r1)[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1, _ = block.forward(x1, r1)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(first, y1)
    print(f"decode step: one token, three replays of a graph, the same bits as the eager call: {same}")
    return err, same


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:4]))
