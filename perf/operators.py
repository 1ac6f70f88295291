"""The feed-forward operators on fp8 operands: what is measured, their plain
forms in 32 bits and their definitions in 64 bits.

Three operators that follow one another in a feed-forward block whose matrix
products run on fp8 codes with scales (activations per 128-element group,
weights per 128x128 block):

* ``norm``    -- residual addition, root-mean-square norm and the cast of the
                 result to fp8 with scales (per 128-group, or per row);
  ``norm_backward`` -- its gradients (the cast passes gradients through);
* ``gated``   -- the gate and up projections, the activation and the product,
                 written in 16 bits or cast to fp8 per 128-group, with the
                 pre-activations kept for a backward pass where asked;
  ``gated_backward`` -- gradients of the input and of both weights;
* ``linear``  -- one projection (the block's second half);
  ``linear_backward`` -- gradients of its input and weight.
"""
import math

import torch

own = False

DEV = "cuda"
HP = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # one token of a decode step: latency
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 7168, "dtype": "bf16", "residual": True,
         "scales": "group", "fmt": "e4m3fn"},
        # the activations of a long prompt or a training step
        {"name": "norm 16384 tokens", "op": "norm", "rows": 16384, "cols": 7168, "dtype": "bf16", "residual": True,
         "scales": "group", "fmt": "e4m3fn"},
        # 32-bit activations, one scale a row, a width of no particular alignment, no residual
        {"name": "norm odd width f32", "op": "norm", "rows": 1999, "cols": 5001, "dtype": "f32", "residual": False,
         "scales": "row", "fmt": "e5m2"},
        # training: gradients of the norm, the residual's gradient joined
        {"name": "norm backward", "op": "norm_backward", "rows": 8192, "cols": 7168, "dtype": "bf16", "dh": True},
        # one token of a decode step through the gate and up projections: the weights' bytes
        {"name": "gated one token", "op": "gated", "rows": 1, "cols": 7168, "width": 18432, "dtype": "bf16",
         "act": "silu", "cast": False, "keep": False, "xfmt": "e4m3fn"},
        # a batch of decode steps, handed to the next projection in fp8
        {"name": "gated 48 tokens", "op": "gated", "rows": 48, "cols": 4096, "width": 4096, "dtype": "bf16",
         "act": "silu", "cast": True, "keep": False, "xfmt": "e4m3fn"},
        # a ragged prompt through an odd width, f16 outputs, e5m2 activations
        {"name": "gated ragged", "op": "gated", "rows": 1003, "cols": 2048, "width": 1501, "dtype": "f16",
         "act": "gelu_tanh", "cast": False, "keep": False, "xfmt": "e5m2"},
        # a training step: fp8 output for the next projection, pre-activations kept
        {"name": "gated 4096 tokens", "op": "gated", "rows": 4096, "cols": 7168, "width": 18432, "dtype": "bf16",
         "act": "silu", "cast": True, "keep": True, "xfmt": "e4m3fn"},
        # its backward pass
        {"name": "gated backward", "op": "gated_backward", "rows": 4096, "cols": 7168, "width": 18432,
         "dtype": "bf16", "act": "silu", "xfmt": "e4m3fn"},
        # a batch of decode steps through the second projection
        {"name": "linear 16 tokens", "op": "linear", "rows": 16, "cols": 18432, "width": 7168, "dtype": "bf16",
         "xfmt": "e4m3fn"},
        # a prompt through the second projection
        {"name": "linear 4096 tokens", "op": "linear", "rows": 4096, "cols": 18432, "width": 7168, "dtype": "bf16",
         "xfmt": "e4m3fn"},
        # a ragged training batch, f16 gradients
        {"name": "linear backward", "op": "linear_backward", "rows": 3001, "cols": 4096, "width": 4096,
         "dtype": "f16", "xfmt": "e4m3fn"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step, spread over the logarithm of step * [lo, hi] (3072
    is no size of this library's workloads)."""
    n = 0
    while n == 0 or n == 3072:
        n = step * max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n


def draw(rng):
    """One more case of the listed ones' ranges: rows from a single token to a
    long prompt, widths from a hundred to the largest listed."""
    op = rng.choice(["norm", "norm", "norm_backward", "gated", "gated", "gated_backward", "linear", "linear",
                     "linear_backward"])
    if op == "norm":
        scales = rng.choice(["group", "row"])
        cols = _log(rng, 1, 64, 128) if scales == "group" else _log(rng, 100, 12000)
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": cols, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "residual": rng.random() < 0.7, "scales": scales, "fmt": rng.choice(["e4m3fn", "e4m3fn", "e5m2"])}
    if op == "norm_backward":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 100, 8192),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "dh": rng.random() < 0.7}
    cols = _log(rng, 2, 56, 128)
    xfmt = rng.choice(["e4m3fn", "e4m3fn", "e5m2"])
    if op == "linear":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 2, 100, 128), "width": _log(rng, 100, 7168),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "xfmt": xfmt}
    if op == "linear_backward":
        return {"op": op, "rows": _log(rng, 64, 4096), "cols": cols, "width": _log(rng, 100, 8192),
                "dtype": rng.choice(["bf16", "f16"]), "xfmt": xfmt}
    act = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    if op == "gated":
        cast = rng.random() < 0.5
        width = _log(rng, 1, 144, 128) if cast else _log(rng, 100, 18432)
        rows = _log(rng, 1, 8192)
        if rows * cols * width > 4096 * 7168 * 18432:
            rows //= 4
        return {"op": op, "rows": rows, "cols": cols, "width": width, "dtype": rng.choice(["bf16", "f16"]),
                "act": act, "cast": cast, "keep": rng.random() < 0.5, "xfmt": xfmt}
    return {"op": op, "rows": _log(rng, 64, 4096), "cols": cols, "width": _log(rng, 100, 18432),
            "dtype": rng.choice(["bf16", "f16"]), "act": act, "xfmt": xfmt}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _activations(gen, rows, cols):
    """N(0, 1) with a few channels 20 times larger and, in longer batches, a
    few all-zero rows (padding)."""
    x = _randn(gen, rows, cols)
    x[:, torch.randint(0, cols, (max(1, cols // 1000),), generator=gen, device=DEV)] *= 20.0
    if rows >= 64:
        x[torch.randint(0, rows, (rows // 64,), generator=gen, device=DEV)] = 0.0
    return x


def _fp8(v, fmt):
    return v.clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(FP8[fmt])


def _cast_groups(x, fmt):
    rows, cols = x.shape
    g = x.view(rows, cols // 128, 128)
    amax = g.abs().amax(dim=2).clamp_min(1e-4)
    return _fp8(g * (FP8_MAX[fmt] / amax)[:, :, None], fmt).view(rows, cols), amax / FP8_MAX[fmt]


def _weight(gen, n, k):
    """A weight of N(0, 1/k), every 128x128 block of its own magnitude, as
    e4m3fn codes with one scale a block."""
    nb, kb = -(-n // 128), k // 128
    w = torch.zeros(nb * 128, k, device=DEV)
    w[:n] = _randn(gen, n, k) * k ** -0.5
    b = w.view(nb, 128, kb, 128)
    b *= torch.exp(0.5 * _randn(gen, nb, 1, kb, 1))
    amax = b.abs().amax(dim=(1, 3)).clamp_min(1e-8)
    q = _fp8(b * (448.0 / amax)[:, None, :, None], "e4m3fn").view(nb * 128, k)[:n].contiguous()
    return q, amax / 448.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    s = {"case": case}
    if op in ("norm", "norm_backward"):
        dt = HP[case["dtype"]]
        s["weight"] = (1.0 + 0.2 * _randn(gen, cols)).to(dt)
        s["x"] = _activations(gen, rows, cols).to(dt)
        if op == "norm":
            s["residual"] = (2.0 * _randn(gen, rows, cols)).to(dt) if case["residual"] else None
            shape = (rows, cols // 128) if case["scales"] == "group" else (rows,)
            s["out"] = (torch.empty(rows, cols, dtype=FP8[case["fmt"]], device=DEV),
                        torch.empty(shape, dtype=torch.float32, device=DEV),
                        torch.empty(rows, cols, dtype=dt, device=DEV) if case["residual"] else s["x"],
                        torch.empty(rows, dtype=torch.float32, device=DEV))
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(dim=1) + EPS)
            s["dy"] = (0.01 * _randn(gen, rows, cols)).to(dt)
            s["dh"] = (0.01 * _randn(gen, rows, cols)).to(dt) if case["dh"] else None
            s["out"] = (torch.empty(rows, cols, dtype=dt, device=DEV), torch.empty(cols, dtype=dt, device=DEV))
        return s
    width, dt = case["width"], HP[case["dtype"]]
    s["x"], s["xs"] = _cast_groups(_activations(gen, rows, cols), case["xfmt"])
    s["w"], s["ws"] = _weight(gen, width, cols)
    if op.startswith("gated"):
        s["w2"], s["ws2"] = _weight(gen, width, cols)
    if op == "gated":
        z = torch.empty(rows, 2 * width, dtype=dt, device=DEV) if case["keep"] else None
        if case["cast"]:
            s["out"] = (torch.empty(rows, width, dtype=FP8["e4m3fn"], device=DEV),
                        torch.empty(rows, width // 128, dtype=torch.float32, device=DEV), z)
        else:
            s["out"] = (torch.empty(rows, width, dtype=dt, device=DEV), z)
    elif op == "linear":
        s["out"] = torch.empty(rows, width, dtype=dt, device=DEV)
    else:
        s["dy"] = (0.01 * _randn(gen, rows, width)).to(dt)
        grads = [torch.empty(rows, cols, dtype=dt, device=DEV), torch.empty(width, cols, dtype=dt, device=DEV)]
        if op == "gated_backward":
            s["z"] = (1.5 * _randn(gen, rows, 2 * width)).to(dt)
            grads.append(torch.empty(width, cols, dtype=dt, device=DEV))
        s["out"] = tuple(grads)
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import dequantize_amax_reduce_amd as fq
    c = s["case"]
    op = c["op"]
    if op == "norm":
        q, si, h, rstd = fq.rmsnorm_cast(s["x"], s["weight"], s["residual"], EPS, c["fmt"],
                                         per_channel_scale=c["scales"] == "row", out=s["out"])
        return {"q": q, "scale_inv": si, "h": h if c["residual"] else None, "rstd": rstd}
    if op == "norm_backward":
        dx, dw = fq.rmsnorm_cast_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dh"], out=s["out"])
        return {"dx": dx, "dweight": dw}
    if op == "gated" and c["cast"]:
        q, si, z = fq.gated_linear_fp8_cast(s["x"], s["xs"], s["w"], s["ws"], s["w2"], s["ws2"], c["act"], "e4m3fn",
                                        out=s["out"])
        return {"q": q, "scale_inv": si, "z": z}
    if op == "gated":
        h, z = fq.gated_linear_fp8(s["x"], s["xs"], s["w"], s["ws"], s["w2"], s["ws2"], c["act"], out=s["out"])
        return {"h": h, "z": z}
    if op == "gated_backward":
        dx, dwg, dwu = fq.gated_linear_fp8_backward(s["dy"], s["z"], s["x"], s["xs"], s["w"], s["ws"], s["w2"],
                                                s["ws2"], c["act"], out=s["out"])
        return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
    if op == "linear":
        return {"y": fq.linear_fp8(s["x"], s["xs"], s["w"], s["ws"], out=s["out"])}
    dx, dw = fq.linear_fp8_backward(s["dy"], s["x"], s["xs"], s["w"], s["ws"], out=s["out"])
    return {"dx": dx, "dw": dw}


# ---------------------------------------------------------------------------
# the plain forms (32 bits, rounded once at the end)
# ---------------------------------------------------------------------------

def _rows32(q, s):
    rows, cols = q.shape
    return (q.float().view(rows, cols // 128, 128) * s[:, :, None]).view(rows, cols)


def _blocks32(q, s):
    n = q.shape[0]
    return q.float() * s.repeat_interleave(128, dim=0)[:n].repeat_interleave(128, dim=1)


def _act32(name, g):
    """(the activation, its derivative)"""
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * 0.7071067811865476))
        return g * c, c + g * 0.3989422804014327 * torch.exp(-0.5 * g * g)
    k = 0.7978845608028654
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op = c["op"]
    if op == "norm":
        h = s["x"].float()
        if c["residual"]:
            h = h + s["residual"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(dim=1) + EPS)
        y = h * rstd[:, None] * s["weight"].float()
        if c["scales"] == "group":
            q, si = _cast_groups(y, c["fmt"])
        else:
            amax = y.abs().amax(dim=1)
            amax = torch.where(amax > 0, amax, torch.ones_like(amax))
            q, si = _fp8(y * (FP8_MAX[c["fmt"]] / amax)[:, None], c["fmt"]), amax / FP8_MAX[c["fmt"]]
        return {"q": q, "scale_inv": si, "h": h.to(s["x"].dtype) if c["residual"] else None, "rstd": rstd}
    if op == "norm_backward":
        n = s["x"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        dn = dy * s["weight"].float()
        dx = (dn - n * (dn * n).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(dim=0).to(s["weight"].dtype)}
    x, w, dt = _rows32(s["x"], s["xs"]), _blocks32(s["w"], s["ws"]), HP[c["dtype"]]
    if op == "linear":
        return {"y": (x @ w.t()).to(dt)}
    if op == "linear_backward":
        dy = s["dy"].float()
        return {"dx": (dy @ w).to(dt), "dw": (dy.t() @ x).to(dt)}
    w2 = _blocks32(s["w2"], s["ws2"])
    if op == "gated":
        g, u = x @ w.t(), x @ w2.t()
        h = _act32(c["act"], g)[0] * u
        z = torch.cat((g, u), dim=1).to(dt) if c["keep"] else None
        if c["cast"]:
            q, si = _cast_groups(h, "e4m3fn")
            return {"q": q, "scale_inv": si, "z": z}
        return {"h": h.to(dt), "z": z}
    width = c["width"]
    dh, g, u = s["dy"].float(), s["z"][:, :width].float(), s["z"][:, width:].float()
    a, da = _act32(c["act"], g)
    dg, du = dh * u * da, dh * a
    return {"dx": (dg @ w + du @ w2).to(dt), "dw_gate": (dg.t() @ x).to(dt), "dw_up": (du.t() @ x).to(dt)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, m, k = case["op"], case["rows"], case["cols"]
    e = BYTES[case["dtype"]]
    if op == "norm":
        scales = m * (k // 128) if case["scales"] == "group" else m
        r = 2 if case["residual"] else 0                    # the residual in, the sum out
        return {"bytes": m * k * (e * (1 + r) + 1) + 4 * (scales + m) + e * k, "flops": 8 * m * k}
    if op == "norm_backward":
        return {"bytes": m * k * e * (3 + case["dh"]) + 4 * m + 2 * e * k, "flops": 12 * m * k}
    n = case["width"]
    x = m * k + 4 * m * (k // 128)
    w = n * k + 4 * (-(-n // 128)) * (k // 128)
    if op == "linear":
        return {"bytes": x + w + m * n * e, "flops": 2 * m * n * k}
    if op == "linear_backward":
        return {"bytes": m * n * e + x + w + m * k * e + n * k * e, "flops": 4 * m * n * k}
    if op == "gated":
        out = m * n + 4 * m * (n // 128) if case["cast"] else m * n * e
        return {"bytes": x + 2 * w + out + (2 * m * n * e if case["keep"] else 0), "flops": 4 * m * n * k + 6 * m * n}
    return {"bytes": 3 * m * n * e + x + 2 * w + m * k * e + 2 * n * k * e, "flops": 8 * m * n * k + 12 * m * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """From the definitions, in 64 bits: fp8 outputs as the scaled values
    before their rounding to 8 bits."""
    s = prepare(case, seed)
    op = case["op"]
    D = torch.float64

    def scaled(y, fmt, group):
        if group:
            v = y.reshape(y.shape[0], -1, 128)
            a = torch.maximum(v.abs().max(dim=2).values, torch.tensor(float(torch.tensor(1e-4)), dtype=D, device=DEV))
            return (v / a[:, :, None] * FP8_MAX[fmt]).reshape(y.shape), a / FP8_MAX[fmt]
        a = y.abs().max(dim=1).values
        a[a == 0] = 1.0
        return y / a[:, None] * FP8_MAX[fmt], a / FP8_MAX[fmt]

    def widen(q, sc, br):
        rows, cols = q.shape
        at = torch.arange(rows, device=DEV) // br
        return q.to(D).mul_(sc.to(D)[at].repeat_interleave(128, dim=1)[:, :cols])

    def act(g):
        if case["act"] == "silu":
            sg = torch.sigmoid(g)
            return g * sg, sg + g * sg * (1 - sg)
        if case["act"] == "gelu":
            p = torch.special.ndtr(g)
            return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t ** 2) * k * (1 + 0.134145 * g ** 2) / 2

    if op == "norm":
        h = s["x"].to(D) if s["residual"] is None else s["x"].to(D) + s["residual"].to(D)
        rstd = (h.square().sum(dim=1) / case["cols"] + EPS) ** -0.5
        q, si = scaled(h * rstd[:, None] * s["weight"].to(D), case["fmt"], case["scales"] == "group")
        return {"q": q, "scale_inv": si, "h": h if case["residual"] else None, "rstd": rstd}
    if op == "norm_backward":
        h, r, dy = s["x"].to(D), s["rstd"].to(D)[:, None], s["dy"].to(D)
        dn = dy * s["weight"].to(D)
        dx = r * dn - r ** 3 * h * ((dn * h).sum(dim=1, keepdim=True) / case["cols"])
        return {"dx": dx if s["dh"] is None else dx + s["dh"].to(D), "dweight": ((dy * r) * h).sum(dim=0)}
    x = widen(s["x"], s["xs"], 1)
    if op == "linear":
        return {"y": x @ widen(s["w"], s["ws"], 128).t()}
    if op == "linear_backward":
        dy = s["dy"].to(D)
        return {"dx": dy @ widen(s["w"], s["ws"], 128), "dw": dy.t() @ x}
    if op == "gated":
        g = x @ widen(s["w"], s["ws"], 128).t()
        u = x @ widen(s["w2"], s["ws2"], 128).t()
        z = torch.cat([g, u], dim=1) if case["keep"] else None
        h = act(g)[0] * u
        if case["cast"]:
            q, si = scaled(h, "e4m3fn", True)
            return {"q": q, "scale_inv": si, "z": z}
        return {"h": h, "z": z}
    n = case["width"]
    a, da = act(s["z"][:, :n].to(D))
    dh = s["dy"].to(D)
    dg, du = dh * da * s["z"][:, n:].to(D), dh * a
    dx = dg @ widen(s["w"], s["ws"], 128) + du @ widen(s["w2"], s["ws2"], 128)
    return {"dx": dx, "dw_gate": dg.t() @ x, "dw_up": du.t() @ x}
