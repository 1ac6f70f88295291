"""The operators of blocks with layer norm and biased projections on fp8
operands: what is measured, their plain forms in 32 bits and their definitions
in 64 bits.

They follow one another as layer norm -> fp8 -> projection, bias, activation ->
fp8 -> projection, bias, residual:

* ``layernorm``          -- residual addition, layer norm, and the result in the
                            input's type or cast to fp8 with scales (per
                            128-group, or per row);
  ``layernorm_backward`` -- gradients of the input, the weight and the bias;
* ``linear_act``         -- a projection of group-cast activations by
                            128x128-block weights with bias, activation and
                            residual in its epilogue;
  ``linear_act_cast``    -- the same with the fp8 cast per 128-group in place of
                            the residual;
  ``linear_act_backward`` -- gradients of the input, the weight and the bias.
"""
import math

import torch

own = False

DEV = "cuda"
HP = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
MOST = 4096 * 7168 * 18432      # the largest product


def listed():
    return [
        # one token of a decode step: latency
        {"name": "layer norm one token", "op": "layernorm", "rows": 1, "cols": 7168, "dtype": "bf16",
         "residual": True, "bias": True, "to": "group", "fmt": "e4m3fn"},
        # the activations of a long prompt or a training step
        {"name": "layer norm 16384 tokens", "op": "layernorm", "rows": 16384, "cols": 7168, "dtype": "bf16",
         "residual": True, "bias": True, "to": "group", "fmt": "e4m3fn"},
        # 32-bit activations of no particular width, not cast (the norm before a head)
        {"name": "layer norm odd width f32", "op": "layernorm", "rows": 1999, "cols": 5001, "dtype": "f32",
         "residual": False, "bias": True, "to": "plain", "fmt": "e4m3fn"},
        # training: gradients of the norm, the residual's gradient joined
        {"name": "layer norm backward", "op": "layernorm_backward", "rows": 8192, "cols": 7168, "dtype": "bf16",
         "dh": True, "bias": True},
        # a ragged batch of an odd width in 32 bits
        {"name": "layer norm backward odd width f32", "op": "layernorm_backward", "rows": 1003, "cols": 1501,
         "dtype": "f32", "dh": False, "bias": True},
        # one token of a decode step through the first projection, cast for the second
        {"name": "linear act cast one token", "op": "linear_act_cast", "rows": 1, "cols": 7168, "width": 18432,
         "dtype": "bf16", "act": "gelu", "bias": True, "keep": False, "xfmt": "e4m3fn"},
        # a training step through the first projection: cast for the second, pre-activations kept
        {"name": "linear act cast 4096 tokens", "op": "linear_act_cast", "rows": 4096, "cols": 7168, "width": 18432,
         "dtype": "bf16", "act": "gelu", "bias": True, "keep": True, "xfmt": "e4m3fn"},
        # a batch of decode steps through the second projection, added to the residual stream
        {"name": "linear residual 48 tokens", "op": "linear_act", "rows": 48, "cols": 18432, "width": 7168,
         "dtype": "bf16", "act": "none", "bias": True, "residual": True, "keep": False, "xfmt": "e4m3fn"},
        # a ragged prompt through an odd width, f16 outputs, e5m2 activations
        {"name": "linear act ragged", "op": "linear_act", "rows": 1003, "cols": 2048, "width": 1501, "dtype": "f16",
         "act": "gelu_tanh", "bias": True, "residual": True, "keep": False, "xfmt": "e5m2"},
        # a prompt through the second projection, added to the residual stream
        {"name": "linear residual 4096 tokens", "op": "linear_act", "rows": 4096, "cols": 18432, "width": 7168,
         "dtype": "bf16", "act": "none", "bias": True, "residual": True, "keep": False, "xfmt": "e4m3fn"},
        # a ragged training batch, f16 gradients, of a projection without an activation
        {"name": "linear bias backward", "op": "linear_act_backward", "rows": 3001, "cols": 4096, "width": 4096,
         "dtype": "f16", "act": "none", "bias": True, "xfmt": "e4m3fn"},
        # the backward pass of a training step's first projection
        {"name": "linear act backward", "op": "linear_act_backward", "rows": 4096, "cols": 7168, "width": 18432,
         "dtype": "bf16", "act": "gelu", "bias": True, "xfmt": "e4m3fn"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step, spread over the logarithm of step * [lo, hi]."""
    return step * max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges: rows from a single token to a
    long prompt, widths from a hundred to the largest listed."""
    op = rng.choice(["layernorm", "layernorm", "layernorm_backward", "linear_act", "linear_act", "linear_act_cast",
                     "linear_act_cast", "linear_act_backward"])
    if op == "layernorm":
        to = rng.choice(["plain", "group", "group", "row"])
        cols = _log(rng, 1, 96, 128) if to == "group" else _log(rng, 100, 12000)
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": cols, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "residual": rng.random() < 0.7, "bias": rng.random() < 0.8, "to": to,
                "fmt": rng.choice(["e4m3fn", "e4m3fn", "e5m2"])}
    if op == "layernorm_backward":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 100, 12000),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "dh": rng.random() < 0.7, "bias": rng.random() < 0.8}
    c = {"op": op, "act": rng.choice(["none", "relu", "silu", "gelu", "gelu", "gelu_tanh"]),
         "bias": rng.random() < 0.8, "xfmt": rng.choice(["e4m3fn", "e4m3fn", "e5m2"])}
    if op == "linear_act_backward":
        c.update(rows=_log(rng, 64, 4096), cols=_log(rng, 2, 56, 128), width=_log(rng, 100, 18432),
                 dtype=rng.choice(["bf16", "f16"]))
        return c
    rows, cols = _log(rng, 1, 8192), _log(rng, 2, 144, 128)
    width = _log(rng, 1, 144, 128) if op == "linear_act_cast" else _log(rng, 100, 18432)
    while rows * cols * width > MOST:
        rows = rows // 2 + 1
    c.update(rows=rows, cols=cols, width=width, keep=rng.random() < 0.5,
             dtype=rng.choice(["bf16", "f16"] if op == "linear_act_cast" else ["bf16", "f16", "f32"]))
    if op == "linear_act":
        c["residual"] = rng.random() < 0.6
    return c


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


def _stats(h):
    """mean and rstd of the rows, as a forward pass leaves them"""
    h = h.double()
    mean = h.mean(dim=1)
    return mean.float(), ((h - mean[:, None]).square().mean(dim=1) + EPS).rsqrt().float()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, rows, cols, dt = case["op"], case["rows"], case["cols"], HP[case["dtype"]]
    s = {"case": case, "bias": None, "residual": None, "z": None, "dh": None}
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=DEV)
    if op.startswith("layernorm"):
        s["weight"] = (1.0 + 0.2 * _randn(gen, cols)).to(dt)
        # rows off zero by up to about their deviation, as a residual stream's are
        x = _activations(gen, rows, cols) + 0.5 * _randn(gen, rows, 1)
        s["x"] = x.to(dt)
        if op == "layernorm":
            if case["bias"]:
                s["bias"] = (0.2 * _randn(gen, cols)).to(dt)
            if case["residual"]:
                s["residual"] = (2.0 * _randn(gen, rows, cols)).to(dt)
            h = new(rows, cols, dtype=dt) if case["residual"] else s["x"]
            if case["to"] == "plain":
                s["out"] = (new(rows, cols, dtype=dt), h, new(rows), new(rows))
            else:
                s["out"] = (new(rows, cols, dtype=FP8[case["fmt"]]),
                            new(rows, cols // 128) if case["to"] == "group" else new(rows), h, new(rows), new(rows))
        else:
            s["mean"], s["rstd"] = _stats(s["x"])
            s["dy"] = (0.01 * _randn(gen, rows, cols)).to(dt)
            if case["dh"]:
                s["dh"] = (0.01 * _randn(gen, rows, cols)).to(dt)
            s["out"] = (new(rows, cols, dtype=dt), new(cols, dtype=dt), new(cols, dtype=dt) if case["bias"] else None)
        return s
    width = case["width"]
    s["x"], s["xs"] = _cast_groups(_activations(gen, rows, cols), case["xfmt"])
    s["w"], s["ws"] = _weight(gen, width, cols)
    if op == "linear_act_backward":
        s["dy"] = (0.01 * _randn(gen, rows, width)).to(dt)
        if case["act"] != "none":
            s["z"] = (1.5 * _randn(gen, rows, width)).to(dt)
        s["out"] = (new(rows, cols, dtype=dt), new(width, cols, dtype=dt), new(width, dtype=dt) if case["bias"] else None)
        return s
    if case["bias"]:
        s["bias"] = (0.2 * _randn(gen, width)).to(dt)
    z = new(rows, width, dtype=dt) if case["keep"] else None
    if op == "linear_act_cast":
        s["out"] = (new(rows, width, dtype=FP8["e4m3fn"]), new(rows, width // 128), z)
    else:
        if case["residual"]:
            s["residual"] = (2.0 * _randn(gen, rows, width)).to(dt)
        s["out"] = (new(rows, width, dtype=dt), z)
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import dequantize_amax_reduce_amd as fq
    c = s["case"]
    op = c["op"]
    if op == "layernorm" and c["to"] == "plain":
        y, h, mean, rstd = fq.layernorm(s["x"], s["weight"], s["bias"], s["residual"], EPS, out=s["out"])
        return {"y": y, "h": h if c["residual"] else None, "mean": mean, "rstd": rstd}
    if op == "layernorm":
        q, si, h, mean, rstd = fq.layernorm_cast(s["x"], s["weight"], s["bias"], s["residual"], EPS, c["fmt"],
                                                 per_channel_scale=c["to"] == "row", out=s["out"])
        return {"q": q, "scale_inv": si, "h": h if c["residual"] else None, "mean": mean, "rstd": rstd}
    if op == "layernorm_backward":
        dx, dw, db = fq.layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dh"],
                                           with_bias=c["bias"], out=s["out"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    act = None if c["act"] == "none" else c["act"]
    if op == "linear_act":
        y, z = fq.linear_act_fp8(s["x"], s["xs"], s["w"], s["ws"], s["bias"], act, s["residual"], out=s["out"])
        return {"y": y, "z": z}
    if op == "linear_act_cast":
        q, si, z = fq.linear_act_fp8_cast(s["x"], s["xs"], s["w"], s["ws"], s["bias"], act, "e4m3fn", out=s["out"])
        return {"q": q, "scale_inv": si, "z": z}
    dx, dw, db = fq.linear_act_fp8_backward(s["dy"], s["z"], s["x"], s["xs"], s["w"], s["ws"], act,
                                            with_bias=c["bias"], out=s["out"])
    return {"dx": dx, "dw": dw, "dbias": db}


# ---------------------------------------------------------------------------
# the plain forms (32 bits, rounded once at the end)
# ---------------------------------------------------------------------------

def _rows32(q, s):
    rows, cols = q.shape
    return (q.float().view(rows, cols // 128, 128) * s[:, :, None]).view(rows, cols)


def _blocks32(q, s):
    n = q.shape[0]
    return q.float() * s.repeat_interleave(128, dim=0)[:n].repeat_interleave(128, dim=1)


def _act32(name, z):
    """(the activation, its derivative)"""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).float()
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return z * sg, sg * (1.0 + z * (1.0 - sg))
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * 0.7071067811865476))
        return z * c, c + z * 0.3989422804014327 * torch.exp(-0.5 * z * z)
    k = 0.7978845608028654
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, dt = c["op"], HP[c["dtype"]]
    if op == "layernorm":
        h = s["x"].float()
        if c["residual"]:
            h = h + s["residual"].float()
        mean = h.mean(dim=1)
        d = h - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + EPS)
        y = d * rstd[:, None] * s["weight"].float()
        if c["bias"]:
            y = y + s["bias"].float()
        o = {"h": h.to(dt) if c["residual"] else None, "mean": mean, "rstd": rstd}
        if c["to"] == "plain":
            return {"y": y.to(dt), **o}
        if c["to"] == "group":
            q, si = _cast_groups(y, c["fmt"])
        else:
            amax = y.abs().amax(dim=1)
            amax = torch.where(amax > 0, amax, torch.ones_like(amax))
            q, si = _fp8(y * (FP8_MAX[c["fmt"]] / amax)[:, None], c["fmt"]), amax / FP8_MAX[c["fmt"]]
        return {"q": q, "scale_inv": si, **o}
    if op == "layernorm_backward":
        rs = s["rstd"][:, None]
        n = (s["x"].float() - s["mean"][:, None]) * rs
        dy = s["dy"].float()
        dn = dy * s["weight"].float()
        dx = (dn - dn.mean(dim=1, keepdim=True) - n * (dn * n).mean(dim=1, keepdim=True)) * rs
        if c["dh"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * n).sum(dim=0).to(dt), "dbias": dy.sum(dim=0).to(dt) if c["bias"] else None}
    x, w = _rows32(s["x"], s["xs"]), _blocks32(s["w"], s["ws"])
    if op == "linear_act_backward":
        dz = s["dy"].float()
        if c["act"] != "none":
            dz = dz * _act32(c["act"], s["z"].float())[1]
        return {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt), "dbias": dz.sum(dim=0).to(dt) if c["bias"] else None}
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act32(c["act"], z)[0]
    kept = z.to(dt) if c["keep"] else None
    if op == "linear_act_cast":
        q, si = _cast_groups(y, "e4m3fn")
        return {"q": q, "scale_inv": si, "z": kept}
    if c["residual"]:
        y = y + s["residual"].float()
    return {"y": y.to(dt), "z": kept}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, m, k = case["op"], case["rows"], case["cols"]
    e = BYTES[case["dtype"]]
    if op == "layernorm":
        scales = {"plain": 0, "row": m, "group": m * (k // 128)}[case["to"]]
        r = 2 if case["residual"] else 0                    # the residual in, the sum out
        out = e if case["to"] == "plain" else 1
        return {"bytes": m * k * (e * (1 + r) + out) + 4 * (scales + 2 * m) + e * k * (1 + case["bias"]),
                "flops": 10 * m * k}
    if op == "layernorm_backward":
        return {"bytes": m * k * e * (3 + case["dh"]) + 8 * m + e * k * (2 + case["bias"]), "flops": 16 * m * k}
    n = case["width"]
    x = m * k + 4 * m * (k // 128)
    w = n * k + 4 * (-(-n // 128)) * (k // 128)
    if op == "linear_act_backward":
        act = case["act"] != "none"
        return {"bytes": m * n * e * (1 + act) + x + w + m * k * e + n * k * e + n * e * case["bias"],
                "flops": 4 * m * n * k + 10 * m * n * act}
    out = m * n + 4 * m * (n // 128) if op == "linear_act_cast" else m * n * e * (1 + case["residual"])
    return {"bytes": x + w + out + m * n * e * case["keep"] + n * e * case["bias"],
            "flops": 2 * m * n * k + (0 if case["act"] == "none" else 6 * m * n)}


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
        at = torch.arange(q.shape[0], device=DEV) // br
        return q.to(D).mul_(sc.to(D)[at].repeat_interleave(128, dim=1))

    def act(g):
        a = case["act"]
        if a == "none":
            return g, torch.ones_like(g)
        if a == "relu":
            return g.clamp_min(0.0), torch.heaviside(g, torch.zeros((), dtype=D, device=DEV))
        if a == "silu":
            sg = torch.sigmoid(g)
            return g * sg, sg + g * sg * (1 - sg)
        if a == "gelu":
            p = torch.special.ndtr(g)
            return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        # (1 + tanh v) / 2 as the logistic function of 2 v, which keeps its tail
        k = 2 * math.sqrt(2 / math.pi)
        t = torch.sigmoid(k * (g + 0.044715 * g ** 3))
        return g * t, t + g * t * (1 - t) * k * (1 + 0.134145 * g ** 2)

    if op == "layernorm":
        h = s["x"].to(D)
        if case["residual"]:
            h = h + s["residual"].to(D)
        var, mean = torch.var_mean(h, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = (h - mean[:, None]) * (rstd[:, None] * s["weight"].to(D))
        if case["bias"]:
            y += s["bias"].to(D)
        o = {"h": h if case["residual"] else None, "mean": mean, "rstd": rstd}
        if case["to"] == "plain":
            return {"y": y, **o}
        q, si = scaled(y, case["fmt"], case["to"] == "group")
        return {"q": q, "scale_inv": si, **o}
    if op == "layernorm_backward":
        r, dy = s["rstd"].to(D)[:, None], s["dy"].to(D)
        c = s["x"].to(D) - s["mean"].to(D)[:, None]
        g = dy * s["weight"].to(D)
        n = case["cols"]
        dx = r * (g - g.sum(dim=1, keepdim=True) / n) - r ** 3 * c * ((g * c).sum(dim=1, keepdim=True) / n)
        return {"dx": dx + s["dh"].to(D) if case["dh"] else dx, "dweight": (dy * (c * r)).sum(dim=0),
                "dbias": dy.sum(dim=0) if case["bias"] else None}
    x, w = widen(s["x"], s["xs"], 1), widen(s["w"], s["ws"], 128)
    if op == "linear_act_backward":
        g = s["dy"].to(D)
        if case["act"] != "none":
            g = g * act(s["z"].to(D))[1]
        return {"dx": g @ w, "dw": g.t() @ x, "dbias": g.sum(dim=0) if case["bias"] else None}
    z = x @ w.t()
    if case["bias"]:
        z += s["bias"].to(D)
    y = act(z)[0]
    kept = z if case["keep"] else None
    if op == "linear_act_cast":
        q, si = scaled(y, "e4m3fn", True)
        return {"q": q, "scale_inv": si, "z": kept}
    return {"y": y + s["residual"].to(D) if case["residual"] else y, "z": kept}
