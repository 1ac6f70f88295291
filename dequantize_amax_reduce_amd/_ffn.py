"""Binding of include/fp8q_ffn.h: the feed-forward operators on fp8 operands.

Re-exported by the package.  As there, two layers: ``fp8q_*`` mirror the C
entry points (caller-allocated outputs and workspaces), and the helpers below
them allocate outputs and workspaces with torch.  Codes are float8 tensors, or
uint8 ones of the formats x_fmt and w_fmt name (e4m3fn where they do not).

    q, s, h, rstd = rmsnorm_cast(x, weight, residual)          # norm -> fp8 per 128-group
    q2, s2, z = gated_linear_fp8_cast(q, s, wg, wgs, wu, wus, keep=torch.bfloat16)
    y = linear_fp8(q2, s2, wd, wds)
    dp, dwd = linear_fp8_backward(dy, q2, s2, wd, wds)
    dn, dwg, dwu = gated_linear_fp8_backward(dp, z, q, s, wg, wgs, wu, wus)
    dx, dweight = rmsnorm_cast_backward(dn, h, weight, rstd, dh)
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

SILU, GELU, GELU_TANH = range(3)
_ACT = {"silu": SILU, "gelu": GELU, "gelu_tanh": GELU_TANH, SILU: SILU, GELU: GELU, GELU_TANH: GELU_TANH}

FFN_HEADER_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8q_ffn.h")

_P, _I64, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_CODES = [_P, _I, _P]                                   # codes, format, scale_inv
_PAIR = [_P, _P, _P, _P, _I]                            # w_gate, scale, w_up, scale, format
FFN_SIGNATURES = {
    "fp8q_rmsnorm_cast_group128": (_I, [_P, _I, _P, _P, _I, _I64, _I64, _F, _I, _P, _P, _P, _P, _P]),
    "fp8q_rmsnorm_cast_per_channel": (_I, [_P, _I, _P, _P, _I, _I64, _I64, _F, _I, _P, _P, _P, _P, _P]),
    "fp8q_rmsnorm_backward_workspace_bytes": (_SZ, [_I64, _I64]),
    "fp8q_rmsnorm_backward": (_I, [_P, _P, _I, _P, _I, _P, _P, _I64, _I64, _P, _P, _P, _P]),
    "fp8q_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8q_linear": (_I, _CODES + _CODES + [_I64, _I64, _I64, _P, _I, _P, _P]),
    "fp8q_linear_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8q_linear_backward": (_I, [_P, _I] + _CODES + _CODES + [_I64, _I64, _I64, _P, _P, _I, _P, _P]),
    "fp8q_gated_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "fp8q_gated_linear": (_I, _CODES + _PAIR + [_I64, _I64, _I64, _I, _P, _I, _P, _I, _P, _P]),
    "fp8q_gated_linear_cast": (_I, _CODES + _PAIR + [_I64, _I64, _I64, _I, _I, _P, _P, _P, _I, _P, _P]),
    "fp8q_gated_linear_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8q_gated_linear_backward": (_I, [_P, _P, _I] + _CODES + _PAIR + [_I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P]),
}
FFN_FUNCTIONS = tuple(FFN_SIGNATURES)


def load_ffn(L):
    """Set the signatures of the feed-forward entry points on a library handle."""
    for name, (res, args) in FFN_SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def ffn_header_functions() -> list:
    """Names of the functions include/fp8q_ffn.h declares."""
    with open(FFN_HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^(?:fp8q_status_t|size_t)\s+(fp8q_\w+)\s*\(", text, re.M)))


# set by the package once its own marshalling helpers exist
lib = _check = _dev = _fmt = _fp8 = _FP8_DTYPE = _DT = None


def _bind(package_lib, helpers):
    global lib
    lib = load_ffn(package_lib)
    globals().update(helpers)


# A call on one token is bound by its host time, so the marshalling asks each
# tensor as little as it can (about 0.25 us a tensor against 0.7 us for _dev).

def _ptr(t, name) -> int:
    try:
        if t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _dev(t, name)                                # raises, or 0 for an empty tensor


# the raw handle of a device's current stream; torch.cuda.current_stream costs 2 us more
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(t, stream):
    if stream is None:
        return _raw_stream(t.get_device()) if t.is_cuda else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _hp_dtype(t, name) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name}: only float32, bfloat16 and float16 are supported (got {t.dtype})")
    return dt


def _act(name) -> int:
    if name not in _ACT:
        raise TypeError(f"unknown activation {name!r} (use 'silu', 'gelu' or 'gelu_tanh')")
    return _ACT[name]


def _opt(t, name):
    return 0 if t is None else _ptr(t, name)


def _f32(t, numel, name):
    if t.dtype != torch.float32 or t.numel() != numel:
        raise ValueError(f"{name} must be float32 with {numel} elements")
    return _ptr(t, name)


def _flat(t, name):
    """(rows, last dimension) of a tensor of at least one dimension."""
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    k = t.shape[-1]
    if t.dim() == 2:
        return t.shape[0], k
    rows = 1
    for d in t.shape[:-1]:
        rows *= d
    return rows, k


def _same(t, shape, dtype, name):
    if t is not None and (t.numel() != shape[0] * shape[1] or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} with {shape[0]} x {shape[1]} elements")
    return t


_AUTO = object()                                        # the helpers' workspaces: allocated within the call


def _ws(t, need, like, name):
    """The workspace tensor of a call (the caller keeps it until the call has
    been enqueued), or None where none is needed."""
    if need == 0:
        return None
    if t is _AUTO:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    if t is None or t.numel() * t.element_size() < need:
        raise ValueError(f"{name}: the workspace needs {need} bytes")
    return t


def _x_codes(x, xs, f):
    """(pointer, format, scale pointer), rows, K of an activation of format f"""
    M, K = _flat(x, "x")
    return (_ptr(x, "x"), f, _f32(xs, M * (K // 128), "x_scale_inv")), M, K


def _w_codes(w, ws, K, name):
    """pointer, scale pointer, rows of a weight"""
    if w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"{name} must be 2-D with {K} columns")
    N = w.shape[0]
    return _ptr(w, name), _f32(ws, ((N + 127) // 128) * (K // 128), "the weight's scale_inv"), N


def _formats(x, x_fmt, w_fmt, *weights):
    """The formats of x and of the weights, before anything else is asked of
    them; x_fmt and w_fmt name those of uint8 codes."""
    xf, wf = _fp8(x, x_fmt, "x"), _fp8(weights[0], w_fmt, "the weight")
    if len(weights) > 1 and _fp8(weights[1], w_fmt, "w_up") != wf:
        raise ValueError("w_gate and w_up must have the same shape and format")
    return xf, wf


def _pair(w_gate, gs, w_up, us, K, f):
    g, gsp, F = _w_codes(w_gate, gs, K, "w_gate")
    u, usp, F2 = _w_codes(w_up, us, K, "w_up")
    if F != F2:
        raise ValueError("w_gate and w_up must have the same shape and format")
    return (g, gsp, u, usp, f), F


# ---------------------------------------------------------------------------
# one function per C entry point
# ---------------------------------------------------------------------------

def _norm(name, x, weight, q, scale_inv, residual, h, rstd, eps, fmt, stream):
    f = _fp8(q, fmt, "q")
    rows, cols = _flat(x, "x")
    dt = _hp_dtype(x, "x")
    if q.numel() != x.numel() or weight.numel() != cols:
        raise ValueError(f"{name}: q must match x and weight must have x's last dimension")
    if residual is not None:
        _same(residual, (rows, cols), x.dtype, "residual")
    if h is not None:
        _same(h, (rows, cols), x.dtype, "h")
    scales = rows if name == "fp8q_rmsnorm_cast_per_channel" else rows * (cols // 128)
    st = getattr(lib, name)(_ptr(x, "x"), dt, 0 if residual is None else _ptr(residual, "residual"),
                            _ptr(weight, "weight"), _hp_dtype(weight, "weight"), rows, cols, eps, f, _ptr(q, "q"),
                            _f32(scale_inv, scales, "scale_inv"), 0 if h is None else _ptr(h, "h"),
                            0 if rstd is None else _f32(rstd, rows, "rstd"), _stream(x, stream))
    if st:
        _check(st, name)


def fp8q_rmsnorm_cast_group128(x, weight, q, scale_inv, residual=None, h=None, rstd=None, eps=1e-6, fmt="e4m3fn",
                               stream=None) -> None:
    _norm("fp8q_rmsnorm_cast_group128", x, weight, q, scale_inv, residual, h, rstd, eps, fmt, stream)


def fp8q_rmsnorm_cast_per_channel(x, weight, q, scale_inv, residual=None, h=None, rstd=None, eps=1e-6, fmt="e4m3fn",
                                  stream=None) -> None:
    _norm("fp8q_rmsnorm_cast_per_channel", x, weight, q, scale_inv, residual, h, rstd, eps, fmt, stream)


def fp8q_rmsnorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return lib.fp8q_rmsnorm_backward_workspace_bytes(rows, cols)


def fp8q_rmsnorm_backward(dy, h, weight, rstd, dx, dweight=None, dh=None, workspace=None, stream=None) -> None:
    rows, cols = _flat(h, "h")
    dt = _hp_dtype(h, "h")
    for t, n in ((dy, "dy"), (dx, "dx"), (dh, "dh")):
        _same(t, (rows, cols), h.dtype, n)
    if weight.numel() != cols:
        raise ValueError("fp8q_rmsnorm_backward: weight must have h's last dimension")
    if dweight is not None and (dweight.numel() != cols or dweight.dtype != weight.dtype):
        raise ValueError("fp8q_rmsnorm_backward: dweight must match weight")
    need = lib.fp8q_rmsnorm_backward_workspace_bytes(rows, cols) if dweight is not None else 0
    ws = _ws(workspace, need, h, "fp8q_rmsnorm_backward")
    _check(lib.fp8q_rmsnorm_backward(_ptr(dy, "dy"), _ptr(h, "h"), dt, _ptr(weight, "weight"),
                                     _hp_dtype(weight, "weight"), _f32(rstd, rows, "rstd"), _opt(dh, "dh"), rows, cols,
                                     _ptr(dx, "dx"), _opt(dweight, "dweight"),
                                     _opt(ws, "workspace"), _stream(h, stream)),
           "fp8q_rmsnorm_backward")


def fp8q_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.fp8q_linear_workspace_bytes(M, N, K)


def fp8q_linear(x, x_scale_inv, w, w_scale_inv, y, workspace=None, stream=None, x_fmt=None, w_fmt=None) -> None:
    xf, wf = _formats(x, x_fmt, w_fmt, w)
    xa, M, K = _x_codes(x, x_scale_inv, xf)
    wp, wsp, N = _w_codes(w, w_scale_inv, K, "w")
    _same(y, (M, N), y.dtype, "y")
    scratch = _ws(workspace, lib.fp8q_linear_workspace_bytes(M, N, K), x, "fp8q_linear")
    _check(lib.fp8q_linear(*xa, wp, wf, wsp, M, N, K, _ptr(y, "y"), _hp_dtype(y, "y"), _opt(scratch, "workspace"),
                           _stream(x, stream)), "fp8q_linear")


def fp8q_linear_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.fp8q_linear_backward_workspace_bytes(M, N, K)


def _grad_dtype(grads):
    d = {t.dtype for t in grads if t is not None}
    if len(d) > 1:
        raise TypeError("the weight gradients must have one dtype")
    return d.pop() if d else None


def fp8q_linear_backward(dy, x, x_scale_inv, w, w_scale_inv, dx=None, dw=None, workspace=None, stream=None,
                         x_fmt=None, w_fmt=None) -> None:
    xf, wf = _formats(x, x_fmt, w_fmt, w)
    xa, M, K = _x_codes(x, x_scale_inv, xf)
    wp, wsp, N = _w_codes(w, w_scale_inv, K, "w")
    dt = _hp_dtype(dy, "dy")
    _same(dy, (M, N), dy.dtype, "dy")
    _same(dx, (M, K), dy.dtype, "dx")
    if dw is not None:
        _same(dw, (N, K), dw.dtype, "dw")
    gdt = dt if dw is None else _hp_dtype(dw, "dw")
    need = lib.fp8q_linear_backward_workspace_bytes(M, N, K)
    scratch = _ws(workspace, need, x, "fp8q_linear_backward")
    _check(lib.fp8q_linear_backward(_ptr(dy, "dy"), dt, *xa, wp, wf, wsp, M, N, K, _opt(dx, "dx"), _opt(dw, "dw"), gdt,
                                    _opt(scratch, "workspace"), _stream(x, stream)),
           "fp8q_linear_backward")


def fp8q_gated_linear_workspace_bytes(M: int, F: int, K: int, cast: bool) -> int:
    return lib.fp8q_gated_linear_workspace_bytes(M, F, K, int(bool(cast)))


def _z_arg(z, M, F):
    if z is None:
        return 0, 0
    _same(z, (M, 2 * F), z.dtype, "z")
    return _ptr(z, "z"), _hp_dtype(z, "z")


def fp8q_gated_linear(x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, h, z=None, activation="silu",
                      workspace=None, stream=None, x_fmt=None, w_fmt=None) -> None:
    xf, wf = _formats(x, x_fmt, w_fmt, w_gate, w_up)
    xa, M, K = _x_codes(x, x_scale_inv, xf)
    pair, F = _pair(w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, K, wf)
    _same(h, (M, F), h.dtype, "h")
    need = lib.fp8q_gated_linear_workspace_bytes(M, F, K, 0)
    scratch = _ws(workspace, need, x, "fp8q_gated_linear")
    _check(lib.fp8q_gated_linear(*xa, *pair, M, F, K, _act(activation), _ptr(h, "h"), _hp_dtype(h, "h"),
                                 *_z_arg(z, M, F), _opt(scratch, "workspace"), _stream(x, stream)),
           "fp8q_gated_linear")


def fp8q_gated_linear_cast(x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, q, scale_inv, z=None,
                           activation="silu", fmt=None, workspace=None, stream=None, x_fmt=None, w_fmt=None) -> None:
    xf, wf = _formats(x, x_fmt, w_fmt, w_gate, w_up)
    xa, M, K = _x_codes(x, x_scale_inv, xf)
    pair, F = _pair(w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, K, wf)
    f = _fp8(q, fmt, "q")
    if q.numel() != M * F:
        raise ValueError("fp8q_gated_linear_cast: q must have M x F elements")
    if F % 128 == 0:
        _f32(scale_inv, M * (F // 128), "scale_inv")
    need = lib.fp8q_gated_linear_workspace_bytes(M, F, K, 1)
    scratch = _ws(workspace, need, x, "fp8q_gated_linear_cast")
    _check(lib.fp8q_gated_linear_cast(*xa, *pair, M, F, K, _act(activation), f, _ptr(q, "q"),
                                      _ptr(scale_inv, "scale_inv"), *_z_arg(z, M, F),
                                      _opt(scratch, "workspace"), _stream(x, stream)),
           "fp8q_gated_linear_cast")


def fp8q_gated_linear_backward_workspace_bytes(M: int, F: int, K: int) -> int:
    return lib.fp8q_gated_linear_backward_workspace_bytes(M, F, K)


def fp8q_gated_linear_backward(dp, z, x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, dx=None,
                               dw_gate=None, dw_up=None, activation="silu", workspace=None, stream=None,
                               x_fmt=None, w_fmt=None) -> None:
    xf, wf = _formats(x, x_fmt, w_fmt, w_gate, w_up)
    xa, M, K = _x_codes(x, x_scale_inv, xf)
    pair, F = _pair(w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, K, wf)
    dt = _hp_dtype(dp, "dp")
    _same(dp, (M, F), dp.dtype, "dp")
    _same(z, (M, 2 * F), dp.dtype, "z")
    _same(dx, (M, K), dp.dtype, "dx")
    for t, n in ((dw_gate, "dw_gate"), (dw_up, "dw_up")):
        if t is not None:
            _same(t, (F, K), t.dtype, n)
    g = _grad_dtype((dw_gate, dw_up))
    gdt = dt if g is None else _hp_dtype(dw_gate if dw_gate is not None else dw_up, "dw")
    need = lib.fp8q_gated_linear_backward_workspace_bytes(M, F, K)
    scratch = _ws(workspace, need, x, "fp8q_gated_linear_backward")
    _check(lib.fp8q_gated_linear_backward(_ptr(dp, "dp"), _ptr(z, "z"), dt, *xa, *pair, M, F, K, _act(activation),
                                          _opt(dx, "dx"), _opt(dw_gate, "dw_gate"), _opt(dw_up, "dw_up"), gdt,
                                          _opt(scratch, "workspace"), _stream(x, stream)),
           "fp8q_gated_linear_backward")


# ---------------------------------------------------------------------------
# helpers that allocate outputs and workspaces
# ---------------------------------------------------------------------------

def rmsnorm_cast(x, weight, residual=None, eps=1e-6, fp8_format="e4m3fn", per_channel_scale=False, out=None):
    """(q, scale_inv, h, rstd): h = x + residual, y = h / sqrt(mean(h^2) + eps)
    * weight cast to fp8 per 128 columns (scale_inv [rows, cols/128]) or per
    row (per_channel_scale=True, scale_inv [rows]).  h has x's dtype and is x
    itself without a residual; h and rstd are what rmsnorm_cast_backward
    reads.  `out`: those four tensors, caller-allocated (without a residual, x
    itself may stand for h; another tensor gets a copy of x)."""
    rows, cols = _flat(x, "x")
    if out is not None:
        q, s, h, rstd = out
    else:
        f, dev = _fmt(fp8_format), x.device
        q = torch.empty(x.shape, dtype=_FP8_DTYPE[f], device=dev)
        s = torch.empty((rows,) if per_channel_scale else (rows, cols // 128), dtype=torch.float32, device=dev)
        h = x if residual is None else torch.empty_like(x)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    name = "fp8q_rmsnorm_cast_per_channel" if per_channel_scale else "fp8q_rmsnorm_cast_group128"
    _norm(name, x, weight, q, s, residual, None if h is x else h, rstd, eps, fp8_format, None)
    return q, s, h, rstd


def rmsnorm_cast_backward(dy, h, weight, rstd, dh=None, out=None):
    """(dx, dweight) of rmsnorm_cast; dx is the gradient of x and of the
    residual.  dh: the gradient that reaches h along the residual path."""
    dx, dw = out if out is not None else (torch.empty_like(h), torch.empty_like(weight))
    fp8q_rmsnorm_backward(dy, h, weight, rstd, dx, dw, dh, _AUTO)
    return dx, dw


def linear_fp8(x, x_scale_inv, w, w_scale_inv, ret_type=torch.bfloat16, out=None, x_fmt=None, w_fmt=None):
    """y = X W^T for codes x [..., K] with scales per 128-group and w [N, K]
    with scales per 128x128 block."""
    y = out if out is not None else torch.empty((*x.shape[:-1], w.shape[0]), dtype=ret_type, device=x.device)
    fp8q_linear(x, x_scale_inv, w, w_scale_inv, y, _AUTO, x_fmt=x_fmt, w_fmt=w_fmt)
    return y


def linear_fp8_backward(dy, x, x_scale_inv, w, w_scale_inv, grad_type=None, out=None, x_fmt=None, w_fmt=None):
    """(dx, dw) of linear_fp8, dx in dy's dtype (bf16 or f16), dw in grad_type
    (dy's dtype by default, or float32)."""
    if out is not None:
        dx, dw = out
    else:
        dx = torch.empty(x.shape, dtype=dy.dtype, device=x.device)
        dw = torch.empty(w.shape, dtype=grad_type or dy.dtype, device=x.device)
    fp8q_linear_backward(dy, x, x_scale_inv, w, w_scale_inv, dx, dw, _AUTO, x_fmt=x_fmt, w_fmt=w_fmt)
    return dx, dw


def gated_linear_fp8(x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, activation="silu",
                     ret_type=torch.bfloat16, keep=None, out=None, x_fmt=None, w_fmt=None):
    """(h, z): h = act(X Wg^T) * (X Wu^T) in ret_type; z [..., 2F] holds both
    products in `keep`'s dtype for the backward pass, or is None."""
    F = w_gate.shape[0]
    if out is not None:
        h, z = out
    else:
        h = torch.empty((*x.shape[:-1], F), dtype=ret_type, device=x.device)
        z = None if keep is None else torch.empty((*x.shape[:-1], 2 * F), dtype=keep, device=x.device)
    fp8q_gated_linear(x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, h, z, activation, _AUTO,
                      x_fmt=x_fmt, w_fmt=w_fmt)
    return h, z


def gated_linear_fp8_cast(x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, activation="silu",
                          fp8_format="e4m3fn", keep=None, out=None, x_fmt=None, w_fmt=None):
    """(q, scale_inv, z): gated_linear_fp8's product cast to fp8 per 128-group
    (F % 128 == 0) without a 16-bit copy in between, and z as there."""
    F = w_gate.shape[0]
    if out is not None:
        q, s, z = out
    else:
        q = torch.empty((*x.shape[:-1], F), dtype=_FP8_DTYPE[_fmt(fp8_format)], device=x.device)
        s = torch.empty((_flat(x, "x")[0], F // 128), dtype=torch.float32, device=x.device)
        z = None if keep is None else torch.empty((*x.shape[:-1], 2 * F), dtype=keep, device=x.device)
    fp8q_gated_linear_cast(x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, q, s, z, activation,
                           fp8_format, _AUTO, x_fmt=x_fmt, w_fmt=w_fmt)
    return q, s, z


def gated_linear_fp8_backward(dp, z, x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv,
                              activation="silu", grad_type=None, out=None, x_fmt=None, w_fmt=None):
    """(dx, dw_gate, dw_up) from dp, the gradient of the product, and the
    forward's z; dtypes as in linear_fp8_backward."""
    if out is not None:
        dx, dg, du = out
    else:
        dx = torch.empty(x.shape, dtype=dp.dtype, device=x.device)
        dg = torch.empty(w_gate.shape, dtype=grad_type or dp.dtype, device=x.device)
        du = torch.empty(w_up.shape, dtype=grad_type or dp.dtype, device=x.device)
    fp8q_gated_linear_backward(dp, z, x, x_scale_inv, w_gate, w_gate_scale_inv, w_up, w_up_scale_inv, dx, dg, du,
                               activation, _AUTO, x_fmt=x_fmt, w_fmt=w_fmt)
    return dx, dg, du


FFN_NAMES = [n for n in dir() if n.startswith("fp8q_")] + [
    "SILU", "GELU", "GELU_TANH", "FFN_HEADER_PATH", "FFN_FUNCTIONS", "ffn_header_functions", "load_ffn",
    "rmsnorm_cast", "rmsnorm_cast_backward", "linear_fp8", "linear_fp8_backward", "gated_linear_fp8",
    "gated_linear_fp8_cast", "gated_linear_fp8_backward"]
