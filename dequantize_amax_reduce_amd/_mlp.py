"""Binding of include/fp8q_mlp.h: layer norm and projections with a bias, an
activation and a residual in their epilogue, on fp8 operands.

Re-exported by the package; laid out as _ffn.py is.

    q, s, h, mean, rstd = layernorm_cast(x, weight, bias, residual)     # norm -> fp8 per 128-group
    p, ps, z = linear_act_fp8_cast(q, s, w1, w1s, b1, "gelu", keep=torch.bfloat16)
    y, _ = linear_act_fp8(p, ps, w2, w2s, b2, residual=h)               # the new residual stream
    dp, dw2, db2 = linear_act_fp8_backward(dy, None, p, ps, w2, w2s)
    dn, dw1, db1 = linear_act_fp8_backward(dp, z, q, s, w1, w1s, "gelu")
    dx, dweight, dbias = layernorm_backward(dn, h, weight, mean, rstd, dy)
"""
from __future__ import annotations

import ctypes
import os
import re
from functools import lru_cache

import torch

from . import _ffn
from ._ffn import _AUTO, _CODES, _flat, _hp_dtype, _raw_stream, _ws

MLP_HEADER_PATH = os.path.join(os.path.dirname(_ffn.FFN_HEADER_PATH), "fp8q_mlp.h")

IDENTITY, RELU = 3, 4
_ACT = {**_ffn._ACT, None: IDENTITY, "identity": IDENTITY, "relu": RELU, IDENTITY: IDENTITY, RELU: RELU}

_P, _I64, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
MLP_SIGNATURES = {
    "fp8q_layernorm": (_I, [_P, _I, _P, _P, _P, _I, _I64, _I64, _F, _P, _P, _P, _P, _P]),
    "fp8q_layernorm_cast_group128": (_I, [_P, _I, _P, _P, _P, _I, _I64, _I64, _F, _I, _P, _P, _P, _P, _P, _P]),
    "fp8q_layernorm_cast_per_channel": (_I, [_P, _I, _P, _P, _P, _I, _I64, _I64, _F, _I, _P, _P, _P, _P, _P, _P]),
    "fp8q_layernorm_backward_workspace_bytes": (_SZ, [_I64, _I64]),
    "fp8q_layernorm_backward": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    "fp8q_linear_act_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "fp8q_linear_act": (_I, _CODES + _CODES + [_I64, _I64, _I64, _P, _I, _I, _P, _P, _I, _P, _I, _P, _P]),
    "fp8q_linear_act_cast": (_I, _CODES + _CODES + [_I64, _I64, _I64, _P, _I, _I, _I, _P, _P, _P, _I, _P, _P]),
    "fp8q_linear_act_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8q_linear_act_backward": (_I, [_P, _P, _I] + _CODES + _CODES + [_I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _P]),
}
MLP_FUNCTIONS = tuple(MLP_SIGNATURES)


def load_mlp(L):
    """Set the signatures of these entry points on a library handle."""
    for name, (res, args) in MLP_SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def mlp_header_functions() -> list:
    """Names of the functions include/fp8q_mlp.h declares."""
    with open(MLP_HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^(?:fp8q_status_t|size_t)\s+(fp8q_\w+)\s*\(", text, re.M)))


# set by the package once its own marshalling helpers exist
lib = _check = _dev = _fmt = _fp8 = _FP8_DTYPE = _FMT = None


def _bind(package_lib, helpers):
    global lib
    lib = load_mlp(package_lib)
    globals().update(helpers)


# As in _ffn.py, a call on one token is bound by its host time, so each tensor is
# asked what it is in one go, and again only to say what is wrong.  `d` is the
# device of the call's first tensor (-1: the host), which every tensor has to be on.

_F32 = torch.float32


def _ten(t, n, dtype, name, d) -> int:
    """the address of n contiguous elements of dtype on device d (0 without a tensor)"""
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.numel() == n and t.get_device() == d and t.is_contiguous() and d >= 0:
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and (t.dtype != dtype or t.numel() != n):
        raise ValueError(f"{name} must be {dtype} with {n} elements")
    return _at(t, name, d)


def _format(t, fmt, name) -> int:
    """the format of fp8 codes; fmt names that of uint8 ones"""
    f = _FMT.get(t.dtype)
    return f if f is not None and (fmt is None or _FMT.get(fmt) == f) else _fp8(t, fmt, name)


# sizes alone decide a workspace's bytes
@lru_cache(maxsize=4096)
def _norm_ws_bytes(rows, cols):
    return lib.fp8q_layernorm_backward_workspace_bytes(rows, cols)


@lru_cache(maxsize=4096)
def _act_ws_bytes(M, N, K, cast):
    return lib.fp8q_linear_act_workspace_bytes(M, N, K, cast)


@lru_cache(maxsize=4096)
def _bwd_ws_bytes(M, N, K):
    return lib.fp8q_linear_act_backward_workspace_bytes(M, N, K)


def _at(t, name, d) -> int:
    """the address of a contiguous tensor on device d (0 of an empty one)"""
    try:
        if t.get_device() == d and d >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = _dev(t, name)                                   # raises, or 0 for an empty tensor
    if p and t.get_device() != d:
        raise ValueError(f"{name} is on another device than the other tensors")
    return p


def _opt(t, name, d) -> int:
    return 0 if t is None else _at(t, name, d)


def _stream(stream, d):
    if stream is None:
        return _raw_stream(d) if d >= 0 else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_current = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _call(name, d, *args):
    """The C call with device d as the thread's current one, which a launch needs."""
    if d >= 0 and d != _current():
        with torch.cuda.device(d):
            st = getattr(lib, name)(*args)
    else:
        st = getattr(lib, name)(*args)
    if st:
        _check(st, name)


# ---------------------------------------------------------------------------
# one function per C entry point
# ---------------------------------------------------------------------------

def _norm(name, x, weight, bias, y, scale_inv, residual, h, mean, rstd, eps, fmt, stream):
    rows, cols = _flat(x, "x")
    n, T, W, d = rows * cols, x.dtype, weight.dtype, x.get_device()
    dt, wdt = _hp_dtype(x, "x"), _hp_dtype(weight, "weight")
    w, b = _ten(weight, cols, W, "weight", d), _ten(bias, cols, W, "bias", d)
    r, ho = _ten(residual, n, T, "residual", d), _ten(h, n, T, "h", d)
    if name == "fp8q_layernorm":
        out = (_ten(y, n, T, "y", d),)
    else:
        scales = rows if name == "fp8q_layernorm_cast_per_channel" else rows * (cols // 128)
        out = (_format(y, fmt, "q"), _ten(y, n, y.dtype, "q", d), _ten(scale_inv, scales, _F32, "scale_inv", d))
    _call(name, d, _at(x, "x", d), dt, r, w, b, wdt, rows, cols, eps, *out, ho, _ten(mean, rows, _F32, "mean", d),
          _ten(rstd, rows, _F32, "rstd", d), _stream(stream, d))


def fp8q_layernorm(x, weight, bias, y, residual=None, h=None, mean=None, rstd=None, eps=1e-5, stream=None) -> None:
    _norm("fp8q_layernorm", x, weight, bias, y, None, residual, h, mean, rstd, eps, None, stream)


def fp8q_layernorm_cast_group128(x, weight, bias, q, scale_inv, residual=None, h=None, mean=None, rstd=None, eps=1e-5,
                                 fmt=None, stream=None) -> None:
    _norm("fp8q_layernorm_cast_group128", x, weight, bias, q, scale_inv, residual, h, mean, rstd, eps, fmt, stream)


def fp8q_layernorm_cast_per_channel(x, weight, bias, q, scale_inv, residual=None, h=None, mean=None, rstd=None,
                                    eps=1e-5, fmt=None, stream=None) -> None:
    _norm("fp8q_layernorm_cast_per_channel", x, weight, bias, q, scale_inv, residual, h, mean, rstd, eps, fmt, stream)


def fp8q_layernorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return lib.fp8q_layernorm_backward_workspace_bytes(rows, cols)


def fp8q_layernorm_backward(dy, h, weight, mean, rstd, dx, dweight=None, dbias=None, dh=None, workspace=None,
                            stream=None) -> None:
    name = "fp8q_layernorm_backward"
    rows, cols = _flat(h, "h")
    n, T, W, d = rows * cols, h.dtype, weight.dtype, h.get_device()
    dt, wdt = _hp_dtype(h, "h"), _hp_dtype(weight, "weight")
    need = _norm_ws_bytes(rows, cols) if dweight is not None or dbias is not None else 0
    ws = _ws(workspace, need, h, name)
    _call(name, d, _ten(dy, n, T, "dy", d), _at(h, "h", d), dt, _ten(weight, cols, W, "weight", d), wdt,
          _ten(mean, rows, _F32, "mean", d), _ten(rstd, rows, _F32, "rstd", d), _ten(dh, n, T, "dh", d), rows, cols,
          _ten(dx, n, T, "dx", d), _ten(dweight, cols, W, "dweight", d), _ten(dbias, cols, W, "dbias", d),
          _opt(ws, "workspace", d), _stream(stream, d))


def _activation(name) -> int:
    if name not in _ACT:
        raise TypeError(f"unknown activation {name!r} (use None, 'relu', 'silu', 'gelu' or 'gelu_tanh')")
    return _ACT[name]


def _typed(t, n, name, d):
    """pointer and type of an optional tensor of n elements of any element type"""
    return (0, 0) if t is None else (_ten(t, n, t.dtype, name, d), _hp_dtype(t, name))


def _codes(x, xs, w, ws, x_fmt, w_fmt):
    """the operands' arguments with the sizes, and M, N, K and the device"""
    xf, wf = _format(x, x_fmt, "x"), _format(w, w_fmt, "the weight")
    M, K = _flat(x, "x")
    d = x.get_device()
    if w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"w must be 2-D with {K} columns")
    N, KB = w.shape[0], K // 128
    return (_at(x, "x", d), xf, _ten(xs, M * KB, _F32, "x_scale_inv", d), _at(w, "w", d), wf,
            _ten(ws, ((N + 127) // 128) * KB, _F32, "the weight's scale_inv", d), M, N, K), M, N, K, d


def fp8q_linear_act_workspace_bytes(M: int, N: int, K: int, cast: bool) -> int:
    return lib.fp8q_linear_act_workspace_bytes(M, N, K, int(bool(cast)))


def fp8q_linear_act(x, x_scale_inv, w, w_scale_inv, bias, y, residual=None, z=None, activation=None, workspace=None,
                    stream=None, x_fmt=None, w_fmt=None) -> None:
    name = "fp8q_linear_act"
    act = _activation(activation)
    args, M, N, K, d = _codes(x, x_scale_inv, w, w_scale_inv, x_fmt, w_fmt)
    n = M * N
    scratch = _ws(workspace, _act_ws_bytes(M, N, K, 0), x, name)
    _call(name, d, *args, *_typed(bias, N, "bias", d), act, _ten(residual, n, y.dtype, "residual", d),
          *_typed(y, n, "y", d), *_typed(z, n, "z", d), _opt(scratch, "workspace", d), _stream(stream, d))


def fp8q_linear_act_cast(x, x_scale_inv, w, w_scale_inv, bias, q, scale_inv, z=None, activation=None, fmt=None,
                         workspace=None, stream=None, x_fmt=None, w_fmt=None) -> None:
    name = "fp8q_linear_act_cast"
    act = _activation(activation)
    args, M, N, K, d = _codes(x, x_scale_inv, w, w_scale_inv, x_fmt, w_fmt)
    n = M * N
    f, codes = _format(q, fmt, "q"), _ten(q, n, q.dtype, "q", d)
    scales = _ten(scale_inv, n // 128, _F32, "scale_inv", d) if N % 128 == 0 else 0     # else the call is refused
    scratch = _ws(workspace, _act_ws_bytes(M, N, K, 1), x, name)
    _call(name, d, *args, *_typed(bias, N, "bias", d), act, f, codes, scales, *_typed(z, n, "z", d),
          _opt(scratch, "workspace", d), _stream(stream, d))


def fp8q_linear_act_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib.fp8q_linear_act_backward_workspace_bytes(M, N, K)


def fp8q_linear_act_backward(dy, z, x, x_scale_inv, w, w_scale_inv, dx=None, dw=None, dbias=None, activation=None,
                             workspace=None, stream=None, x_fmt=None, w_fmt=None) -> None:
    name = "fp8q_linear_act_backward"
    act, g = _activation(activation), _ffn._grad_dtype((dw, dbias))
    args, M, N, K, d = _codes(x, x_scale_inv, w, w_scale_inv, x_fmt, w_fmt)
    T, dt, n = dy.dtype, _hp_dtype(dy, "dy"), M * N
    if act == IDENTITY:
        z = None
    elif z is None:
        raise ValueError(f"{name}: an activation's gradient needs z")
    GT, gdt = (T, dt) if g is None else (g, _hp_dtype(dw if dw is not None else dbias, "dw"))
    scratch = _ws(workspace, _bwd_ws_bytes(M, N, K), x, name)
    _call(name, d, _ten(dy, n, T, "dy", d), _ten(z, n, T, "z", d), dt, *args, act, _ten(dx, M * K, T, "dx", d),
          _ten(dw, N * K, GT, "dw", d), _ten(dbias, N, GT, "dbias", d), gdt, _opt(scratch, "workspace", d),
          _stream(stream, d))


# ---------------------------------------------------------------------------
# helpers that allocate outputs and workspaces
# ---------------------------------------------------------------------------

def _stats(x, rows, residual):
    mean = torch.empty(rows, dtype=_F32, device=x.device)
    return x if residual is None else torch.empty_like(x, memory_format=torch.contiguous_format), mean, torch.empty_like(mean)


def layernorm(x, weight, bias=None, residual=None, eps=1e-5, out=None):
    """(y, h, mean, rstd): h = x + residual, y = (h - mean) / sqrt(var + eps) *
    weight + bias over the last dimension, in x's dtype.  h is x itself without
    a residual; h, mean and rstd are what layernorm_backward reads.  `out`:
    those four tensors, caller-allocated.  h may be x there: without a residual
    it is left as it is, with one h is written over x (another tensor gets a copy
    of x without a residual)."""
    if out is not None:
        y, h, mean, rstd = out
    else:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        h, mean, rstd = _stats(x, _flat(x, "x")[0], residual)
    _norm("fp8q_layernorm", x, weight, bias, y, None, residual, None if h is x and residual is None else h, mean, rstd,
          eps, None, None)
    return y, h, mean, rstd


def layernorm_cast(x, weight, bias=None, residual=None, eps=1e-5, fp8_format="e4m3fn", per_channel_scale=False,
                   out=None):
    """(q, scale_inv, h, mean, rstd): layernorm's y cast to fp8 per 128 columns
    (scale_inv [rows, cols/128]) or per row (per_channel_scale=True, scale_inv
    [rows]) without a copy in x's dtype in between; h and `out` as there."""
    rows, cols = _flat(x, "x")
    if out is not None:
        q, s, h, mean, rstd = out
    else:
        q = torch.empty_like(x, dtype=_FP8_DTYPE[_fmt(fp8_format)], memory_format=torch.contiguous_format)
        s = torch.empty((rows,) if per_channel_scale else (rows, cols // 128), dtype=torch.float32, device=x.device)
        h, mean, rstd = _stats(x, rows, residual)
    name = "fp8q_layernorm_cast_per_channel" if per_channel_scale else "fp8q_layernorm_cast_group128"
    _norm(name, x, weight, bias, q, s, residual, None if h is x and residual is None else h, mean, rstd, eps, fp8_format,
          None)
    return q, s, h, mean, rstd


def layernorm_backward(dy, h, weight, mean, rstd, dh=None, with_bias=True, out=None):
    """(dx, dweight, dbias) of layernorm and layernorm_cast; dx is the gradient
    of x and of the residual, dbias None with with_bias=False.  dh: the gradient
    that reaches h along the residual path."""
    if out is not None:
        dx, dw, db = out
    else:
        dx, dw = torch.empty_like(h), torch.empty_like(weight)
        db = torch.empty_like(weight) if with_bias else None
    fp8q_layernorm_backward(dy, h, weight, mean, rstd, dx, dw, db if with_bias else None, dh, _AUTO)
    return dx, dw, db if with_bias else None


def linear_act_fp8(x, x_scale_inv, w, w_scale_inv, bias=None, activation=None, residual=None, ret_type=torch.bfloat16,
                   keep=None, out=None, x_fmt=None, w_fmt=None):
    """(y, z): z = X W^T + bias for codes x [..., K] with scales per 128-group
    and w [N, K] with scales per 128x128 block; y = act(z) + residual in
    ret_type (the residual's dtype where there is one).  activation: None,
    'relu', 'silu', 'gelu' or 'gelu_tanh'.  z is returned in `keep`'s dtype for
    the backward pass, or is None.  `out`: y and z (or None), caller-allocated;
    y may be the residual itself."""
    if out is not None:
        y, z = out
    else:
        shape = (*x.shape[:-1], w.shape[0])
        y = torch.empty(shape, dtype=ret_type if residual is None else residual.dtype, device=x.device)
        z = None if keep is None else torch.empty(shape, dtype=keep, device=x.device)
    fp8q_linear_act(x, x_scale_inv, w, w_scale_inv, bias, y, residual, z, activation, _AUTO, x_fmt=x_fmt, w_fmt=w_fmt)
    return y, z


def linear_act_fp8_cast(x, x_scale_inv, w, w_scale_inv, bias=None, activation=None, fp8_format="e4m3fn", keep=None,
                        out=None, x_fmt=None, w_fmt=None):
    """(q, scale_inv, z): linear_act_fp8's act(z) cast to fp8 per 128-group (N %
    128 == 0) without a 16-bit copy in between, and z as there."""
    N = w.shape[0]
    if out is not None:
        q, s, z = out
    else:
        shape = (*x.shape[:-1], N)
        q = torch.empty(shape, dtype=_FP8_DTYPE[_fmt(fp8_format)], device=x.device)
        s = torch.empty((_flat(x, "x")[0], N // 128), dtype=torch.float32, device=x.device)
        z = None if keep is None else torch.empty(shape, dtype=keep, device=x.device)
    fp8q_linear_act_cast(x, x_scale_inv, w, w_scale_inv, bias, q, s, z, activation, fp8_format, _AUTO, x_fmt=x_fmt,
                         w_fmt=w_fmt)
    return q, s, z


def linear_act_fp8_backward(dy, z, x, x_scale_inv, w, w_scale_inv, activation=None, grad_type=None, with_bias=True,
                            out=None, x_fmt=None, w_fmt=None):
    """(dx, dw, dbias) of linear_act_fp8 and of linear_act_fp8_cast from dy and
    the forward's z (None without an activation), dx in dy's dtype (bf16 or
    f16), dw and dbias in grad_type (dy's dtype by default, or float32); dbias is
    None with with_bias=False.  The residual's gradient is dy itself.  `out`:
    those three, caller-allocated, or None for one that is not computed (dw of
    frozen weights)."""
    if out is not None:
        dx, dw, db = out
    else:
        dx = torch.empty(x.shape, dtype=dy.dtype, device=x.device)
        dw = torch.empty(w.shape, dtype=grad_type or dy.dtype, device=x.device)
        db = torch.empty(w.shape[0], dtype=dw.dtype, device=x.device) if with_bias else None
    if not with_bias:
        db = None
    fp8q_linear_act_backward(dy, z, x, x_scale_inv, w, w_scale_inv, dx, dw, db, activation, _AUTO, x_fmt=x_fmt, w_fmt=w_fmt)
    return dx, dw, db


MLP_NAMES = [n for n in dir() if n.startswith("fp8q_")] + [
    "IDENTITY", "RELU", "MLP_HEADER_PATH", "MLP_FUNCTIONS", "mlp_header_functions", "load_mlp",
    "layernorm", "layernorm_cast", "layernorm_backward", "linear_act_fp8", "linear_act_fp8_cast",
    "linear_act_fp8_backward"]
