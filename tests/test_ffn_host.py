"""CPU tests of the feed-forward operators' C ABI (include/fp8q_ffn.h): the
library exports what the header declares, and every argument error is reported
before any HIP call (nothing is enqueued, so no GPU is needed; the fake device
addresses are never dereferenced).  The last test reruns this file on the ABI
layer built with AddressSanitizer and UBSan over host-only launcher stubs."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import dequantize_amax_reduce_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB_PATH = os.environ.get("FP8Q_FFN_ABI_LIB") or fq.LIB_PATH
L = fq.load_ffn(ctypes.CDLL(LIB_PATH))
STUBS = hasattr(L, "fp8q_ffn_stub_count")
P = lambda a: ctypes.c_void_p(a)
A = 0x7F0000000000                                      # 256-byte aligned fake base
E4, E5, F32, BF16, F16 = 0, 1, 0, 1, 2
at = lambda i: P(A + (i << 40))                         # far-apart fake buffers


def test_exports_match_header():
    declared = fq.ffn_header_functions()
    assert set(declared) == set(fq.FFN_FUNCTIONS)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r" T (fp8q_\w+)$", out, re.M))
    assert set(declared) <= exported


def _norm(fn, **k):
    a = dict(x=at(1), xdt=BF16, res=at(2), w=at(3), wdt=BF16, rows=4, cols=256, eps=1e-6, fmt=E4, q=at(4), s=at(5),
             h=at(6), rstd=at(7), st=None)
    a.update(k)
    return fn(*a.values())


@pytest.mark.parametrize("name", ["fp8q_rmsnorm_cast_group128", "fp8q_rmsnorm_cast_per_channel"])
def test_norm_errors(name):
    f = getattr(L, name)
    group = name.endswith("128")
    assert _norm(f, xdt=3) == fq.EDTYPE
    assert _norm(f, fmt=2) == fq.EDTYPE
    assert _norm(f, wdt=F16) == fq.EDTYPE                  # neither x's type nor f32
    assert _norm(f, xdt=F32, wdt=BF16) == fq.EDTYPE
    assert _norm(f, rows=-1) == fq.EINVAL
    assert _norm(f, cols=-128) == fq.EINVAL
    assert _norm(f, rows=2 ** 31) == fq.EINVAL
    assert _norm(f, cols=2 ** 30 + 128) == fq.EINVAL
    for k in ("x", "w", "q", "s"):
        assert _norm(f, **{k: None}) == fq.EINVAL, k
    for k in ("x", "res", "w", "h"):
        assert _norm(f, **{k: P(A + 1)}) == fq.EALIGN, k
    for k in ("s", "rstd"):
        assert _norm(f, **{k: P(A + 2)}) == fq.EALIGN, k
    assert _norm(f, q=P(A + (1 << 40) + 8)) == fq.EINVAL   # q in x
    assert _norm(f, h=P(A + (1 << 40) + 2)) == fq.EINVAL   # h meets x but is not x
    assert _norm(f, q=at(6)) == fq.EINVAL                  # q = h
    assert _norm(f, rstd=at(5)) == fq.EINVAL
    if group:
        assert _norm(f, cols=100) == fq.ESHAPE
    assert _norm(f, rows=0, x=None, w=None, q=None, s=None, h=None, rstd=None) == fq.OK


def _norm_bwd(**k):
    a = dict(dy=at(1), h=at(2), dt=BF16, w=at(3), wdt=BF16, rstd=at(4), dh=at(5), rows=4, cols=250, dx=at(6), dw=at(7),
             ws=at(8), st=None)
    a.update(k)
    return L.fp8q_rmsnorm_backward(*a.values())


def test_norm_backward_errors():
    assert _norm_bwd(dt=7) == fq.EDTYPE
    assert _norm_bwd(wdt=F16) == fq.EDTYPE
    assert _norm_bwd(rows=-1) == fq.EINVAL
    for k in ("dy", "h", "w", "rstd", "dx", "ws"):
        assert _norm_bwd(**{k: None}) == fq.EINVAL, k
    for k in ("dy", "h", "w", "dh", "dx", "dw"):
        assert _norm_bwd(**{k: P(A + 1)}) == fq.EALIGN, k
    assert _norm_bwd(rstd=P(A + 2)) == fq.EALIGN
    assert _norm_bwd(ws=P(A + 4)) == fq.EALIGN
    assert _norm_bwd(dx=at(2)) == fq.EINVAL                # dx = h
    assert _norm_bwd(dx=P(A + (1 << 40) + 4)) == fq.EINVAL
    assert _norm_bwd(dw=at(6)) == fq.EINVAL
    assert _norm_bwd(ws=at(1)) == fq.EINVAL
    assert _norm_bwd(cols=0) == fq.OK
    assert _norm_bwd(rows=0, dw=None, dy=None, h=None, w=None, rstd=None, dx=None, ws=None) == fq.OK
    assert L.fp8q_rmsnorm_backward_workspace_bytes(4, 250) >= 4 * 250 * 4
    assert L.fp8q_rmsnorm_backward_workspace_bytes(-4, 250) == 0


def _linear(**k):
    a = dict(x=at(1), xf=E4, xs=at(2), w=at(3), wf=E4, wsc=at(4), M=300, N=200, K=256, y=at(5), ydt=BF16, ws=at(6), st=None)
    a.update(k)
    return L.fp8q_linear(*a.values())


def test_linear_errors():
    assert _linear(xf=2) == fq.EDTYPE
    assert _linear(wf=-1) == fq.EDTYPE
    assert _linear(ydt=3) == fq.EDTYPE
    assert _linear(K=200) == fq.ESHAPE
    for k in ("M", "N", "K"):
        assert _linear(**{k: -128}) == fq.EINVAL, k
    assert _linear(M=2 ** 31 + 1) == fq.EINVAL
    assert _linear(N=2 ** 21 + 1) == fq.EINVAL
    assert _linear(K=2 ** 21 + 128) == fq.EINVAL
    assert _linear(M=2 ** 31, N=2 ** 21) == fq.EINVAL      # more tiles than a grid holds
    for k in ("x", "xs", "w", "wsc", "y"):
        assert _linear(**{k: None}) == fq.EINVAL, k
    for k in ("x", "w"):
        assert _linear(**{k: P(A + 8)}) == fq.EALIGN, k    # codes need 16 bytes
    for k in ("xs", "wsc"):
        assert _linear(**{k: P(A + 2)}) == fq.EALIGN, k
    assert _linear(y=P(A + 1)) == fq.EALIGN
    assert _linear(y=at(1)) == fq.EINVAL
    assert _linear(y=P(A + (4 << 40) + 2)) == fq.EINVAL    # y meets w's scales
    assert _linear(M=0, x=None, y=None) == fq.OK
    assert _linear(N=0, w=None, y=None) == fq.OK
    # a split contraction needs its workspace
    need = L.fp8q_linear_workspace_bytes(100, 128, 1 << 15)
    assert need > 0
    assert _linear(M=100, N=128, K=1 << 15, ydt=F32, ws=None) == fq.EINVAL
    assert _linear(M=100, N=128, K=1 << 15, ydt=F32, ws=P(A + 16)) == fq.EALIGN
    assert _linear(M=100, N=128, K=1 << 15, ydt=F32, ws=at(1)) == fq.EINVAL
    assert L.fp8q_linear_workspace_bytes(-1, 128, 128) == 0 and L.fp8q_linear_workspace_bytes(1, 128, 100) == 0


def _gated(cast=False, **k):
    a = dict(x=at(1), xf=E4, xs=at(2), g=at(3), gs=at(4), u=at(5), us=at(6), wf=E4, M=300, F=256, K=256, act=0)
    a.update(dict(fmt=E4, q=at(7), s=at(8)) if cast else dict(h=at(7), hdt=BF16))
    a.update(z=at(9), zdt=BF16, ws=at(10), st=None)
    a.update(k)
    return (L.fp8q_gated_linear_cast if cast else L.fp8q_gated_linear)(*a.values())


@pytest.mark.parametrize("cast", [False, True])
def test_gated_errors(cast):
    f = lambda **k: _gated(cast, **k)
    assert f(act=3) == fq.EDTYPE
    assert f(act=-1) == fq.EDTYPE
    assert f(xf=5) == fq.EDTYPE
    assert f(zdt=4) == fq.EDTYPE
    assert f(K=130) == fq.ESHAPE
    assert f(F=-128) == fq.EINVAL
    for k in ("x", "xs", "g", "gs", "u", "us", "q" if cast else "h"):
        assert f(**{k: None}) == fq.EINVAL, k
    for k in ("x", "g", "u"):
        assert f(**{k: P(A + 8)}) == fq.EALIGN, k
    assert f(z=P(A + 1)) == fq.EALIGN
    assert f(z=at(7)) == fq.EINVAL                         # z = the output
    assert f(**{"q" if cast else "h": at(3)}) == fq.EINVAL
    if cast:
        assert f(fmt=2) == fq.EDTYPE
        assert f(F=200) == fq.ESHAPE
        assert f(s=None) == fq.EINVAL
        assert f(s=P(A + 2)) == fq.EALIGN
        assert L.fp8q_gated_linear_workspace_bytes(8, 256, 256, 1) >= 8 * 256 * 4
        assert f(M=8, ws=None) == fq.EINVAL
    else:
        assert f(hdt=3) == fq.EDTYPE
    assert f(M=0, x=None, ws=None) == fq.OK
    assert f(F=0, g=None, u=None, ws=None) == fq.OK


def _lin_bwd(**k):
    a = dict(dy=at(1), dt=BF16, x=at(2), xf=E4, xs=at(3), w=at(4), wf=E4, wsc=at(5), M=300, N=200, K=256, dx=at(6),
             dw=at(7), gdt=BF16, ws=at(8), st=None)
    a.update(k)
    return L.fp8q_linear_backward(*a.values())


def _gated_bwd(**k):
    a = dict(dp=at(1), z=at(11), dt=BF16, x=at(2), xf=E4, xs=at(3), g=at(4), gs=at(5), u=at(9), us=at(10), wf=E4, M=300,
             F=200, K=256, act=0, dx=at(6), dwg=at(7), dwu=at(12), gdt=BF16, ws=at(8), st=None)
    a.update(k)
    return L.fp8q_gated_linear_backward(*a.values())


def test_backward_errors():
    for f, dws in ((_lin_bwd, ("dw",)), (_gated_bwd, ("dwg", "dwu"))):
        n = "N" if f is _lin_bwd else "F"
        dy = "dy" if f is _lin_bwd else "dp"
        assert f(dt=F32, gdt=F32) == fq.EDTYPE             # gradients are 16-bit
        assert f(gdt=F16) == fq.EDTYPE
        assert f(xf=2) == fq.EDTYPE
        assert f(K=100) == fq.ESHAPE
        assert f(M=-1) == fq.EINVAL
        assert f(M=4194241) == fq.EINVAL
        assert f(**{n: 2 ** 21 + 1}) == fq.EINVAL
        assert f(**{n: 2 ** 21, "K": 2 ** 21}) == fq.EINVAL
        for k in (dy, "x", "xs", "ws"):
            assert f(**{k: None}) == fq.EINVAL, k
        assert f(x=P(A + 8)) == fq.EALIGN
        assert f(dx=P(A + 1)) == fq.EALIGN
        assert f(**{dws[0]: P(A + 1)}) == fq.EALIGN
        assert f(ws=P(A + 128)) == fq.EALIGN
        assert f(dx=at(7)) == fq.EINVAL                    # dx = a weight gradient
        assert f(dx=at(1)) == fq.EINVAL
        assert f(**{"dx": None, **{k: None for k in dws}}) == fq.OK
        assert f(K=0) == fq.OK
    assert _gated_bwd(act=9) == fq.EDTYPE
    assert _gated_bwd(z=None) == fq.EINVAL
    assert _gated_bwd(dwu=None) == fq.EINVAL               # both weight gradients or none
    assert L.fp8q_linear_backward_workspace_bytes(0, 200, 256) == 0
    assert L.fp8q_gated_linear_backward_workspace_bytes(300, 200, 256) > \
        L.fp8q_linear_backward_workspace_bytes(300, 200, 256) > 0


def test_python_binding_refuses():
    E = torch.float8_e4m3fn
    x, xs = torch.zeros(4, 256).to(E), torch.zeros(4, 2)
    w, ws = torch.zeros(200, 256).to(E), torch.zeros(2, 2)
    with pytest.raises(ValueError):                        # host tensors
        fq.linear_fp8(x, xs, w, ws)
    with pytest.raises(ValueError):                        # scales of another shape
        fq.linear_fp8(x, torch.zeros(4, 3), w, ws)
    with pytest.raises(ValueError):
        fq.linear_fp8(x, xs, torch.zeros(200, 128).to(E), ws)
    with pytest.raises(TypeError):                         # not codes
        fq.linear_fp8(x.float(), xs, w, ws)
    with pytest.raises(TypeError):
        fq.rmsnorm_cast(torch.zeros(4, 128, dtype=torch.float64), torch.zeros(128))
    with pytest.raises(ValueError):
        fq.rmsnorm_cast(torch.zeros(4, 128), torch.zeros(64))
    with pytest.raises(TypeError):
        fq.rmsnorm_cast(torch.zeros(4, 128), torch.zeros(128), fp8_format="e3m4")
    for bad in ("relu", None, 7):
        with pytest.raises((TypeError, ValueError)):
            fq.gated_linear_fp8(x, xs, w, ws, w, ws, bad)


@pytest.mark.skipif(not STUBS, reason="needs the launcher-stub build of the ABI layer (test_ffn_abi_under_asan_ubsan)")
def test_fuzz_validation():
    """Random calls with sizes at and beyond every limit: a documented status
    each time, no undefined behaviour, no broken launcher precondition."""
    import numpy as np
    rng = np.random.Generator(np.random.PCG64(78))
    sizes = [0, 1, 2, 63, 64, 65, 127, 128, 256, 4096, 2 ** 21, 2 ** 21 + 128, 4194240, 2 ** 30, 2 ** 31, 2 ** 40,
             2 ** 62, 2 ** 63 - 1, -1, -128, -(2 ** 63)]
    ptrs = [None, A, A + 1, A + 2, A + 4, A + 16, A + 4096] + [A + (i << 40) for i in range(1, 14)] + [2 ** 64 - 4096]
    enums = [0, 1, 2, 3, -1, 2 ** 31 - 1, -(2 ** 31)]
    codes = {fq.OK, fq.EINVAL, fq.EDTYPE, fq.ESHAPE, fq.EALIGN, fq.EHIP}
    reached = 0
    for name in fq.FFN_FUNCTIONS:
        fn = getattr(L, name)
        for _ in range(4000):
            args = []
            for t in fn.argtypes:
                if t is ctypes.c_void_p:
                    p = ptrs[int(rng.integers(0, len(ptrs)))] if rng.random() < 0.3 else A + (len(args) + 20 << 40)
                    args.append(None if p is None else P(p))
                elif t is ctypes.c_int64:
                    args.append(sizes[int(rng.integers(0, len(sizes)))] if rng.random() < 0.5
                                else 128 * int(rng.integers(0, 40)))
                elif t is ctypes.c_float:
                    args.append(1e-6)
                else:
                    args.append(enums[int(rng.integers(0, len(enums)))] if rng.random() < 0.1 else int(rng.integers(0, 2)))
            if name.endswith("_bytes"):
                assert fn(*args) >= 0
            else:
                args[-1] = None
                L.fp8q_ffn_stub_reset()
                st = fn(*args)
                assert st in codes, (name, args)
                reached += L.fp8q_ffn_stub_count()
                assert st == fq.OK or L.fp8q_ffn_stub_count() == 0, (name, args)
    assert reached > 100


def test_ffn_abi_under_asan_ubsan(tmp_path):
    if STUBS:
        pytest.skip("already the sanitizer build")
    from test_sanitizers import SAN, _run
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    lib = str(tmp_path / "libfp8q_ffn_abi_san.so")
    csrc = os.path.join(ROOT, "dequantize_amax_reduce_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-Wall", *SAN, "-D__HIP_PLATFORM_AMD__", "-I",
                    "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "fp8q_ffn_abi.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "fp8q_ffn_launch_stubs.cpp"), "-o", lib], check=True)
    out = _run("tests/test_ffn_host.py", {"FP8Q_FFN_ABI_LIB": lib})
    assert " passed" in out
