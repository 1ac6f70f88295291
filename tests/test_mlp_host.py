"""CPU tests of the C ABI of layer norm and biased projections
(include/fp8q_mlp.h): the library exports what the header declares, and every
argument error is reported before any HIP call (nothing is enqueued, so no GPU
is needed; the fake device addresses are never dereferenced).  The last test
reruns this file on the ABI layer built with AddressSanitizer and UBSan over
host-only launcher stubs."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import dequantize_amax_reduce_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB_PATH = os.environ.get("FP8Q_MLP_ABI_LIB") or fq.LIB_PATH
L = fq.load_mlp(ctypes.CDLL(LIB_PATH))
STUBS = hasattr(L, "fp8q_mlp_stub_count")
P = lambda a: ctypes.c_void_p(a)
A = 0x7F0000000000                                      # 256-byte aligned fake base
E4, E5, F32, BF16, F16 = 0, 1, 0, 1, 2
at = lambda i, d=0: P(A + (i << 40) + d)                # far-apart fake buffers


def test_exports_match_header():
    declared = fq.mlp_header_functions()
    assert set(declared) == set(fq.MLP_FUNCTIONS)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert set(declared) <= set(re.findall(r" T (fp8q_\w+)$", out, re.M))


def _norm(name, **k):
    a = dict(x=at(1), xdt=BF16, res=at(2), w=at(3), b=at(9), wdt=BF16, rows=4, cols=256, eps=1e-5)
    a.update(dict(y=at(4)) if name == "fp8q_layernorm" else dict(fmt=E4, y=at(4), s=at(5)))
    a.update(h=at(6), mean=at(8), rstd=at(7), st=None)
    a.update(k)
    return getattr(L, name)(*a.values())


@pytest.mark.parametrize("name", ["fp8q_layernorm", "fp8q_layernorm_cast_group128", "fp8q_layernorm_cast_per_channel"])
def test_layernorm_errors(name):
    f = lambda **k: _norm(name, **k)
    plain = name == "fp8q_layernorm"
    assert f(xdt=3) == fq.EDTYPE
    assert f(wdt=F16) == fq.EDTYPE                         # neither x's type nor f32
    assert f(xdt=F32, wdt=BF16) == fq.EDTYPE
    assert f(rows=-1) == fq.EINVAL
    assert f(cols=-128) == fq.EINVAL
    assert f(rows=2 ** 31) == fq.EINVAL
    assert f(cols=2 ** 30 + 128) == fq.EINVAL
    for k in ("x", "w", "y"):
        assert f(**{k: None}) == fq.EINVAL, k
    for k in ("x", "res", "w", "b", "h"):
        assert f(**{k: P(A + 1)}) == fq.EALIGN, k
    for k in ("mean", "rstd"):
        assert f(**{k: P(A + 2)}) == fq.EALIGN, k
    assert f(y=at(1, 8)) == fq.EINVAL                      # y meets x but is not x
    assert f(h=at(1, 2)) == fq.EINVAL
    assert f(y=at(6)) == fq.EINVAL                         # y = h
    assert f(y=at(3)) == fq.EINVAL                         # y = the weight
    assert f(h=at(9)) == fq.EINVAL                         # h = the bias
    assert f(mean=at(7)) == fq.EINVAL
    assert f(mean=at(1)) == fq.EINVAL
    if plain:
        assert f(y=at(1), h=at(1)) == fq.EINVAL            # both over x
        assert f(y=P(A + 1)) == fq.EALIGN
    else:
        assert f(fmt=2) == fq.EDTYPE
        assert f(s=None) == fq.EINVAL
        assert f(s=P(A + 2)) == fq.EALIGN
        assert f(y=at(1)) == fq.EINVAL                     # codes never lie over x
        assert f(rstd=at(5)) == fq.EINVAL
    if name.endswith("128"):
        assert f(cols=100) == fq.ESHAPE
    assert f(rows=0, x=None, w=None, b=None, y=None, h=None) == fq.OK


def _norm_bwd(**k):
    a = dict(dy=at(1), h=at(2), dt=BF16, w=at(3), wdt=BF16, mean=at(9), rstd=at(4), dh=at(5), rows=4, cols=250, dx=at(6),
             dw=at(7), db=at(10), ws=at(8), st=None)
    a.update(k)
    return L.fp8q_layernorm_backward(*a.values())


def test_layernorm_backward_errors():
    assert _norm_bwd(dt=7) == fq.EDTYPE
    assert _norm_bwd(wdt=F16) == fq.EDTYPE
    assert _norm_bwd(rows=-1) == fq.EINVAL
    assert _norm_bwd(cols=2 ** 30 + 1) == fq.EINVAL
    for k in ("dy", "h", "w", "mean", "rstd", "dx", "ws"):
        assert _norm_bwd(**{k: None}) == fq.EINVAL, k
    assert _norm_bwd(ws=None, dw=None) == fq.EINVAL        # dbias needs it too
    for k in ("dy", "h", "w", "dh", "dx", "dw", "db"):
        assert _norm_bwd(**{k: P(A + 1)}) == fq.EALIGN, k
    for k in ("mean", "rstd"):
        assert _norm_bwd(**{k: P(A + 2)}) == fq.EALIGN, k
    assert _norm_bwd(ws=P(A + 4)) == fq.EALIGN
    assert _norm_bwd(dx=at(2)) == fq.EINVAL                # dx = h
    assert _norm_bwd(dx=at(1, 4)) == fq.EINVAL
    assert _norm_bwd(dw=at(6)) == fq.EINVAL
    assert _norm_bwd(db=at(7)) == fq.EINVAL                # dbias = dweight
    assert _norm_bwd(dx=at(1), db=at(1)) == fq.EINVAL      # dx in place, and dbias over it
    assert _norm_bwd(ws=at(1)) == fq.EINVAL
    assert _norm_bwd(cols=0) == fq.OK
    assert _norm_bwd(rows=0, dw=None, db=None, dy=None, h=None, w=None, mean=None, rstd=None, dx=None, ws=None) == fq.OK
    assert L.fp8q_layernorm_backward_workspace_bytes(4, 250) >= 2 * 4 * 250 * 4
    assert L.fp8q_layernorm_backward_workspace_bytes(-4, 250) == 0


def _act(cast=False, **k):
    a = dict(x=at(1), xf=E4, xs=at(2), w=at(3), wf=E4, wsc=at(4), M=300, N=256, K=256, b=at(5), bdt=BF16, act=1)
    a.update(dict(fmt=E4, q=at(7), s=at(8)) if cast else dict(res=at(6), y=at(7), ydt=BF16))
    a.update(z=at(9), zdt=BF16, ws=at(10), st=None)
    a.update(k)
    return (L.fp8q_linear_act_cast if cast else L.fp8q_linear_act)(*a.values())


@pytest.mark.parametrize("cast", [False, True])
def test_linear_act_errors(cast):
    f = lambda **k: _act(cast, **k)
    out = "q" if cast else "y"
    for bad in (5, -1):
        assert f(act=bad) == fq.EDTYPE
    for k in ("xf", "wf", "bdt", "zdt") + (("fmt",) if cast else ("ydt",)):
        assert f(**{k: 7}) == fq.EDTYPE, k
    assert f(K=130) == fq.ESHAPE
    for k in ("M", "N", "K"):
        assert f(**{k: -128}) == fq.EINVAL, k
    assert f(M=2 ** 31 + 1) == fq.EINVAL
    assert f(N=2 ** 21 + 128) == fq.EINVAL
    assert f(K=2 ** 21 + 128) == fq.EINVAL
    assert f(M=2 ** 31, N=2 ** 21) == fq.EINVAL            # more tiles than a grid holds
    for k in ("x", "xs", "w", "wsc", out):
        assert f(**{k: None}) == fq.EINVAL, k
    for k in ("x", "w"):
        assert f(**{k: P(A + 8)}) == fq.EALIGN, k
    for k in ("xs", "wsc"):
        assert f(**{k: P(A + 2)}) == fq.EALIGN, k
    for k in ("b", "z") + (() if cast else ("y", "res")):
        assert f(**{k: P(A + 1)}) == fq.EALIGN, k
    assert f(b=P(A + 2), bdt=F32) == fq.EALIGN
    assert f(z=at(7)) == fq.EINVAL                         # z = the output
    assert f(z=at(5, 64)) == fq.EINVAL                     # z meets the bias
    assert f(**{out: at(3)}) == fq.EINVAL
    assert f(**{out: at(5)}) == fq.EINVAL
    if cast:
        assert f(N=200) == fq.ESHAPE
        assert f(s=None) == fq.EINVAL
        assert f(s=P(A + 2)) == fq.EALIGN
        assert L.fp8q_linear_act_workspace_bytes(8, 256, 256, 1) >= 8 * 256 * 4
        assert f(M=8, ws=None) == fq.EINVAL
    else:
        assert f(y=at(6, 2)) == fq.EINVAL                  # y meets the residual but is not it
        assert f(z=at(6)) == fq.EINVAL
        need = L.fp8q_linear_act_workspace_bytes(100, 128, 1 << 15, 0)
        assert need > 0
        assert f(M=100, N=128, K=1 << 15, ydt=F32, bdt=F32, ws=None) == fq.EINVAL
        assert f(M=100, N=128, K=1 << 15, ydt=F32, bdt=F32, ws=P(A + 16)) == fq.EALIGN
        assert f(M=100, N=128, K=1 << 15, ydt=F32, bdt=F32, ws=at(6)) == fq.EINVAL
    assert f(M=0, x=None, ws=None) == fq.OK
    assert f(N=0, w=None, ws=None) == fq.OK
    assert L.fp8q_linear_act_workspace_bytes(-1, 128, 128, 0) == 0


def _act_bwd(**k):
    a = dict(dy=at(1), z=at(9), dt=BF16, x=at(2), xf=E4, xs=at(3), w=at(4), wf=E4, wsc=at(5), M=300, N=200, K=256, act=1,
             dx=at(6), dw=at(7), db=at(10), gdt=BF16, ws=at(8), st=None)
    a.update(k)
    return L.fp8q_linear_act_backward(*a.values())


def test_linear_act_backward_errors():
    f = _act_bwd
    assert f(dt=F32, gdt=F32) == fq.EDTYPE                 # gradients are 16-bit
    assert f(gdt=F16) == fq.EDTYPE
    assert f(xf=2) == fq.EDTYPE
    assert f(act=5) == fq.EDTYPE
    assert f(K=100) == fq.ESHAPE
    assert f(M=-1) == fq.EINVAL
    assert f(M=4194241) == fq.EINVAL
    assert f(N=2 ** 21 + 1) == fq.EINVAL
    assert f(N=2 ** 21, K=2 ** 21) == fq.EINVAL
    for k in ("dy", "z", "x", "xs", "w", "wsc", "ws"):
        assert f(**{k: None}) == fq.EINVAL, k
    assert f(x=P(A + 8)) == fq.EALIGN
    for k in ("dy", "z", "dx", "dw", "db"):
        assert f(**{k: P(A + 1)}) == fq.EALIGN, k
    assert f(ws=P(A + 128)) == fq.EALIGN
    assert f(dx=at(7)) == fq.EINVAL                        # dx = dw
    assert f(dx=at(1)) == fq.EINVAL
    assert f(db=at(9)) == fq.EINVAL
    assert f(db=at(7, 64)) == fq.EINVAL                    # dbias within dw
    assert f(dx=None, dw=None, db=None) == fq.OK
    assert f(K=0, db=None) == fq.OK
    assert f(M=0, dw=None, db=None) == fq.OK
    assert f(N=0, dx=None) == fq.OK
    w = L.fp8q_linear_act_backward_workspace_bytes
    assert w(0, 200, 256) == 0 and w(300, 200, 256) > w(300, 200, 0) > 0 and w(1, 1, 100) == 0


def test_python_linear_act_refuses():
    E = torch.float8_e4m3fn
    x, xs = torch.zeros(4, 256).to(E), torch.zeros(4, 2)
    w, ws = torch.zeros(200, 256).to(E), torch.zeros(2, 2)
    with pytest.raises(ValueError):                        # host tensors
        fq.linear_act_fp8(x, xs, w, ws)
    with pytest.raises(ValueError):                        # scales of another shape
        fq.linear_act_fp8(x, torch.zeros(4, 3), w, ws)
    with pytest.raises(ValueError):
        fq.linear_act_fp8(x, xs, w, ws, torch.zeros(199))
    with pytest.raises(TypeError):                         # not codes
        fq.linear_act_fp8(x.float(), xs, w, ws)
    with pytest.raises(TypeError):
        fq.linear_act_fp8(x, xs, w, ws, activation="swish2")
    with pytest.raises(TypeError):
        fq.linear_act_fp8(x, xs, w, ws, x_fmt="e5m2")
    with pytest.raises(ValueError):                        # residual of another type than y
        fq.linear_act_fp8(x, xs, w, ws, residual=torch.zeros(4, 200), out=(torch.zeros(4, 200).half(), None))
    with pytest.raises((ValueError, TypeError)):
        fq.linear_act_fp8_cast(x, xs, w, ws)               # 200 columns are no groups
    dy = torch.zeros(4, 200).bfloat16()
    with pytest.raises(ValueError):                        # no z
        fq.linear_act_fp8_backward(dy, None, x, xs, w, ws, "gelu")
    with pytest.raises(ValueError):                        # z of another type
        fq.linear_act_fp8_backward(dy, dy.half(), x, xs, w, ws, "gelu")
    with pytest.raises(TypeError):                         # weight gradients of two types
        fq.linear_act_fp8_backward(dy, None, x, xs, w, ws, out=(torch.zeros(4, 256).bfloat16(), torch.zeros(200, 256),
                                                                torch.zeros(200).bfloat16()))


def test_python_layernorm_refuses():
    x, w = torch.zeros(4, 128), torch.zeros(128)
    with pytest.raises(ValueError):                        # host tensors
        fq.layernorm(x, w)
    with pytest.raises(TypeError):
        fq.layernorm(x.double(), w)
    with pytest.raises(ValueError):
        fq.layernorm(x, torch.zeros(64))
    with pytest.raises(ValueError):                        # bias and weight of two types, or lengths
        fq.layernorm(x, w, torch.zeros(128).half())
    with pytest.raises(ValueError):
        fq.layernorm(x, w, torch.zeros(127))
    with pytest.raises(ValueError):
        fq.layernorm(x, w, residual=torch.zeros(4, 128).half())
    with pytest.raises(TypeError):
        fq.layernorm_cast(x, w, fp8_format="e3m4")
    with pytest.raises(ValueError):
        fq.layernorm(torch.zeros(()), w)
    s = torch.zeros(4)
    with pytest.raises(ValueError):
        fq.layernorm_backward(x.half(), x, w, s, s)
    with pytest.raises(ValueError):
        fq.layernorm_backward(x, x, w, s[:3], s)
    with pytest.raises(ValueError):                        # a workspace that is too small
        fq.fp8q_layernorm_backward(x, x, w, s, s, x, w, w, workspace=torch.zeros(16))


def test_calls_run_on_the_tensors_device(monkeypatch):
    """A call on tensors of another device than the current one makes theirs
    current for the launch; tensors of two devices are refused."""
    from dequantize_amax_reduce_amd import _mlp

    class T:
        def __init__(self, d):
            self.d = d

        def get_device(self):
            return self.d

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 7

    log = []

    class Dev:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            log.append(("enter", self.d))

        def __exit__(self, *_):
            log.append(("exit", self.d))

    class Lib:
        @staticmethod
        def f(*a):
            log.append(a)
            return 0

    monkeypatch.setattr(_mlp, "_current", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Dev)
    monkeypatch.setattr(_mlp, "lib", Lib)
    monkeypatch.setattr(_mlp, "_dev", lambda t, name: t.data_ptr())
    _mlp._call("f", 0, 1)
    assert log == [(1,)]
    log.clear()
    _mlp._call("f", 1, 2)
    assert log == [("enter", 1), (2,), ("exit", 1)]
    assert _mlp._at(T(1), "t", 1) == 7
    with pytest.raises(ValueError):
        _mlp._at(T(1), "t", 0)


@pytest.mark.skipif(not STUBS, reason="needs the launcher-stub build of the ABI layer (test_mlp_abi_under_asan_ubsan)")
def test_fuzz_validation():
    """Random calls with sizes at and beyond every limit: a documented status
    each time, no undefined behaviour, no broken launcher precondition."""
    import numpy as np
    rng = np.random.Generator(np.random.PCG64(79))
    sizes = [0, 1, 2, 63, 64, 65, 127, 128, 256, 4096, 2 ** 21, 2 ** 21 + 128, 4194240, 2 ** 30, 2 ** 31, 2 ** 40,
             2 ** 62, 2 ** 63 - 1, -1, -128, -(2 ** 63)]
    ptrs = [None, A, A + 1, A + 2, A + 4, A + 16, A + 4096] + [A + (i << 40) for i in range(1, 14)] + [2 ** 64 - 4096]
    enums = [0, 1, 2, 3, -1, 2 ** 31 - 1, -(2 ** 31)]
    codes = {fq.OK, fq.EINVAL, fq.EDTYPE, fq.ESHAPE, fq.EALIGN, fq.EHIP}
    reached = 0
    for name in fq.MLP_FUNCTIONS:
        fn = getattr(L, name)
        for _ in range(4000):
            args = []
            for t in fn.argtypes:
                if t is ctypes.c_void_p:
                    p = ptrs[int(rng.integers(0, len(ptrs)))] if rng.random() < 0.2 else A + (len(args) + 20 << 40)
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
                L.fp8q_mlp_stub_reset()
                st = fn(*args)
                assert st in codes, (name, args)
                reached += L.fp8q_mlp_stub_count()
                assert st == fq.OK or L.fp8q_mlp_stub_count() == 0, (name, args)
    assert reached > 100


def test_mlp_abi_under_asan_ubsan(tmp_path):
    if STUBS:
        pytest.skip("already the sanitizer build")
    from test_sanitizers import SAN, _run
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    lib = str(tmp_path / "libfp8q_mlp_abi_san.so")
    csrc = os.path.join(ROOT, "dequantize_amax_reduce_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-Wall", *SAN, "-D__HIP_PLATFORM_AMD__", "-I",
                    "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "fp8q_mlp_abi.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "fp8q_mlp_launch_stubs.cpp"), "-o", lib], check=True)
    out = _run("tests/test_mlp_host.py", {"FP8Q_MLP_ABI_LIB": lib})
    assert " passed" in out
