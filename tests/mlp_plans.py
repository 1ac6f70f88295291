"""Sizes of layer norm, and of a projection's backward pass through an
activation with f16 gradients, at which every kernel variant runs past its first
row or steps.  As in ffn_plans.py, the host's choice is asked of
csrc/fp8q_ffn_plan.h: test_mlp_plans.py checks the tables on the CPU,
test_gpu_layernorm.py and test_gpu_linear_act.py run them."""
import ctypes
import os
import subprocess

from ffn_plans import CSRC, ROOT, vectors

# (rows, columns, dtype): (a wave a row, vectors a thread, threads, rows the grid takes at once)
LAYERNORM = {
    (8300, 256, "bf16"): (True, 1, 256, 8192),
    (8300, 384, "f32"): (True, 2, 256, 8192),
    (8300, 201, "f32"): (True, 1, 256, 8192),
    (8300, 701, "bf16"): (True, 2, 256, 8192),
    (2900, 1152, "bf16"): (False, 1, 192, 2560),
    (2900, 1153, "f16"): (False, 1, 192, 2560),
    (600, 7168, "bf16"): (False, 1, 896, 512),
    (600, 4001, "f32"): (False, 1, 1024, 512),
    (600, 5120, "f32"): (False, 2, 640, 512),
    (600, 5001, "f32"): (False, 2, 640, 512),
    (300, 14336, "f16"): (False, 2, 896, 256),
    (300, 8001, "f32"): (False, 2, 1024, 256),
    (300, 32768, "f16"): (False, 4, 1024, 256),
    (300, 17001, "bf16"): (False, 4, 576, 256),
}

# (M, K, N): (rows a tile, splits, steps of 64 a split) of dx and of dw; a split
# may hold steps of the rest alone, of both, or of neither
BACKWARD_REST = {
    (17, 128, 72): ((64, 1, 3), (64, 1, 3)),
    (17, 128, 640): ((64, 2, 8), (64, 1, 3)),
    (513, 128, 64): ((64, 1, 3), (64, 2, 8)),
    (200, 384, 8200): ((64, 28, 7), (128, 1, 6)),
    (2100, 128, 4104): ((128, 15, 7), (64, 2, 26)),
    (3000, 128, 4104): ((64, 4, 25), (128, 4, 18)),
    (4100, 128, 4104): ((256, 15, 7), (256, 15, 7)),
    (4100, 1024, 256): ((128, 1, 6), (64, 15, 7)),
    (4100, 2048, 130): ((256, 1, 6), (64, 8, 13)),
    (200, 640, 12300): ((64, 16, 19), (256, 1, 6)),
}


class LayerNormPlan:
    def __init__(self, folder):
        lib = os.path.join(str(folder), "libmlp_plan_shim.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fPIC", "-shared", "-I", CSRC,
                        os.path.join(ROOT, "tests", "mlp_plan_shim.cpp"), "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)

    def __call__(self, rows, cols, dt):
        out = (ctypes.c_int64 * 4)()
        self.lib.shim_layernorm(ctypes.c_int64(rows), ctypes.c_int64(vectors(cols, dt)),
                                ctypes.c_int(cols < (4 if dt == "f32" else 8)), out)
        return (bool(out[0]), *tuple(out)[1:])
