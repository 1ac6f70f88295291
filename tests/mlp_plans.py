"""Sizes of layer norm, of a projection with an epilogue, and of its backward
pass, at which every kernel variant runs past its first row or steps.  As in ffn_plans.py, the host's choice is asked of
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

# (M, K, N): (rows a tile, splits, steps of 64 a split) of dx and of dw, and whether
# one launch has both
BACKWARD = {
    (200, 128, 1280): ((64, 4, 5), (64, 1, 4), False),
    (1000, 128, 72): ((64, 1, 2), (64, 4, 4), False),
    (200, 384, 8200): ((64, 26, 5), (128, 1, 4), False),
    (130, 128, 130): ((128, 1, 3), (128, 1, 3), True),
    (4100, 128, 2053): ((64, 2, 17), (128, 13, 5), False),
    (200, 640, 12300): ((64, 15, 13), (192, 1, 4), False),
    (200, 1024, 12300): ((64, 15, 13), (256, 1, 4), False),
    (17, 128, 1280): ((64, 4, 5), (64, 1, 1), False),
    (6000, 640, 130): ((128, 1, 3), (64, 16, 6), False),
    (2100, 128, 4104): ((128, 13, 5), (64, 2, 17), False),
    (4100, 2048, 130): ((192, 1, 3), (64, 8, 9), False),
    (4100, 2048, 250): ((192, 1, 4), (64, 8, 9), False),
    (8192, 128, 4104): ((64, 2, 33), (256, 8, 16), False),
    (4100, 128, 8192): ((256, 8, 16), (64, 2, 33), False),
    (1000, 5120, 640): ((192, 1, 10), (192, 1, 16), True),
    (1000, 5120, 1280): ((256, 1, 20), (256, 1, 16), True),
    (1000, 128, 130): ((64, 1, 3), (64, 4, 4), False),
    (4100, 3584, 130): ((256, 1, 3), (64, 4, 17), False),
}

# the same of f16 gradients through an activation, whose contractions begin with the
# rest's steps: a split may hold steps of the rest alone, of both, or of neither
BACKWARD_REST = {
    (17, 128, 640): ((64, 2, 8), (64, 1, 3), False),
    (513, 128, 72): ((64, 1, 3), (64, 2, 8), False),
    (200, 384, 8200): ((64, 28, 7), (128, 1, 6), False),
    (130, 128, 130): ((128, 1, 6), (128, 1, 6), True),
    (4100, 128, 2053): ((64, 2, 26), (128, 15, 7), False),
    (200, 640, 12300): ((64, 16, 19), (192, 1, 6), False),
    (200, 1024, 12300): ((64, 16, 19), (256, 1, 6), False),
    (2100, 128, 4104): ((128, 15, 7), (64, 2, 26), False),
    (6000, 640, 72): ((128, 1, 3), (64, 29, 5), False),
    (4100, 2048, 72): ((192, 1, 3), (64, 15, 7), False),
    (4100, 3584, 72): ((256, 1, 3), (64, 8, 13), False),
    (4100, 128, 4104): ((256, 15, 7), (256, 15, 7), False),
    (1000, 5120, 640): ((192, 1, 15), (192, 1, 24), True),
    (1000, 5120, 1280): ((256, 1, 30), (256, 1, 24), True),
    (3000, 128, 4104): ((64, 4, 25), (128, 4, 18), False),
}

# (M, K, N) whose gradients one launch has: rows a tile of dx and of dw, each without the other
ALONE = {
    (130, 128, 130): (64, 64),
    (65, 4736, 834): (64, 128),
    (811, 4992, 65): (128, 64),
    (257, 4992, 1580): (64, 192),
    (1713, 4992, 339): (192, 64),
    (1000, 5120, 640): (128, 64),
    (2048, 4096, 4096): (128, 256),
}
ALONE_REST = {(64, 128, 65): (64, 64), (129, 4992, 787): (64, 128), (887, 4736, 138): (128, 64), (2048, 4096, 4096): (128, 256)}

# (M, K, N, binary32 sums): (rows a tile, splits, blocks a split, column tiles of
# 256, narrower ones, their width / 64) of a projection with an epilogue; a
# pipeline has 3 stages (2 of 256 rows), and one block more is its steady step
ACT = {
    (70, 640, 72, True): (64, 1, 5, 0, 1, 2),
    (300, 640, 8200, True): (64, 1, 5, 0, 65, 2),
    (200, 640, 300, False): (64, 1, 5, 0, 3, 2),
    (1003, 1024, 1501, False): (64, 1, 8, 0, 12, 2),
    (400, 1280, 7168, True): (64, 1, 10, 28, 0, 4),
    (500, 7168, 4104, False): (64, 1, 56, 17, 0, 4),
    (1900, 1024, 4224, False): (128, 1, 8, 17, 0, 4),
    (1900, 1024, 4224, True): (128, 1, 8, 17, 0, 4),
    (4000, 640, 4096, False): (256, 1, 5, 16, 0, 4),
    (4096, 640, 5120, False): (256, 1, 5, 8, 16, 3),
    (2050, 512, 8300, False): (256, 1, 4, 19, 18, 3),
    (65, 7168, 300, False): (64, 14, 4, 2, 0, 4),
    (70, 7168, 128, True): (64, 14, 4, 1, 0, 4),
}

# (rows, columns, dtype) of the norm's backward pass: (vectors a thread, threads, workgroups)
LAYERNORM_BACKWARD = {
    (600, 1501, "bf16"): (1, 192, 512),
    (520, 2048, "f16"): (1, 256, 512),
    (600, 1001, "f32"): (1, 256, 512),
    (530, 7168, "f16"): (2, 448, 512),
    (515, 4101, "bf16"): (2, 320, 512),
    (600, 4001, "f32"): (2, 512, 512),
    (600, 8200, "bf16"): (2, 576, 512),
    (515, 12001, "bf16"): (2, 768, 512),
    (520, 16384, "f16"): (2, 1024, 512),
    (600, 5001, "f32"): (2, 640, 512),
    (515, 8192, "f32"): (2, 1024, 512),
    (514, 16400, "bf16"): (0, 1024, 512),
    (514, 16401, "f16"): (0, 1024, 512),
    (600, 8193, "f32"): (0, 1024, 512),
}


class MlpPlans:
    def __init__(self, folder):
        lib = os.path.join(str(folder), "libmlp_plan_shim.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fPIC", "-shared", "-I", CSRC,
                        os.path.join(ROOT, "tests", "mlp_plan_shim.cpp"), "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)

        self.lib.shim_mixed_rounds.restype = self.lib.shim_time16.restype = ctypes.c_double

    def layernorm(self, rows, cols, dt):
        out = (ctypes.c_int64 * 4)()
        self.lib.shim_layernorm(ctypes.c_int64(rows), ctypes.c_int64(vectors(cols, dt)),
                                ctypes.c_int(cols < (4 if dt == "f32" else 8)), out)
        return (bool(out[0]), *tuple(out)[1:])

    def layernorm_backward(self, rows, cols, dt):
        out = (ctypes.c_int64 * 3)()
        self.lib.shim_layernorm_bwd(ctypes.c_int64(rows), ctypes.c_int64(vectors(cols, dt)), out)
        return tuple(out)

    def act(self, M, K, N, exact):
        out = (ctypes.c_int64 * 7)()
        self.lib.shim_act(*(ctypes.c_int64(v) for v in (M, N, K)), ctypes.c_int(exact), out)
        return tuple(out)

    def mixed_rounds(self, whole, part, r):
        return self.lib.shim_mixed_rounds(ctypes.c_int64(whole), ctypes.c_int64(part), ctypes.c_double(r))

    def backward(self, M, K, N, rest):
        out = (ctypes.c_int64 * 7)()
        self.lib.shim_bwd_act(*(ctypes.c_int64(v) for v in (M, N, K)), ctypes.c_int(rest), out)
        return tuple(out)[:3], tuple(out)[3:6], bool(out[6])

    def alone(self, M, K, N, rest):
        out = (ctypes.c_int64 * 2)()
        self.lib.shim_bwd_alone(*(ctypes.c_int64(v) for v in (M, N, K)), ctypes.c_int(rest), out)
        return tuple(out)

    def time16(self, M, N, steps, bm):
        return self.lib.shim_time16(*(ctypes.c_int64(v) for v in (M, N, steps)), ctypes.c_int(bm))
