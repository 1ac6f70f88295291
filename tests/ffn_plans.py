"""Sizes of the feed-forward operators at which every kernel variant runs past
its first steps, with the variant each is meant to reach.  The host's choice
(csrc/fp8q_ffn_plan.h) is compiled with g++ and asked: tests/test_ffn_plans.py
checks the tables on the CPU, tests/test_gpu_ffn_plans.py runs them."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dequantize_amax_reduce_amd", "csrc")

# (M, K, N, gated, binary32 sums): (rows a tile, splits of K, blocks of 128 a split).
# A tile's pipeline has 3 stages (2 at 256 rows); one block more reaches its steady step.
FORWARD = {
    (17, 640, 72, False, True): (64, 1, 5),
    (1030, 7168, 72, False, True): (64, 8, 7),
    (1000, 640, 4104, False, True): (128, 1, 5),
    (4100, 3584, 72, False, True): (128, 4, 7),
    (65, 640, 72, False, False): (64, 1, 5),
    (1030, 7168, 61, False, False): (64, 8, 7),
    (1000, 640, 4101, False, False): (128, 1, 5),
    (4100, 3584, 72, False, False): (128, 4, 7),
    (1000, 512, 8200, False, False): (256, 1, 4),
    (4100, 3840, 33, False, False): (256, 8, 4),
    (17, 640, 128, True, True): (64, 1, 5),
    (17, 3584, 128, True, True): (64, 7, 4),
    (200, 512, 8320, True, True): (128, 1, 4),
    (400, 10240, 640, True, True): (128, 8, 10),
    (65, 640, 72, True, False): (64, 1, 5),
    (65, 3584, 61, True, False): (64, 7, 4),
    (200, 640, 8200, True, False): (128, 1, 5),
    (4100, 3584, 61, True, False): (128, 4, 7),
    (1000, 512, 4101, True, False): (256, 1, 4),
    (4100, 3840, 16, True, False): (256, 8, 4),
}

# (M, K, N, gated): (rows a tile, splits, steps of 64 a split) of dx and of the weight gradients
BACKWARD = {
    (200, 128, 200, False): ((64, 1, 4), (64, 1, 4)),
    (200, 128, 72, False): ((64, 1, 2), (64, 1, 4)),
    (1000, 128, 72, False): ((64, 1, 2), (64, 4, 4)),
    (17, 128, 1024, False): ((64, 4, 4), (64, 1, 1)),
    (4100, 1024, 256, False): ((128, 1, 4), (64, 8, 9)),
    (200, 384, 8200, False): ((64, 26, 5), (128, 1, 4)),
    (2100, 128, 4104, False): ((128, 13, 5), (64, 2, 17)),
    (5000, 128, 4104, False): ((64, 2, 33), (128, 4, 20)),
    (4100, 2048, 256, False): ((256, 1, 4), (64, 8, 9)),
    (200, 1024, 8200, False): ((64, 15, 9), (256, 1, 4)),
    (8192, 128, 4104, False): ((64, 2, 33), (256, 8, 16)),
    (4100, 128, 8192, False): ((256, 8, 16), (64, 2, 33)),
    (1000, 128, 72, True): ((64, 1, 4), (64, 4, 4)),
    (17, 128, 640, True): ((64, 4, 5), (64, 1, 1)),
    (200, 128, 8200, True): ((64, 29, 9), (128, 1, 4)),
    (2100, 128, 4104, True): ((128, 15, 9), (64, 1, 33)),
    (5000, 128, 2176, True): ((64, 2, 34), (128, 4, 20)),
    (4100, 2048, 100, True): ((256, 1, 4), (64, 8, 9)),
    (200, 384, 8200, True): ((64, 29, 9), (256, 1, 4)),
    (8192, 128, 2177, True): ((64, 2, 35), (256, 8, 16)),
    (4100, 128, 4104, True): ((256, 15, 9), (64, 1, 65)),
    (4100, 1024, 100, True): ((128, 1, 4), (64, 13, 5)),
}

# (M, K, F) of a gated pair with f16 gradients, whose contractions begin with the
# rest's steps; a split may hold steps of the rest alone, of both, or of neither
BACKWARD_REST = {
    (17, 128, 72): ((64, 1, 6), (64, 1, 3)),
    (17, 128, 640): ((64, 4, 8), (64, 1, 3)),
    (513, 128, 64): ((64, 1, 3), (64, 2, 8)),
    (200, 128, 200): ((64, 1, 12), (64, 1, 6)),
    (200, 128, 8200): ((64, 30, 13), (128, 1, 6)),
    (200, 384, 8200): ((64, 30, 13), (256, 1, 6)),
    (2100, 128, 2053): ((128, 15, 7), (64, 2, 26)),
    (3000, 128, 2052): ((64, 4, 25), (128, 4, 18)),
    (4100, 128, 2053): ((256, 15, 7), (256, 15, 7)),
    (4100, 2048, 72): ((256, 1, 6), (64, 8, 13)),
    (6000, 640, 72): ((128, 1, 6), (64, 16, 9)),
}

# (rows, columns, dtype): (a wave a row, lane vectors a thread, threads, rows the grid takes at once)
NORM = {
    (8300, 256, "bf16"): (True, 1, 256, 8192),
    (8300, 384, "f32"): (True, 2, 256, 8192),
    (2700, 1152, "bf16"): (False, 1, 192, 2560),
    (2700, 2304, "f16"): (False, 2, 192, 2560),
    (1300, 5120, "f32"): (False, 2, 640, 768),
    (530, 32768, "f16"): (False, 4, 1024, 512),
}
NORM_ODD = {                                                # a scale a row
    (8300, 201, "f32"): (True, 1, 256, 8192),
    (8300, 701, "bf16"): (True, 2, 256, 8192),
    (2700, 1153, "f16"): (False, 1, 192, 2560),
    (1600, 5001, "bf16"): (False, 2, 320, 1536),
    (1300, 5001, "f32"): (False, 2, 640, 768),
    (800, 17001, "bf16"): (False, 4, 576, 768),
}
NORM_BACKWARD = {
    (1100, 1153, "bf16"): (False, 1, 192, 512),
    (1100, 7168, "bf16"): (False, 2, 448, 512),
    (1100, 5001, "f32"): (False, 2, 640, 512),
    (600, 8197, "f32"): (False, 0, 1024, 512),
}


def vectors(cols, dt):
    ve = 4 if dt == "f32" else 8
    return (cols + ve - 1) // ve


class Plans:
    def __init__(self, folder):
        lib = os.path.join(str(folder), "libffn_plan_shim.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fPIC", "-shared", "-I", CSRC,
                        os.path.join(ROOT, "tests", "ffn_plan_shim.cpp"), "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)

    def _ask(self, name, n, sizes, flags=()):
        out = (ctypes.c_int64 * 4)()
        getattr(self.lib, name)(*(ctypes.c_int64(v) for v in sizes), *(ctypes.c_int(int(f)) for f in flags), out)
        return tuple(out)[:n]

    def forward(self, M, K, N, gated, exact):
        return self._ask("shim_fwd", 3, (M, N, K), (gated, exact))

    def backward(self, M, K, N, gated, rest=False):
        return tuple(self._ask(f, 3, (M, N, K), (gated, rest)) for f in ("shim_dx", "shim_dw"))

    def norm(self, rows, cols, dt):
        w, *rest = self._ask("shim_norm", 4, (rows, vectors(cols, dt)))
        return (bool(w), *rest)

    def norm_backward(self, rows, cols, dt):
        w, *rest = self._ask("shim_norm_bwd", 4, (rows, vectors(cols, dt)))
        return (bool(w), *rest)
