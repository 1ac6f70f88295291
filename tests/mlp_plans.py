"""Sizes of a projection's backward pass through an activation, with f16
gradients, at which every variant of the products whose contractions begin with
the rest's steps runs past its first steps.  As in ffn_plans.py, the host's
choice is asked of csrc/fp8q_ffn_plan.h: test_mlp_plans.py checks the table on
the CPU, test_gpu_linear_act.py runs it."""

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
