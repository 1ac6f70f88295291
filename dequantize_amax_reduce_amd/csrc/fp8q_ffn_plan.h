// fp8q_ffn_plan.h -- which kernel a feed-forward operator runs on, and in what
// shape: host arithmetic on sizes alone, without a HIP header, so that a CPU
// test can ask which sizes reach which kernel.  Internal; not part of the ABI.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace fp8q {

// ---------------------------------------------------------------------------
// forward products
// ---------------------------------------------------------------------------

constexpr int64_t kRowsMax = 16;       // rows that k_mm_rows takes
constexpr int64_t kExactMax = 64;      // rows up to which sums are binary32 whatever the outputs

// How a product is tiled: rows a tile, and workgroups over K (splits)
struct Plan {
    bool rows;
    int bm, splits, kper;
    int64_t tm, tn;
};

// The tile height and the split of K with the least estimated time.  A round
// of 256 workgroups takes the measured microseconds below per block of K (8192
// columns, K = 7168, every round full: fp8 sums 257, 282 and 350 us for 4096
// rows at heights 256, 128 and 64; binary32 sums 413 and 492 at 128 and 64)
// and about 4 to fill and drain; a split writes its partial sums and the join
// reads them, at about 5 TB/s and a launch.  ex: binary32 sums (k_mm's EX),
// whose tiles are at most 128 rows tall: the widened fragments leave registers
// for no more.
inline Plan plan(int64_t M, int64_t N, int64_t K, bool gated, bool ex) {
    Plan p{};
    const int64_t KB = K / 128;
    if (M <= kRowsMax) {
        p.rows = true;
        p.splits = 1;
        return p;
    }
    p.tn = (N + (gated ? 127 : 255)) / (gated ? 128 : 256);
    double best = 0.0;
    for (int bm = ex ? 128 : 256; bm >= 64; bm /= 2) {
        const double block = ex ? (bm == 128 ? 1.84 : 1.10) : (bm == 256 ? 2.30 : bm == 128 ? 1.26 : 0.78);
        const int64_t tm = (M + bm - 1) / bm, tiles = tm * p.tn;
        for (int64_t s = 1; s == 1 || (s <= 16 && tiles * s <= 512 && KB / s >= 2); s *= 2) {
            const int64_t kper = std::max<int64_t>(1, (KB + s - 1) / s);
            const double t = (double)((tiles * s + 255) / 256) * ((double)kper * block + 4.0) +
                             (s > 1 ? 3.0 + (double)(s * M * N * (gated ? 16 : 8)) / 5e6 : 0.0);
            if (best > 0.0 && t >= best) continue;
            best = t;
            p.bm = bm;
            p.tm = tm;
            p.kper = (int)kper;
            p.splits = (int)std::max<int64_t>(1, (KB + kper - 1) / kper);
        }
    }
    return p;
}

inline int64_t part_bytes(const Plan& p, int64_t M, int64_t N, bool gated) {
    return p.splits > 1 ? p.splits * M * N * (gated ? 8 : 4) : 0;
}

// Few rows through a projection with an epilogue: two MFMA tiles a workgroup
// tile where that leaves 144 workgroups or more, which draw from memory what 256
// draw, each the same number of tiles.  (Weights that no cache holds, one token:
// 7168 -> 18432 26.4 us with one MFMA tile and 256 workgroups, 28.4 with two and
// 256, 25.7 with two and 192; 12 tokens 18432 -> 7168 33.7 with one, 27.1 with
// two; one token 7168 -> 2048 6.7 with one, 7.2 with two and 64 workgroups.  A
// cast within the kernel, by workgroups that take whole groups of 128 columns,
// was slower than its own launch of 2 us but from 200 to 256 groups: 30.0 against
// 27.7 at 144, 43.5 against 50.4 at 224.)
inline bool wide_rows(int64_t N) { return (N + 31) / 32 >= 144; }
inline int64_t even_groups(int64_t tiles) {
    const int64_t rounds = (tiles + 255) / 256;
    return (tiles + rounds - 1) / rounds;
}

// ---------------------------------------------------------------------------
// backward products
// ---------------------------------------------------------------------------

inline int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

// The tile height and the split of the contraction with the least estimated
// time: a round of 256 workgroups takes the measured microseconds below per
// step of 64 (4096 x 8192 outputs of 4096-long sums: 200, 232 and 256 us at
// heights 256, 128 and 64) and about 4 to fill and drain; a split writes
// binary32 sums that the join reads, at about 5 TB/s and a launch.
struct Plan16 {
    int bm, splits, kper;
    int64_t part;          // bytes of partial sums
};
inline Plan16 plan16(int64_t M, int64_t N, int64_t K) {
    Plan16 p{};
    const int64_t KB = K / 64, tn = (N + 255) / 256;
    double best = 0.0;
    for (int h = 256; h >= 64; h /= 2) {
        const double each = h == 256 ? 1.56 : h == 128 ? 0.90 : 0.50;
        const int64_t tiles = (M + h - 1) / h * tn;
        for (int64_t s = 1; s == 1 || (s <= 32 && tiles * s <= 512 && KB / s >= 4); s *= 2) {
            const int64_t kper = (KB + s - 1) / s, n = (KB + kper - 1) / kper;
            const double t = (double)((tiles * n + 255) / 256) * ((double)kper * each + 4.0) +
                             (n > 1 ? 3.0 + (double)(n * M * N * 8) / 5e6 : 0.0);
            if (best > 0.0 && t >= best) continue;
            best = t;
            p = Plan16{h, (int)n, (int)kper, n > 1 ? n * M * N * 4 : 0};
        }
    }
    return p;
}
// The two products of a backward pass: dx, and the weight gradients (for a
// gated pair one product, the gate's rows padded to 64).  With a rest the
// contraction is padded to 128 and half as long again in time.
inline int64_t rows_padded(int64_t M, bool rest) { return rest ? (M + 127) / 128 * 128 : up64(M); }
// columns of dz: of a gated pair twice N padded to 64, so a multiple of 128
inline int64_t dz_columns(int64_t N, bool gated, bool rest) {
    return gated ? 2 * up64(N) : rest ? (N + 127) / 128 * 128 : up64(N);
}
inline Plan16 plan_dx(int64_t M, int64_t N, int64_t K, bool gated, bool rest) {
    const int64_t C = dz_columns(N, gated, rest);
    return plan16(M, K, rest ? C + C / 2 : C);
}
inline Plan16 plan_dw(int64_t M, int64_t N, int64_t K, bool gated, bool rest) {
    const int64_t C = rows_padded(M, rest);
    return plan16(gated ? up64(N) + N : N, K, rest ? C + C / 2 : C);
}

// ---------------------------------------------------------------------------
// norms
// ---------------------------------------------------------------------------

constexpr int kNormWaves = 8192;  // waves a launch of the forward pass asks for: what the chip holds at once
constexpr int kBwdParts = 512;   // workgroups (and partial dweight rows) of the backward pass

// How a norm's rows are held: a wave or a workgroup a row, with V lane vectors
// a thread; or in passes over a row that is too long for registers (V = 0)
struct NormPlan {
    bool wave;
    int V, threads;
    int64_t groups;        // workgroups
    int64_t at_once;       // rows that the grid takes at once
};

// Lane vectors a thread (V) for a row of nv vectors held by one workgroup:
// two, so that the workgroup is about nv / 2 threads and several fit a CU;
// one or four where the row is short or long.
inline int pick_v(int64_t nv) {
    if (nv <= 256) return 1;
    return nv <= 2048 ? 2 : 4;
}
inline int threads_for(int64_t nv, int V) { return (int)std::min<int64_t>(1024, ((nv + V - 1) / V + 63) / 64 * 64); }

// nv: 16-byte vectors of a row
inline NormPlan norm_plan(int64_t rows, int64_t nv) {
    if (nv <= 128 && rows > 256) {                          // short rows: a wave each, no barrier
        const int64_t g = std::min<int64_t>((rows + 3) / 4, kNormWaves / 4);
        return NormPlan{true, nv <= 64 ? 1 : 2, 256, g, 4 * g};
    }
    if (nv <= 4096) {
        const int V = pick_v(nv), T = threads_for(nv, V);
        const int64_t g = std::min<int64_t>(rows, std::max(256, kNormWaves / (T / 64) / 256 * 256));
        return NormPlan{false, V, T, g, g};
    }
    const int64_t g = std::min<int64_t>(rows, int64_t(1) << 20);
    return NormPlan{false, 0, 1024, g, g};
}

// Layer norm: one vector a thread up to 1024 vectors, whose rows' next loads
// are in flight beside at most 64 registers, so that 32 waves fit a CU (16384 x
// 7168 bf16: 155 us against 161 with two vectors and half the threads); two
// vectors up to 2048 (20 waves), four up to 4096 (16; 512 x 32768 bf16 36 us,
// 43 in passes).  As many workgroups as fit (1999 x 5001 f32: 17.1 us with the two
// of 10 waves that fit, 18.4 with three).  tiny: rows shorter than a vector.
inline NormPlan layernorm_plan(int64_t rows, int64_t nv, bool tiny) {
    if (nv > 4096 || tiny) {
        const int64_t g = std::min<int64_t>(rows, int64_t(1) << 20);
        return NormPlan{false, 0, 1024, g, g};
    }
    if (nv <= 128 && rows > 256) return norm_plan(rows, nv);
    const int V = nv <= 1024 ? 1 : nv <= 2048 ? 2 : 4, T = threads_for(nv, V);
    const int64_t fit = std::max(1, (V == 1 ? 32 : V == 2 ? 20 : 16) / (T / 64));
    const int64_t g = std::min<int64_t>(rows, 256 * fit);
    return NormPlan{false, V, T, g, g};
}

inline int64_t norm_bwd_parts(int64_t rows) { return std::min<int64_t>(rows < 1 ? 1 : rows, kBwdParts); }
inline NormPlan norm_bwd_plan(int64_t rows, int64_t nv) {
    const int64_t g = norm_bwd_parts(rows);
    if (nv > 2048) return NormPlan{false, 0, 1024, g, g};
    const int V = nv <= 256 ? 1 : 2;
    return NormPlan{false, V, threads_for(nv, V), g, g};
}

}  // namespace fp8q
