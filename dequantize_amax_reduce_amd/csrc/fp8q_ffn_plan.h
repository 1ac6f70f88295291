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

// A projection with an epilogue: as plan(), and two more kinds of tiles.
// Where 64 x 256 tiles are few, 64 x 128, of which two fit a CU; they take 0.44
// us (binary32 sums: 0.67) a block of K, as many at once or in turn.  In us,
// 16-bit output with residual / group cast: 1003 x 4096 -> 2048 26.7 and 31.4 with
// 64 x 256, 18.7 and 25.3 with 64 x 128; 100 x 512 -> 512 8.0 and 12.3, 5.9 and 8.1;
// the other way 300 x 7168 -> 2048 21.4 and 25.2 (split), 26.0 and 37.7.
// And where 256 x 256 tiles do not fill their last round of 256 workgroups, the
// last columns in tiles of 192, of which a workgroup takes one after its whole
// tiles: 8192 x 2048 -> 4608 137.4 us with one width, 113.8 with two; 4096 x 4096
// -> 5120 135.3 and 122.9; 4096 x 18432 -> 7168 528.0 and 513.7.
struct PlanAct {
    Plan p;                // p.tn: column tiles of 256
    int64_t tn2;           // then those of 64 nt2
    int nt2;               // 4: none
};

// The rounds (in whole tiles' time) after which 256 workgroups have taken
// `whole` tiles and then `part` tiles of r rounds each
inline double mixed_rounds(int64_t whole, int64_t part, double r) {
    const int64_t q = whole / 256, rem = whole % 256;      // rem workgroups have taken q + 1
    const double least = (double)(q + (rem > 0));
    if (part == 0) return least;
    double best = 1e30;
    for (int late = 0; late < 2; ++late)
        for (int64_t k = 1 - late;; ++k) {                  // ends at a multiple of r after q, or after q + 1
            const double t = (double)(q + late) + (double)k * r;
            if (t >= best) break;
            const int64_t first = (int64_t)((t - (double)q) / r + 1e-6);
            const int64_t second = t > (double)(q + 1) ? (int64_t)((t - (double)(q + 1)) / r + 1e-6) : 0;
            if ((256 - rem) * first + rem * second < part) continue;
            best = t;
            break;
        }
    return std::max(best, least);
}

inline PlanAct plan_act(int64_t M, int64_t N, int64_t K, bool ex) {
    PlanAct r{plan(M, N, K, false, ex), 0, 4};
    if (r.p.rows || K == 0) return r;
    const double KB = (double)(K / 128);
    const double each = ex ? (r.p.bm == 128 ? 1.84 : 1.10) : (r.p.bm == 256 ? 2.30 : r.p.bm == 128 ? 1.26 : 0.78);
    const int64_t tiles = r.p.tm * r.p.tn;
    double best = (double)((tiles * r.p.splits + 255) / 256) * ((double)r.p.kper * each + 6.0) +
                  (r.p.splits > 1 ? 5.0 + (double)(r.p.splits * M * N * 8) / 5e6 : 0.0);
    // 64 x 128
    const int64_t tm = (M + 63) / 64, tn = (N + 127) / 128, rounds = (tm * tn + 255) / 256;
    const double t = (double)rounds * KB * (ex ? 0.67 : 0.44) + 4.5 * (double)((rounds + 1) / 2);
    if (t < best) {
        best = t;
        r.p.bm = 64;
        r.p.splits = 1;
        r.p.kper = (int)(K / 128);
        r.p.tm = tm;
        r.p.tn = 0;
        r.tn2 = tn;
        r.nt2 = 2;
    }
    // 256 x 256 and 256 x 192
    const int64_t th = (M + 255) / 256, whole = (N + 255) / 256;
    if (!ex && th * whole > 128 && th * whole <= 2048) {
        const double w = KB * 2.30 + 6.0, part = (KB * 1.80 + 5.0) / w;
        for (int64_t b = 1; b <= 32 && 192 * b < N + 192; ++b) {
            const int64_t a = std::max<int64_t>(0, (N - 192 * b + 255) / 256);
            if (256 * a + 192 * (b - 1) >= N) continue;     // the last would begin past the end
            const double u = mixed_rounds(th * a, th * b, part) * w;
            if (u >= best) continue;
            best = u;
            r.p.bm = 256;
            r.p.splits = 1;
            r.p.kper = (int)(K / 128);
            r.p.tm = th;
            r.p.tn = a;
            r.tn2 = b;
            r.nt2 = 3;
        }
    }
    return r;
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

// The backward pass of a projection with an epilogue: a height of 192 besides
// (1.21 us a step), and both products in one launch, the longer tiles first, where
// that takes less.  3001 x 4096 -> 4096 has 192 tiles of 256 rows for dx and 256 for
// dw, which are two rounds in any order, and 256 and 256 with tiles of 192 rows for
// dx: 223.5 -> 214.4 us.  4096 x 7168 -> 18432 has 448 tiles of 288 steps and 2016
// of 64: 2028 -> 1990 in one launch; 2048 x 4096 -> 4096 154.3 -> 146.4; 4096 x 2048
// -> 5120 241.5 -> 225.2.
struct PlanBwd {
    Plan16 dx, dw;
    bool both;
};
inline double each16(int bm) { return bm == 256 ? 1.56 : bm == 192 ? 1.21 : bm == 128 ? 0.90 : 0.50; }
inline double time16(const Plan16& p, int64_t M, int64_t N) {
    const int64_t tiles = (M + p.bm - 1) / p.bm * ((N + 255) / 256) * p.splits;
    return (double)((tiles + 255) / 256) * ((double)p.kper * each16(p.bm) + 4.0) +
           (p.splits > 1 ? 3.0 + (double)(p.splits * M * N * 8) / 5e6 : 0.0);
}
// One product of a joint launch, asked for without the other: the height of its own
// least time for M x N outputs of `steps` steps.  Unsplit as in the joint launch, so
// that a gradient has the same bits with and without the other.  (dx of 2048 x 4096 ->
// 4096 114.9 us at the joint launch's height, 86.7 so; dw of 1000 x 5120 -> 640 41.9 / 34.2.)
inline Plan16 alone16(int64_t M, int64_t N, int64_t steps) {
    Plan16 p{256, 1, (int)steps, 0};
    for (int h : {192, 128, 64}) {
        const Plan16 alt{h, 1, (int)steps, 0};
        if (time16(alt, M, N) < time16(p, M, N)) p = alt;
    }
    return p;
}
inline PlanBwd plan_bwd_act(int64_t M, int64_t N, int64_t K, bool rest) {
    const int64_t C = dz_columns(N, false, rest), R = rows_padded(M, rest);
    const int64_t s1 = (rest ? C + C / 2 : C) / 64, s2 = (rest ? R + R / 2 : R) / 64;   // steps
    PlanBwd p{plan_dx(M, N, K, false, rest), plan_dw(M, N, K, false, rest), false};
    auto taller = [&](Plan16& q, int64_t rows, int64_t steps) {
        const Plan16 alt{192, 1, (int)steps, 0};
        if (time16(alt, rows, K) < time16(q, rows, K)) q = alt;
    };
    taller(p.dx, M, s1);
    taller(p.dw, N, s2);
    double best = time16(p.dx, M, K) + time16(p.dw, N, K);
    for (int h : {256, 192, 128}) {
        const int64_t tn = (K + 255) / 256, t1 = (M + h - 1) / h * tn, t2 = (N + h - 1) / h * tn;
        if (t1 + t2 > 8192) continue;                       // the last round is little of so many
        const double d1 = (double)s1 * each16(h) + 4.0, d2 = (double)s2 * each16(h) + 4.0;
        const double t = d1 >= d2 ? mixed_rounds(t1, t2, d2 / d1) * d1 : mixed_rounds(t2, t1, d1 / d2) * d2;
        if (t >= best) continue;
        best = t;
        p = PlanBwd{Plan16{h, 1, (int)s1, 0}, Plan16{h, 1, (int)s2, 0}, true};
    }
    return p;
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
// of 10 waves that fit, 18.4 with three; both before the sums over waves took fewer
// instructions, as the 155 and 161 above: 146 and 16.1 now).  tiny: rows shorter than a vector.
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
