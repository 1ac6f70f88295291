// fp8q_layernorm.hip -- residual addition, layer norm and the cast of its
// result to fp8 (or its rounding to the input's type), and the norm's backward
// pass.
//
//   h = x + r;  mean = sum h / C;  rstd = 1 / sqrt(sum (h - mean)^2 / C + eps);
//   y = ((h - mean) * rstd) * w + b;  q, scale_inv = cast(y).
//
// Bound by HBM: x and r are read once, h and y (or its codes and scales)
// written once.  A row stays in registers between its reductions, as binary32.
// The instructions are close behind: 41 an element (a quarter of them the three sums
// over the workgroup and their divisions) took 160 to 180 us for 16384 x 7168 as the
// clock fell under load, 32 take 149 to 157.
//
// The mean is m0 + m1: m0 the rounded mean of h, m1 the mean of d = h - m0,
// which is exact where h is near m0; the variance is mean(d^2) - m1^2.  So a
// row of values far from zero keeps the bits that its deviations have in h (and m1
// is left out where it would add roundings instead: second_mean).
// (With m0 alone a constant row of 1000s, whose y is b, would be off by what
// m0's rounding leaves: 6e-5 / sqrt(eps), 2 % of the weight at eps = 1e-5.)
// Rows too long for registers have m0 + m1 from a binary64 sum.
#include "fp8q_ffn_plan.h"
#include "fp8q_mlp_launch.h"
#include "fp8q_rows.h"

namespace fp8q {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// x of another lane by DPP, which needs no LDS access as shuffles do; 0 in rows left out
template <int CTRL, int ROWS = 0xF> __device__ __forceinline__ float dpp(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS = 0xF> __device__ __forceinline__ double dpp(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ float last_lane(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}
__device__ __forceinline__ double last_lane(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// the sum over each 4, 8 or 16 consecutive lanes, in all of them
template <int LANES, typename T> __device__ __forceinline__ T part_sum(T v) {
    v += dpp<0xB1>(v);                                      // quad_perm [1,0,3,2]
    v += dpp<0x4E>(v);                                      // quad_perm [2,3,0,1]
    if constexpr (LANES >= 8) v += dpp<0x141>(v);           // row_half_mirror
    if constexpr (LANES >= 16) v += dpp<0x140>(v);          // row_mirror
    return v;
}
// the sum over a wave's lanes, in every lane
template <typename T> __device__ __forceinline__ T lane_sum(T v) {
    v = part_sum<16>(v);
    v += dpp<0x142, 0xA>(v);                                // row_bcast:15 into rows 1 and 3
    v += dpp<0x143, 0xC>(v);                                // row_bcast:31 into rows 2 and 3
    return last_lane(v);
}

// Sums of N values over the lanes of a row: one wave (NW = 0), or a workgroup of
// up to NW waves through lds, N x sum_words(NW) words of which those of waves that
// are not there are zero (clear_sums).  The words may be written again after the
// workgroup's next barrier.  Each lane reads one wave's sum and adds by DPP: a sum
// takes 4 additions, where all of them in every lane took 15, a tenth of the
// instructions of a row of 7168.
constexpr int sum_words(int nw) { return nw <= 4 ? 4 : nw <= 8 ? 8 : 16; }
template <int NW, int N, typename T> __device__ __forceinline__ void row_sums(T (&v)[N], T* lds) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_sum(v[i]);
    if constexpr (NW > 0) {
        constexpr int W = sum_words(NW);
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i * W + (threadIdx.x >> 6)] = v[i];
        lds_barrier();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = part_sum<W>(lds[i * W + (threadIdx.x & (W - 1))]);
    }
}
// before the first of them, by every thread
template <int WORDS, typename T> __device__ __forceinline__ void clear_sums(T* lds) {
    for (int i = (int)threadIdx.x; i < WORDS; i += (int)blockDim.x) lds[i] = T(0);
    __syncthreads();
}

// s / n from rn = 1 / n: exact where the quotient is a binary32 number, so that a
// constant row, whose d are equal and add up exactly, has y = b to the last bit (and
// zeros in a cast, whose scale would show whatever is left).  They add up exactly in
// rows held in registers: d is at most 2^6 units of h's last place there, of at most
// 2^15 columns.
__device__ __forceinline__ float mean_of(float s, float n, float rn) {
    const float q = s * rn;
    return __builtin_fmaf(__builtin_fmaf(-q, n, s), rn, q);
}

// m1 of a row held in registers, from the sum of d and q = mean(d^2): 0 where the
// deviation is over 4 |m0|.  There m0 is within a few of its own roundings (16-bit
// rows sum without any), while each d has one of the deviation's size, whose mean
// beside a small m0 would be all that shows: 4e-6 of it for 1 in 100 rows of 7168
// around zero, against 2e-7.  Squares under 2^-100 or past binary32 tell nothing.
__device__ __forceinline__ float second_mean(float s, float m0, float q, float n, float rn) {
    const float t = __builtin_fmaf(-16.0f * m0, m0, q);
    return t >= 0x1p-100f && t <= 3.4028234663852886e38f ? 0.0f : mean_of(s, n, rn);
}

// rstd from q = mean(d^2) and the mean of d (a NaN passes the clamp).  An infinite q
// stays infinite beside any finite m1 (whose square may be, and would leave NaN).
// The instruction is within 2^-23 and takes subnormal values as 0.
__device__ __forceinline__ float rstd_of(float q, float m1, float eps) {
    float v = __builtin_fmaf(-m1, m1, q);
    v = (v < 0.0f ? 0.0f : v) + eps;
    const bool tiny = v < 0x1p-100f;
    const float r = __builtin_amdgcn_rsqf(tiny ? v * 0x1p100f : v);
    return tiny ? r * 0x1p50f : r;
}

// y of one lane vector from d = h - m0
template <int VE> __device__ __forceinline__ void norm_y(float* d, float m1, float rs, const float* w, const float* b) {
#pragma unroll
    for (int k = 0; k < VE; ++k) d[k] = __builtin_fmaf((d[k] - m1) * rs, w[k], b[k]);
}

// VE weights from column c, kept as loaded; WF32: they are binary32 whatever
// the activations are
template <int DT, bool WF32> struct Affine {
    static constexpr bool kWide = WF32 && DT != kF32;
    v4u r[kWide ? 2 : 1];
    __device__ __forceinline__ void load(const void* w, int c) {
        const v4u_a2* p = (const v4u_a2*)((const char*)w + (int64_t)c * (kWide ? 4 : ESize<DT>::value));
#pragma unroll
        for (int i = 0; i < (kWide ? 2 : 1); ++i) r[i] = v4u{p[i].x, p[i].y, p[i].z, p[i].w};
    }
    __device__ __forceinline__ void clear() {
        for (v4u& x : r) x = v4u{0, 0, 0, 0};
    }
    // the asm keeps the compiler from widening once for all rows, which holds twice the registers
    __device__ __forceinline__ void widen(float* v) {
#pragma unroll
        for (int i = 0; i < (kWide ? 2 : 1); ++i) {
            asm volatile("" : "+v"(r[i]));
            widen16<kWide ? kF32 : DT>(r[i], v + 4 * i);
        }
    }
};

// Where a thread's lane vector v of a row stands: from column c, of which the
// first `dup` elements are another lane's.  The last vector of a row whose width
// is not whole vectors ends at the row's end instead of past it, and so repeats
// elements of the one before: they are computed again, to the same bits, stored
// twice and summed once, and no access has a partial path.  (Such paths, taken by
// one lane, held a mask for every element across the loop: 20 to 250 spilled
// registers.)  Vectors past the end are all `dup`, and are not stored.
template <int VE> struct Place {
    int c, dup;
    __device__ __forceinline__ Place(int at, int cols) {
        c = at + VE <= cols ? at : cols - VE;
        dup = min(at - c, VE);
    }
    __device__ __forceinline__ bool in() const { return dup < VE; }
};

template <int DT, bool NT> __device__ __forceinline__ v4u ld_at(const void* row, int c) {
    const v4u_a2* p = (const v4u_a2*)((const char*)row + (int64_t)c * ESize<DT>::value);
    const v4u_a2 t = NT ? __builtin_nontemporal_load(p) : *p;
    return v4u{t.x, t.y, t.z, t.w};
}
template <int DT, bool NT> __device__ __forceinline__ void st_at(void* row, int c, const float* y) {
    const v4u t = pack_out16<DT>(y);
    v4u_a2* d = (v4u_a2*)((char*)row + (int64_t)c * ESize<DT>::value);
    if constexpr (NT) __builtin_nontemporal_store(v4u_a2{t.x, t.y, t.z, t.w}, d);
    else *d = v4u_a2{t.x, t.y, t.z, t.w};
}

// One row per workgroup (or, WAVE, per wave) at a time, V lane vectors a
// thread.  A workgroup takes several rows, so that the next row's loads are in
// flight through the reductions and stores of this one, where V and the threads
// leave registers for that.  WHOLE: rows of whole 128-byte lines, streamed past
// the caches, and without a mask on every element (6 us more of 16384 x 7168 bf16
// with residual and group cast, which takes 146, 5.7 TB/s; 1999 x 5001 f32 16.1).
// A reduction's LDS words are written again after another
// reduction's barrier.
template <int DT, bool WF32, int FMT, int TO, bool WHOLE, bool WAVE, int V, int TB>
__global__ void __launch_bounds__(TB, V == 1 ? 8 : 4) k_ln_rows(LayerNorm a) {
    constexpr bool PF = V == 1 || (V == 2 && TB <= 768), NT = WHOLE;
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    constexpr int NW = WAVE ? 0 : TB / 64, SW = NW ? sum_words(NW) : 1;
    __shared__ float lds_s[3 * SW];
    __shared__ uint32_t lds_m[16];
    const int cols = (int)a.cols;
    const float fc = (float)cols, rn = 1.0f / fc;
    const int lanes = WAVE ? 64 : (int)blockDim.x;
    const int t = WAVE ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
    const int per = WAVE ? (int)blockDim.x >> 6 : 1;        // rows a workgroup takes at once
    const int64_t first = (int64_t)blockIdx.x * per + (WAVE ? threadIdx.x >> 6 : 0), next = (int64_t)gridDim.x * per;
    if (first >= a.rows) return;                            // whole waves; whole workgroups unless WAVE
    auto place = [&](int v) { return Place<VE>((v * lanes + t) * VE, cols); };
    v4u xv[V], rv[V];
    auto load = [&](int64_t row) {
        const int64_t off = row * a.cols * ES;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = place(v).c;
            xv[v] = ld_at<DT, NT>((const char*)a.x + off, c);
            if (a.res) rv[v] = ld_at<DT, NT>((const char*)a.res + off, c);
        }
    };
    load(first);
    if (NW) clear_sums<3 * SW>(lds_s);
    // one vector's weights stay in registers; two and four vectors leave none for theirs
    // beside the next row's loads (or spill already), and load them again for every row
    constexpr bool HOLD = V <= 1;
    Affine<DT, WF32> w[V], b[V];
    auto load_wb = [&](int v) {
        w[v].load(a.w, place(v).c);
        if (a.b) b[v].load(a.b, place(v).c);
        else b[v].clear();
    };
    if (HOLD)
#pragma unroll
        for (int v = 0; v < V; ++v) load_wb(v);
    for (int64_t row = first; row < a.rows; row += next) {
        float h[V][VE];
        float s[1] = {0.0f};
        // the asm keeps the compiler from holding a mask for every element across the rows
        int dup[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dup[v] = place(v).dup;
            asm volatile("" : "+v"(dup[v]));
            sum_h<DT>(xv[v], rv[v], a.res != nullptr, h[v]);
            float p = 0.0f;
#pragma unroll
            for (int k = 0; k < VE; ++k) p += WHOLE || k >= dup[v] ? h[v][k] : 0.0f;
            s[0] += WHOLE && dup[v] ? 0.0f : p;
        }
        if (PF && row + next < a.rows) load(row + next);
        row_sums<NW>(s, lds_s);
        const float m0 = s[0] * rn;
        if (a.h) {
            void* hr = (char*)a.h + row * a.cols * ES;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (place(v).in()) st_at<DT, NT>(hr, place(v).c, h[v]);
        }
        float d2[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float p = 0.0f, q = 0.0f;
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                h[v][k] -= m0;
                const float d = WHOLE || k >= dup[v] ? h[v][k] : 0.0f;
                p += d;
                q = __builtin_fmaf(d, d, q);
            }
            d2[0] += WHOLE && dup[v] ? 0.0f : p;
            d2[1] += WHOLE && dup[v] ? 0.0f : q;
        }
        row_sums<NW>(d2, lds_s + SW);
        const float ms = d2[1] * rn, m1 = second_mean(d2[0], m0, ms, fc, rn), rs = rstd_of(ms, m1, a.eps);
        if (t == 0) {
            if (a.mean) a.mean[row] = m0 + m1;
            if (a.rstd) a.rstd[row] = rs;
        }
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float wv[VE], bv[VE];
            if (!HOLD) load_wb(v);
            w[v].widen(wv);
            b[v].widen(bv);
            norm_y<VE>(h[v], m1, rs, wv, bv);
            if constexpr (TO == kToRow)                     // elements seen twice change no maximum
#pragma unroll
                for (int k = 0; k < VE; ++k) m = umax(m, __float_as_uint(h[v][k]) & 0x7FFFFFFFu);
            if (!HOLD) __builtin_amdgcn_sched_barrier(0);   // no registers for several vectors' weights at once
        }
        float scale = 0.0f;
        bool satur = false;
        if constexpr (TO == kToRow) scale = row_scale<FMT>(row_max<WAVE>(m, lds_m), a.sinv + row, t == 0, &satur);
        uint8_t* yr = (uint8_t*)a.y + row * a.cols * (TO == kToPlain ? ES : 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Place<VE> p = place(v);
            if constexpr (TO == kToPlain) {
                if (p.in()) st_at<DT, NT>(yr, p.c, h[v]);
            } else if constexpr (TO == kToGroup) {
                // whole vectors; the lanes of a group stay together for its maximum
                cast_vec<DT, FMT, true>(h[v], (v * lanes + t) * VE, cols, yr, a.sinv + row * (cols >> 7), 0.0f, false);
            } else if (p.in()) {
                float q[VE];
#pragma unroll
                for (int k = 0; k < VE; ++k) q[k] = satur ? sat<FMT>(h[v][k] * scale) : h[v][k] * scale;
                st_codes<FMT, VE, false>(yr, p.c, p.c + VE, q);
            }
        }
        if (!PF && row + next < a.rows) load(row + next);
    }
}

// one lane vector's part of the long rows' outputs
template <int DT, int FMT, int TO>
__device__ __forceinline__ void put_y(const LayerNorm& a, int64_t row, int c, const float* y, float scale, bool satur) {
    if constexpr (TO == kToPlain) {
        if (c < (int)a.cols) st_row<DT, false>((char*)a.y + row * a.cols * ESize<DT>::value, c, (int)a.cols, y);
    } else {
        cast_vec<DT, FMT, TO == kToGroup>(y, c, (int)a.cols, (uint8_t*)a.y + row * a.cols,
                                          TO == kToGroup ? a.sinv + row * (a.cols >> 7) : nullptr, scale, satur);
    }
}

// Rows too long for registers, or shorter than a vector: passes over the row, the later ones mostly from
// cache.  h and y are written in the last pass, after a lane's own reads of the
// same columns, so that they may be x or the residual itself.  The mean is a
// binary64 sum's, in the two halves m0 + m1: of a constant row of so many columns
// the differences from a binary32 m0 need not add up exactly (they did not in a
// quarter of such rows of 10^6, and a cast without a bias scales what is left to
// full range).  It costs 2 to 7 % where the row's reductions are the time (20000 x 5
// bf16 320 us against 312, 1 x 40960 9.8 / 9.2) and nothing where the bytes are
// (512 x 40960 with residual 56.9 / 56.8).
template <int DT, bool WF32, int FMT, int TO> __global__ void __launch_bounds__(1024) k_ln_long(LayerNorm a) {
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    __shared__ double lds_s[16];
    __shared__ float lds_q[16];
    __shared__ uint32_t lds_m[16];
    clear_sums<16>(lds_s);
    clear_sums<16>(lds_q);
    const int cols = (int)a.cols, step = (int)blockDim.x * VE, c0 = (int)threadIdx.x * VE;
    const double rn64 = 1.0 / (double)cols;
    const float rn = (float)rn64;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t off = row * a.cols * ES;
        const void* xr = (const char*)a.x + off;
        const void* rr = a.res ? (const char*)a.res + off : nullptr;
        double s[1] = {0.0};
        for (int64_t c = c0; c < cols; c += step) {
            float h[VE];
            load_h<DT>(xr, rr, (int)c, cols, h);
            double p = 0.0;
#pragma unroll
            for (int k = 0; k < VE; k += 2) p += (double)h[k] + (double)h[k + 1];
            s[0] += p;
        }
        row_sums<16>(s, lds_s);
        const double mean = s[0] * rn64;
        const float m0 = (float)mean, m1 = (float)(mean - (double)m0);
        // d of the columns from c on, zero past the row's end
        auto diff = [&](int64_t c, float* d) {
            load_h<DT>(xr, rr, (int)c, cols, d);
#pragma unroll
            for (int k = 0; k < VE; ++k) d[k] = c + k < cols ? d[k] - m0 : 0.0f;
        };
        float d2[1] = {0.0f};
        for (int64_t c = c0; c < cols; c += step) {
            float d[VE];
            diff(c, d);
#pragma unroll
            for (int k = 0; k < VE; ++k) d2[0] = __builtin_fmaf(d[k], d[k], d2[0]);
        }
        row_sums<16>(d2, lds_q);
        const float rs = rstd_of(d2[0] * rn, m1, a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = m0 + m1;
            if (a.rstd) a.rstd[row] = rs;
        }
        auto affine = [&](int64_t c, float* d) {
            float w[VE], b[VE];
            ld_weight<DT, WF32>(a.w, (int)c, cols, w);
            ld_weight<DT, WF32>(a.b ? a.b : a.w, (int)c, a.b ? cols : 0, b);
            norm_y<VE>(d, m1, rs, w, b);
        };
        float scale = 0.0f;
        bool satur = false;
        if constexpr (TO == kToRow) {
            uint32_t m = 0;
            for (int64_t c = c0; c < cols; c += step) {
                float d[VE];
                diff(c, d);
                affine(c, d);
#pragma unroll
                for (int k = 0; k < VE; ++k) m = umax(m, c + k < cols ? __float_as_uint(d[k]) & 0x7FFFFFFFu : 0u);
            }
            scale = row_scale<FMT>(row_max<false>(m, lds_m), a.sinv + row, threadIdx.x == 0, &satur);
        }
        void* hr = a.h ? (char*)a.h + off : nullptr;
        const int64_t end = ((int64_t)cols + step - 1) / step * step;      // whole waves stay in the group max
        for (int64_t cc = c0; cc < end; cc += step) {
            const int c = (int)(cc < cols ? cc : cols);
            float d[VE];
            load_h<DT>(xr, rr, c, cols, d);
            if (hr && c < cols) st_row<DT>(hr, c, cols, d);
#pragma unroll
            for (int k = 0; k < VE; ++k) d[k] -= m0;
            affine(c, d);
            put_y<DT, FMT, TO>(a, row, c, d, scale, satur);
        }
        __syncthreads();                                    // the first reduction's LDS is used again
    }
}

// ---------------------------------------------------------------------------
// backward: n = (h - mean) rstd, dn = dy w,
// dx = (dn - mean(dn) - n mean(dn n)) rstd + dh, and over the rows
// dweight = sum dy n, dbias = sum dy.  Each workgroup takes every G-th row and
// keeps its columns' sums in registers; the G partial rows are summed in order
// by a second kernel, so the result does not depend on timing.
// ---------------------------------------------------------------------------

struct LnBwdArgs {
    LayerNormBwd f;
    float* pw;             // [gridDim.x][cols] partial dweight, or nullptr
    float* pb;             // the same of dbias
};

// dy and h stay as loaded and are widened again after the reduction, and the
// sums over the rows live in LDS, in words that one thread alone touches: that
// leaves the registers for the next row's loads.  (Sums in registers spilled 30
// of them: 8192 x 7168 bf16 with dh 148 us; 100 us so, of which 7 are the column
// sums; 104 with one vector a thread and twice the threads.)
template <int DT, bool WF32, int V, int TB> __global__ void __launch_bounds__(TB, 4) k_ln_bwd(LnBwdArgs g) {
    const LayerNormBwd& a = g.f;
    constexpr bool PF = TB <= 512;
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value, Q = VE / 4;
    extern __shared__ v4f sums[];                           // [2][V][Q][T]: 4 columns each of dweight, then of dbias
    constexpr int NW = TB / 64, SW = sum_words(NW);
    __shared__ float lds[2][2 * SW];
    const int T = (int)blockDim.x, t = (int)threadIdx.x, cols = (int)a.cols;
    const float rn = 1.0f / (float)cols;
    auto place = [&](int v) { return Place<VE>((v * T + t) * VE, cols); };
    auto sum = [&](int which, int v, int q) -> v4f& { return sums[((which * V + v) * Q + q) * T + t]; };
    Affine<DT, WF32> w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v].load(a.w, place(v).c);
#pragma unroll
        for (int q = 0; q < Q; ++q) sum(0, v, q) = sum(1, v, q) = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    int flip = 0;
    v4u dyr[V], hr[V], dyn[V], hn[V], dhr[V];
    float rs = 0.0f, mu = 0.0f, rsn = 0.0f, mun = 0.0f;
    auto load = [&](int64_t row) {
        const int64_t off = row * a.cols * ES;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dyn[v] = ld_at<DT, true>((const char*)a.dy + off, place(v).c);
            hn[v] = ld_at<DT, true>((const char*)a.h + off, place(v).c);
        }
        rsn = a.rstd[row];
        mun = a.mean[row];
    };
    // n and dy of one lane vector
    auto widen = [&](int v, float* n, float* dy) {
        asm volatile("" : "+v"(dyr[v]), "+v"(hr[v]));
        widen16<DT>(dyr[v], dy);
        widen16<DT>(hr[v], n);
#pragma unroll
        for (int k = 0; k < VE; ++k) n[k] = (n[k] - mu) * rs;
    };
    if ((int64_t)blockIdx.x < a.rows) load(blockIdx.x);
    clear_sums<4 * SW>(lds[0]);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const int64_t off = row * a.cols * ES;
        rs = rsn;
        mu = mun;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dyr[v] = dyn[v];
            hr[v] = hn[v];
        }
        if (a.dh)
#pragma unroll
            for (int v = 0; v < V; ++v) dhr[v] = ld_at<DT, true>((const char*)a.dh + off, place(v).c);
        if (PF && row + gridDim.x < a.rows) load(row + gridDim.x);   // in flight through the reduction and the stores
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float wv[VE], n[VE], dy[VE];
            int dup = place(v).dup;
            asm volatile("" : "+v"(dup));                   // no mask for every element held across the rows
            widen(v, n, dy);
            w[v].widen(wv);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (g.pw) {
                    v4f& p = sum(0, v, q);
                    v4f x = p;
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = __builtin_fmaf(dy[4 * q + k], n[4 * q + k], x[k]);
                    p = x;
                }
                if (g.pb) {
                    v4f& p = sum(1, v, q);
                    v4f x = p;
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] += dy[4 * q + k];
                    p = x;
                }
            }
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float dn = k >= dup ? dy[k] * wv[k] : 0.0f, nk = k >= dup ? n[k] : 0.0f;
                s[0] += dn;
                s[1] = __builtin_fmaf(dn, nk, s[1]);
            }
            __builtin_amdgcn_sched_barrier(0);              // one vector widened at a time
        }
        // dx over dh: elements that two lanes hold are loaded by both before either stores them
        // (dy and h have been used, so their loads are done)
        if (a.dx == a.dh)
#pragma unroll
            for (int v = 0; v < V; ++v) asm volatile("" : "+v"(dhr[v]));
        row_sums<NW>(s, lds[flip]);
        const float m1 = s[0] * rn, m2 = s[1] * rn;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float wv[VE], n[VE], dy[VE], o[VE];
            widen(v, n, dy);
            w[v].widen(wv);
#pragma unroll
            for (int k = 0; k < VE; ++k) o[k] = __builtin_fmaf(-n[k], m2, dy[k] * wv[k] - m1) * rs;
            if (a.dh) {
                float d[VE];
                widen16<DT>(dhr[v], d);
#pragma unroll
                for (int k = 0; k < VE; ++k) o[k] += d[k];
            }
            if (place(v).in()) st_at<DT, true>((char*)a.dx + off, place(v).c, o);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!PF && row + gridDim.x < a.rows) load(row + gridDim.x);
    }
    for (int which = 0; which < 2; ++which) {
        float* p = which ? g.pb : g.pw;
        if (!p) continue;
        p += (int64_t)blockIdx.x * a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const v4f x = sum(which, v, q);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (4 * q + k >= place(v).dup) p[place(v).c + 4 * q + k] = x[k];
            }
    }
}

// Rows too long for registers, or shorter than a vector: the row is read twice, and the sums over the
// rows live in the workgroup's own partial rows (zeroed first; each word is
// touched by one thread only).
template <int DT, bool WF32> __global__ void __launch_bounds__(1024) k_ln_bwd_long(LnBwdArgs g) {
    const LayerNormBwd& a = g.f;
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    __shared__ float lds[2][32];
    clear_sums<64>(lds[0]);
    const int cols = (int)a.cols, step = (int)blockDim.x * VE, c0 = (int)threadIdx.x * VE;
    const float rn = 1.0f / (float)cols;
    float* pw = g.pw ? g.pw + (int64_t)blockIdx.x * a.cols : nullptr;
    float* pb = g.pb ? g.pb + (int64_t)blockIdx.x * a.cols : nullptr;
    for (float* p : {pw, pb})
        if (p)
            for (int64_t c = c0; c < cols; c += step)
                for (int k = 0; k < VE; ++k)
                    if (c + k < cols) p[c + k] = 0.0f;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const int64_t off = row * a.cols * ES;
        const float rs = a.rstd[row], mu = a.mean[row];
        // dy, w and n of the columns from c on (dy and w zero past the row's end)
        auto load = [&](int64_t c, float* dy, float* w, float* n) {
            widen16<DT>(ld_row<DT>((const char*)a.dy + off, (int)c, cols), dy);
            widen16<DT>(ld_row<DT>((const char*)a.h + off, (int)c, cols), n);
            ld_weight<DT, WF32>(a.w, (int)c, cols, w);
#pragma unroll
            for (int k = 0; k < VE; ++k) n[k] = (n[k] - mu) * rs;
        };
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = c0; c < cols; c += step) {
            float dy[VE], w[VE], n[VE];
            load(c, dy, w, n);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                s[0] += dy[k] * w[k];
                s[1] = __builtin_fmaf(dy[k] * w[k], n[k], s[1]);
                if (pw && c + k < cols) pw[c + k] = __builtin_fmaf(dy[k], n[k], pw[c + k]);
                if (pb && c + k < cols) pb[c + k] += dy[k];
            }
        }
        row_sums<16>(s, lds[flip]);
        const float m1 = s[0] * rn, m2 = s[1] * rn;
        for (int64_t c = c0; c < cols; c += step) {
            float dy[VE], w[VE], n[VE], o[VE];
            load(c, dy, w, n);
#pragma unroll
            for (int k = 0; k < VE; ++k) o[k] = __builtin_fmaf(-n[k], m2, dy[k] * w[k] - m1) * rs;
            if (a.dh) {
                float d[VE];
                widen16<DT>(ld_row<DT>((const char*)a.dh + off, (int)c, cols), d);
#pragma unroll
                for (int k = 0; k < VE; ++k) o[k] += d[k];
            }
            st_row<DT>((char*)a.dx + off, (int)c, cols, o);
        }
    }
}

// out[c] = sum of part[0 .. parts)[c] in a fixed order: 32 columns a workgroup
// at a time, 32 row lanes, then a tree over the row lanes in LDS.  y = 1: the
// second output, from the second half of the partial rows.
template <int DT> __global__ void __launch_bounds__(1024) k_column_sums(const float* part, int64_t parts, int64_t cols,
                                                                        void* out0, void* out1) {
    __shared__ float lds[32][33];
    const int cl = (int)threadIdx.x & 31, rl = (int)threadIdx.x >> 5;
    void* out = blockIdx.y ? out1 : out0;
    if (!out) return;
    if (blockIdx.y) part += parts * cols;
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < cols; c0 += (int64_t)gridDim.x * 32) {
        const int64_t c = c0 + cl;
        float s = 0.0f;
        if (c < cols)
#pragma unroll 8
            for (int64_t p = rl; p < parts; p += 32) s += part[p * cols + c];
        lds[rl][cl] = s;
        __syncthreads();
        for (int o = 16; o > 0; o >>= 1) {
            if (rl < o) lds[rl][cl] += lds[rl + o][cl];
            __syncthreads();
        }
        if (rl == 0 && c < cols) store1<DT>(out, c, lds[0][cl]);
    }
}

template <int DT, bool WF, int FMT, int TO, bool WHOLE> void ln_rows(const LayerNorm& a, const NormPlan& p, hipStream_t st) {
    const unsigned g = (unsigned)p.groups;
    const int T = p.threads;
    if (p.wave && p.V == 1) k_ln_rows<DT, WF, FMT, TO, WHOLE, true, 1, 256><<<g, T, 0, st>>>(a);
    else if (p.wave) k_ln_rows<DT, WF, FMT, TO, WHOLE, true, 2, 256><<<g, T, 0, st>>>(a);
    else if (p.V == 1 && T <= 256) k_ln_rows<DT, WF, FMT, TO, WHOLE, false, 1, 256><<<g, T, 0, st>>>(a);
    else if (p.V == 1) k_ln_rows<DT, WF, FMT, TO, WHOLE, false, 1, 1024><<<g, T, 0, st>>>(a);
    else if (p.V == 2 && T <= 768) k_ln_rows<DT, WF, FMT, TO, WHOLE, false, 2, 768><<<g, T, 0, st>>>(a);
    else if (p.V == 2) k_ln_rows<DT, WF, FMT, TO, WHOLE, false, 2, 1024><<<g, T, 0, st>>>(a);
    else k_ln_rows<DT, WF, FMT, TO, WHOLE, false, 4, 1024><<<g, T, 0, st>>>(a);
}

template <int DT, bool WF> void ln_to(const LayerNorm& a, hipStream_t st) {
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    const NormPlan p = layernorm_plan(a.rows, (a.cols + VE - 1) / VE, a.cols < VE);
    const bool whole = a.cols * ES % 128 == 0;
    auto run = [&](auto F, auto TOc) {
        constexpr int FMT = decltype(F)::value ? kE5M2 : kE4M3, TO = decltype(TOc)::value;
        if (p.V == 0) k_ln_long<DT, WF, FMT, TO><<<(unsigned)p.groups, p.threads, 0, st>>>(a);
        else if (TO == kToGroup || whole) ln_rows<DT, WF, FMT, TO, true>(a, p, st);
        else if constexpr (TO != kToGroup) ln_rows<DT, WF, FMT, TO, false>(a, p, st);
    };
    if (a.to == kToPlain) return run(std::false_type{}, KC<kToPlain>{});
    with_bool(a.fmt == kE5M2, [&](auto F) {
        if (a.to == kToGroup) run(F, KC<kToGroup>{});
        else run(F, KC<kToRow>{});
    });
}

template <int DT, bool WF> void ln_bwd(const LnBwdArgs& a, hipStream_t st) {
    constexpr int VE = LaneVE<DT>::value;
    const NormPlan p = norm_bwd_plan(a.f.rows, (a.f.cols + VE - 1) / VE);
    const unsigned g = (unsigned)p.groups;
    const int T = p.threads;
    const unsigned lds = (unsigned)(2 * p.V * VE * T * 4);  // the sums: at most 128 KB
    if (p.V == 0 || a.f.cols < VE) k_ln_bwd_long<DT, WF><<<g, T, 0, st>>>(a);
    else if (p.V == 1) k_ln_bwd<DT, WF, 1, 256><<<g, T, lds, st>>>(a);
    else if (T <= 512) k_ln_bwd<DT, WF, 2, 512><<<g, T, lds, st>>>(a);
    else k_ln_bwd<DT, WF, 2, 1024><<<g, T, lds, st>>>(a);
}

// go(DT, WF32) over the types of the activations and of the weight
template <typename F> void with_types(int dt, int wdt, F&& go) {
    if (dt == kF32) go(KC<kF32>{}, std::false_type{});
    else if (dt == kBF16) with_bool(wdt == kF32, [&](auto W) { go(KC<kBF16>{}, W); });
    else with_bool(wdt == kF32, [&](auto W) { go(KC<kF16>{}, W); });
}

}  // namespace

void launch_layernorm(const LayerNorm& a, hipStream_t st) {
    with_types(a.dt, a.wdt, [&](auto DT, auto W) { ln_to<decltype(DT)::value, decltype(W)::value>(a, st); });
}

int64_t layernorm_bwd_parts(int64_t rows) { return norm_bwd_parts(rows); }

void launch_column_sums(const float* part, int64_t parts, int64_t cols, void* out0, void* out1, int dt, hipStream_t st) {
    const dim3 g(grid((cols + 31) / 32), out1 ? 2 : 1);     // 1024 threads each: a grid holds fewer than 2^32
    if (dt == kF32) k_column_sums<kF32><<<g, 1024, 0, st>>>(part, parts, cols, out0, out1);
    else if (dt == kBF16) k_column_sums<kBF16><<<g, 1024, 0, st>>>(part, parts, cols, out0, out1);
    else k_column_sums<kF16><<<g, 1024, 0, st>>>(part, parts, cols, out0, out1);
}

void launch_layernorm_bwd(const LayerNormBwd& f, hipStream_t st) {
    const int64_t parts = layernorm_bwd_parts(f.rows);
    const LnBwdArgs a{f, f.dw ? f.ws : nullptr, f.db ? f.ws + parts * f.cols : nullptr};
    with_types(f.dt, f.wdt, [&](auto DT, auto W) { ln_bwd<decltype(DT)::value, decltype(W)::value>(a, st); });
    if (f.dw || f.db) launch_column_sums(f.ws, parts, f.cols, f.dw, f.db, f.wdt, st);
}

}  // namespace fp8q
