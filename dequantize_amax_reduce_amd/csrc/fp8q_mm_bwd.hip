// fp8q_mm_bwd.hip -- the backward products of the projections.
//
//   dg = dp u act'(g), du = dp act(g)         (a projection: dg = dy, with an
//                                              activation dg = dy act'(z), dbias = sum_m dg)
//   dx = [dg | du] [Wg ; Wu]                  contraction over the columns
//   [dWg ; dWu] = [dg | du]^T X               contraction over the rows
//
// Both products run on one 16-bit MFMA kernel (k_mm16) whose operands are
// contiguous in the contraction, so the operands are laid out first: dz =
// [dg | du] and its transpose, the transposed dequantized W, and the transposed
// dequantized X, in one launch (k_prep) after the two that find their exponents
// (k_scales, k_keys).  It moves 8-10 bytes per element of the operands; the
// products then run without a transposing read.  Gated, 4096 x 7168 -> 18432:
// 122 us for the exponents, 389 for the layout, 1774 and 1723 for the products.
// Contractions are padded with zeros to 64 elements (128 with a rest, below).
//
// Operands are rounded to f16 (11 bits), each once, below powers of two that
// the epilogue takes off the sums again:
//
//   X[m, k] = sx[m] X'[m, k],   W[n, k] = sw[n/128] W'[n, k],
//   dx = (dz sw) W',            dW = (dz sx)^T X',
//
// where sx[m] is the largest scale of row m of X and sw that of a block row of
// W, so that X' and W' are the codes themselves, exactly, where that scale is
// theirs (of a projection its power of two: a 16-bit dy times that is exact in
// f16, so that one operand alone is rounded).  The gradient's operand then has
// one exponent a row for dx (a row of dx depends on its own row of dz alone) and
// one a column for dW; X' and W' have one per 128 columns of K.  So what a row
// or column holds does not reach the others, a row of X or W that meets no
// gradient costs nothing whatever its scale, and no gradient needs scaling:
// every value down to 2^-28 of the largest that it is added to keeps 11 bits.
// bf16 operands, the simpler choice at the same MFMA rate, gave 2.4e-3 where f16
// results allow 2.1e-4, and 2.9e-3 where bf16 results allow 1.7e-3.
//
// An f16 gradient keeps as many bits as an operand, so each operand's rounding
// shows: of a dz that is computed, both (3.6e-4 of a gated pair; a projection's f16
// dy is exact as it is).  There dz has a rest beside it, dz - f16(dz) as e5m2, and
// the contraction starts with the rest's products by X' or W' as e5m2, on the
// fp8 instruction at twice the rate: 2.4e-4 to 2.8e-4, for half the products'
// time more (4096 x 7168 -> 18432: 2644 and 2565 us).
#include "fp8q_ffn_plan.h"
#include "fp8q_host.h"
#include "fp8q_mlp_launch.h"
#include "fp8q_mm.h"

namespace fp8q {

namespace {

struct Mm16Args {
    const void* a;         // [M, K] f16, each row after its rest where there is one (K e5m2)
    const void* b;         // [N, K] f16, likewise
    int64_t M;
    int N, KB, K8;         // steps of 128 bytes a row, of which K8 are of the rest
    uint32_t tm, tn;
    void* c0;              // rows [0, split): c0, pitch N
    void* c1;              // rows [gap, M): c1[row - gap]
    int64_t split, gap;
    int cdt, vec;
    const uint32_t* ka;    // the key of each row of a
    const uint32_t* kb;    // of 128 rows of b (columns of c) each,
    int qb;                // whose values are codes below 2^qb times what the key bounds
    int kper, splits;      // steps a split takes
    float* part;           // [splits][M][N] sums as they are, where splits > 1
};

// what dz is made of: dy itself, a gated pair's, or dy and one activation's slope
enum { kOfLinear = 0, kOfGated = 1, kOfUnary = 2 };
constexpr bool has_rest(int dt, int mode) { return mode != kOfLinear && dt == kF16; }

// Keys hold exponents in a form that an unsigned max folds: a finite nonzero
// binary32 v has a key k > 0 with |v| < 2^(k - kKeyBias - 126), 0 stands for
// none.  `shift`: the key of v 2^shift.
constexpr int kKeyBias = 1024;
__device__ __forceinline__ uint32_t finite_bits(float v) {   // |v|, 0 for NaN and infinity
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t key_of(uint32_t finite, int shift) {
    return finite ? (finite >> 23) + (uint32_t)(shift + kKeyBias) : 0u;
}
// a top scale as m 2^e, m in [0.5, 1): a product by m cannot overflow
__device__ __forceinline__ float mant_of(float top) { return __builtin_amdgcn_frexp_mantf(top); }
__device__ __forceinline__ int exponent_of(float top) { return __builtin_amdgcn_frexp_expf(top); }
// s / top, exactly 1 for the top itself
__device__ __forceinline__ float ratio_to(float s, float top) { return ldexpf(s, -exponent_of(top)) / mant_of(top); }
// the exponent that brings codes below 2^q times what the key bounds under 2^15
__device__ __forceinline__ int exp_of(uint32_t key, int q) { return key ? 141 + kKeyBias - q - (int)key : 0; }

// The rest of an f16 operand below 2^15 is at most 2^3; times 2^11 it has e5m2's
// range for itself.
constexpr float kRestScale = 2048.0f;

// row of c0 or c1 that row `row` of the product is, or none (padding)
__device__ __forceinline__ bool out_row(const Mm16Args& a, int64_t row, void** c, int64_t* r) {
    if (row < a.split) {
        *c = a.c0;
        *r = row;
        return true;
    }
    *c = a.c1;
    *r = row - a.gap;
    return row >= a.gap && row < a.M;
}

template <int BM, bool PART, bool REST>
__device__ __forceinline__ void mm16_tile(const Mm16Args& a, char* smem, uint32_t im, uint32_t in) {
    constexpr int MT = BM / 32, kStage = (BM + kMmBN) * 128;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int64_t m0 = (int64_t)im * BM;
    const int n0 = (int)in * 256;
    TileLoad<BM> ld;
    ld.init(a.a, m0, a.M, a.b, a.b, n0, n0 + 128, a.N, a.N, (int64_t)a.KB * 128, wave, lane);
    const uint32_t lds0 = lds_offset(smem);

    v4f acc[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[t][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int col = lane & 15, lr = lane >> 4;
    const uint32_t c0 = (uint32_t)((lr ^ (col & 7)) * 16), c1 = (uint32_t)(((lr + 4) ^ (col & 7)) * 16);
    const uint32_t ra = (uint32_t)((wm * (BM / 2) + col) * 128), rb = (uint32_t)((BM + wn * 32 + col) * 128);

    // Two halves of 32 elements a step, each half's fragments read while the
    // other half's MFMAs run.  The barrier sits between the halves: by then a
    // step's fragments are all in registers, so its buffer takes the tiles of
    // the step after next, which have a whole step to arrive.
    struct Half {
        v4i b[4], x[MT];
    } f0, f1;
    auto read = [&](Half& f, const char* s, uint32_t c) {
#pragma unroll
        for (int n = 0; n < 4; ++n) f.b[n] = *(const v4i*)(s + rb + (n >> 1) * (128 * 128) + (n & 1) * (16 * 128) + c);
#pragma unroll
        for (int t = 0; t < MT; ++t) f.x[t] = *(const v4i*)(s + ra + t * (16 * 128) + c);
    };
    auto mul = [&](const Half& f) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < 4; ++n) acc[t][n] = mfma_f16(f.b[n], f.x[t], acc[t][n]);
    };
    const int kb0 = PART ? (int)blockIdx.y * a.kper : 0, kb1 = PART ? min(a.KB, kb0 + a.kper) : a.KB;
    // 128 elements of the rest: both halves are one fragment of the fp8 instruction
    auto step8 = [&](int kb) {
        const int cur = (kb - kb0) & 1;
        read(f1, smem + cur * kStage, c1);
        dma_wait<0>();
        wg_barrier();
        if (kb < kb1 - 2) ld.issue(lds0 + cur * kStage, kb + 2);
        auto join = [](v4i p, v4i q) { return v8i{p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}; };
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                acc[t][n] = mfma_fp8<kE5M2, kE5M2>(join(f0.b[n], f1.b[n]), join(f0.x[t], f1.x[t]), acc[t][n]);
        __builtin_amdgcn_sched_barrier(0);
        if (kb < kb1 - 1) read(f0, smem + (cur ^ 1) * kStage, c0);
    };
    auto step = [&](int kb, auto NEXT, auto LOAD) {
        const int cur = (kb - kb0) & 1;
        const char* s = smem + cur * kStage;
        read(f1, s, c1);
        __builtin_amdgcn_sched_barrier(0);
        mul(f0);
        __builtin_amdgcn_sched_barrier(0);
        dma_wait<0>();
        wg_barrier();
        if constexpr (decltype(LOAD)::value) ld.issue(lds0 + cur * kStage, kb + 2);
        if constexpr (decltype(NEXT)::value) read(f0, smem + (cur ^ 1) * kStage, c0);
        __builtin_amdgcn_sched_barrier(0);
        mul(f1);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (kb0 < kb1) {
        ld.issue(lds0, kb0);
        dma_wait<0>();
        wg_barrier();
        if (kb1 - kb0 > 1) ld.issue(lds0 + kStage, kb0 + 1);
        read(f0, smem, c0);
        int kb = kb0;
        if constexpr (REST) {
            for (; kb < min(kb1, a.K8); ++kb) step8(kb);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int n = 0; n < 4; ++n) acc[t][n] *= 1.0f / kRestScale;
        }
        for (; kb < kb1 - 2; ++kb) step(kb, std::true_type{}, std::true_type{});
        if (kb < kb1 - 1) step(kb++, std::true_type{}, std::false_type{});
        if (!REST || kb < kb1) step(kb, std::false_type{}, std::false_type{});
    }
    const int nc = n0 + wn * 32 + lr * 8;
    const int last = (a.N - 1) >> 7;
    const int eb[2] = {exp_of(a.kb[min(n0 >> 7, last)], a.qb), exp_of(a.kb[min((n0 >> 7) + 1, last)], a.qb)};
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t row = m0 + wm * (BM / 2) + t * 16 + col;
        if constexpr (PART) {
            if (row >= a.M) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = acc[t][2 * half + (k >> 2)][k & 3];
                put8(a.part + (int64_t)blockIdx.y * a.M * a.N, kF32, row, a.N, nc + half * 128, a.N, true, v);
            }
            continue;
        }
        void* c;
        int64_t r;
        if (!out_row(a, row, &c, &r)) continue;
        const int ea = exp_of(a.ka[row], 0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = ldexpf(acc[t][2 * half + (k >> 2)][k & 3], -(ea + eb[half]));
            put8(c, a.cdt, r, a.N, nc + half * 128, a.N, a.vec, v);
        }
    }
}

template <int BM, bool PART, bool REST> __global__ void __launch_bounds__(kMmThreads, 2) k_mm16(Mm16Args a) {
    __shared__ __attribute__((aligned(1024))) char smem[2 * (BM + kMmBN) * 128];
    uint32_t im, in;
    tile_of(blockIdx.x, a.tm, a.tn, &im, &in);
    mm16_tile<BM, PART, REST>(a, smem, im, in);
}

// two whole products in one launch: the first's tiles, then the second's
template <int BM, bool REST> __global__ void __launch_bounds__(kMmThreads, 2) k_mm16_two(Mm16Args a, Mm16Args b) {
    __shared__ __attribute__((aligned(1024))) char smem[2 * (BM + kMmBN) * 128];
    const uint32_t first = a.tm * a.tn;
    const bool second = blockIdx.x >= first;
    Mm16Args g = a;
    if (second) g = b;
    uint32_t im, in;
    tile_of(second ? blockIdx.x - first : blockIdx.x, g.tm, g.tn, &im, &in);
    // (wave-uniform as they are; the compiler loses it across the choice)
    mm16_tile<BM, false, REST>(g, smem, __builtin_amdgcn_readfirstlane(im), __builtin_amdgcn_readfirstlane(in));
}

// the end of a split product: the partial sums in order; a thread takes 8
// columns (the columns are a multiple of 128)
__global__ void __launch_bounds__(256) k_mm16_join(Mm16Args a) {
    const int64_t per = a.N / 8, total = a.M * per, step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
        const int64_t row = i / per;
        const int n = (int)(i - row * per) * 8;
        void* c;
        int64_t r;
        if (!out_row(a, row, &c, &r)) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        const float* p = a.part + row * a.N + n;
        for (int s = 0; s < a.splits; ++s, p += a.M * a.N) {
            const v4f x = *(const v4f*)p, y = *(const v4f*)(p + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] += x[k];
                v[4 + k] += y[k];
            }
        }
        const int e = -(exp_of(a.ka[row], 0) + exp_of(a.kb[n >> 7], a.qb));
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = ldexpf(v[k], e);
        put8(c, a.cdt, r, a.N, n, a.N, a.vec, v);
    }
}

// ---------------------------------------------------------------------------
// operand layout
// ---------------------------------------------------------------------------

typedef unsigned int v4u_a2 __attribute__((ext_vector_type(4), aligned(2)));

// A 64 (rows) x 64 (columns) tile transposed through LDS as pairs of rows:
// word [c][i] holds column c of rows 2i and 2i + 1.  The pitch of 33 words
// spreads both the column-wise writes and the row-wise reads over the banks.
struct TileT {
    uint32_t w[64][33];
};

// the same of bytes: half word [c][i] holds column c of rows 2i and 2i + 1; rows
// of 80 bytes, so that 16 of them are read at once
struct TileT8 {
    uint16_t w[64][40];
};

// 8 elements from column c of a row (zero from column `cols` on); FULL: c + 8 <= cols
template <int DT, bool FULL> __device__ __forceinline__ void ld8(const uint16_t* row, int c, int cols, float* v) {
    HpVec<DT> t;
    if (FULL || c + 8 <= cols) {
        const v4u_a2 r = *(const v4u_a2*)(row + c);
        t.r = v4u{r.x, r.y, r.z, r.w};
    } else {
        union { v4u q; uint16_t e[8]; } u;
        u.q = v4u{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < cols) u.e[k] = row[c + k];
        t.r = u.q;
    }
    t.widen(v);
}

// this workgroup's 64 columns of t as rows of dst (pitch `pitch` bytes), 64
// elements each from byte `at`
__device__ __forceinline__ void store_t(const TileT& t, char* dst, int64_t pitch, int64_t at) {
    const int c = (int)threadIdx.x >> 2, q = (int)threadIdx.x & 3;
    char* d = dst + c * pitch + at + q * 32;
    const uint32_t* s = &t.w[c][q * 8];
    *(v4u*)d = v4u{s[0], s[1], s[2], s[3]};
    *(v4u*)(d + 16) = v4u{s[4], s[5], s[6], s[7]};
}
__device__ __forceinline__ void store_t(const TileT8& t, char* dst, int64_t pitch, int64_t at) {
    const int c = (int)threadIdx.x >> 2, q = (int)threadIdx.x & 3;
    *(v4u*)(dst + c * pitch + at + q * 16) = *(const v4u*)&t.w[c][q * 8];
}

// two f16 values as e5m2, rounded half up; infinities and NaN as 0 (the f16
// operand has them)
__device__ __forceinline__ uint16_t e5m2_pair(uint32_t h2) {
    const uint32_t a = h2 & 0xFFFFu, b = h2 >> 16;
    const uint32_t p = (a & 0x7C00u) == 0x7C00u ? 0u : (a + 0x80u) >> 8, q = (b & 0x7C00u) == 0x7C00u ? 0u : (b + 0x80u) >> 8;
    return (uint16_t)(p | q << 8);
}
// what f16 leaves of v, times kRestScale (0 where v is not finite)
__device__ __forceinline__ float rest_of(float v, uint32_t half) {
    const float h = (float)__builtin_bit_cast(_Float16, (uint16_t)half);
    return finite_bits(h) == (__float_as_uint(h) & 0x7FFFFFFFu) ? (v - h) * kRestScale : 0.0f;
}

// ---------------------------------------------------------------------------
// exponents
// ---------------------------------------------------------------------------

// the largest finite scale of every row of X and block row of W (1 where there
// is none; where dz is dy itself, down to its power of two), and the keys cleared for
// k_keys; 16 lanes a row
struct ScaleArgs {
    const float* xs;       // [M, KB]
    int64_t M;
    const float* ws0;      // [nb, KB] each
    const float* ws1;      // or nullptr
    int nb, KB;
    float* sx;             // [M]
    float* sw;             // [ws1 ? 2 nb : nb]
    uint32_t* keys;
    int64_t nkeys;
    bool whole;            // as they are; else their powers of two
};
__global__ void __launch_bounds__(256) k_scales(ScaleArgs a) {
    const int64_t total = a.M + (a.ws1 ? 2 : 1) * (int64_t)a.nb;
    const int64_t first = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int l = (int)threadIdx.x & 15;
    for (int64_t row = first; row < total; row += (int64_t)gridDim.x * 16) {
        const float* s;
        if (row < a.M) s = a.xs + row * a.KB;
        else if (row < a.M + a.nb) s = a.ws0 + (row - a.M) * a.KB;
        else s = a.ws1 + (row - a.M - a.nb) * a.KB;
        uint32_t m = 0;
        for (int kb = l; kb < a.KB; kb += 16) m = umax(m, finite_bits(s[kb]));
        m = max_lanes<16>(m);
        if (!a.whole && m) m = umax(m & 0x7F800000u, 0x00800000u);
        if (l == 0) (row < a.M ? a.sx + row : a.sw + (row - a.M))[0] = m ? __uint_as_float(m) : 1.0f;
    }
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.nkeys; i += (int64_t)gridDim.x * 256) a.keys[i] = 0;
}

// 8 columns of dg (dz without a gate) and du from column c of row m < M;
// zero from column N on (FULL: there are none); QUICK as in act_at
template <int DT, int MODE, bool FULL, bool QUICK>
__device__ __forceinline__ void dz_values(const uint16_t* dy, const uint16_t* z, int64_t m, int c, int N, int act,
                                          float* g, float* u) {
    static_assert(MODE != kOfUnary || !QUICK, "the keys of one activation's dz come from bounds on its slope");
    ld8<DT, FULL>(dy + m * N, c, N, g);
    if constexpr (MODE == kOfUnary) {
        float zv[8];
        ld8<DT, FULL>(z + m * N, c, N, zv);
        with_slope(act, [&](auto A) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float d = unary_grad<decltype(A)::value>(g[k], zv[k]);
                g[k] = FULL || c + k < N ? d : 0.0f;
            }
        });
    }
    if constexpr (MODE == kOfGated) {
        float zg[8], zu[8];
        ld8<DT, FULL>(z + m * 2 * N, c, N, zg);
        ld8<DT, FULL>(z + m * 2 * N + N, c, N, zu);
        with_act(act, [&](auto A) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // the slope before u: where it is 0, no large dp * u comes first
                const Act r = act_at<decltype(A)::value, true, QUICK>(zg[k]);
                u[k] = FULL || c + k < N ? g[k] * r.a * r.e : 0.0f;
                g[k] = FULL || c + k < N ? g[k] * r.d * zu[k] * r.e : 0.0f;
            }
        });
    }
}

// The keys of dz's rows and columns, and of X' and W' per 128 columns of K.
// Of a dz that is dy times one activation's slope they come from dy's exponents and
// bounds on the slopes' (4096 x 18432 bf16 through GELU: 157 us with the slope
// itself, 94 with a binary32 bound on it, 81 with the integer one; each bound by its
// instructions, 32 an element in the second, 22 in the third.)
// Workgroups [0, e0) take 128 x 128 of dz, 16 lanes a row and 8 columns a lane;
// [e0, e1) 32 rows of X's scales, the rest as many block rows of W's.  The
// maxima of integers do not depend on the order of the atomics.  A key of dz is of
// |dz| 2^e, twice |dz sx| or |dz sw| at most.
struct KeyArgs {
    const uint16_t* dy;
    const uint16_t* z;
    int64_t M;
    int N, act;
    const float* sx;
    const float* sw;
    uint32_t* krow;        // [M], or nullptr
    uint32_t* kcol;        // [Np] of dg, then of du, or nullptr
    int Np;
    const float* xs;
    const float* ws0;
    const float* ws1;
    int nb, KB;
    uint32_t* kx;          // [KB]
    uint32_t* kw;
    uint32_t e0, e1, cols; // cols: tiles of dz in a row of them
};
// A workgroup takes few rows, with 8 loads in flight a thread, so that it does
// not end after dz's (3001 x 4096 f16: 11.2 us, 16.7 with 256 rows).
constexpr int kKeyRows = 32;
__device__ __forceinline__ void scale_keys(const float* s, const float* top, int64_t rows, int64_t r0, int KB, uint32_t* out,
                                           uint32_t* lds) {
    const int64_t last = (r0 + kKeyRows < rows ? r0 + kKeyRows : rows) - 1;
    const int per = KB < 256 ? 256 / KB : 1, rl = KB < 256 ? (int)threadIdx.x / KB : 0;
    lds[threadIdx.x] = 0;
    __syncthreads();
    for (int kb = KB < 256 ? (int)threadIdx.x % KB : (int)threadIdx.x; rl < per && kb < KB; kb += 256) {
        uint32_t m = 0;
        for (int64_t r = r0 + rl; r <= last; r += 8 * per) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {                   // rows past the last are the last one again
                const int64_t ri = r + i * per < last ? r + i * per : last;
                m = umax(m, key_of(finite_bits(ratio_to(s[ri * KB + kb], top[ri])), 0));
            }
        }
        if (KB < 256) atomicMax(lds + kb, m);               // LDS; a word of `out` takes 8 ns an atomic
        else if (m) atomicMax(out + kb, m);
    }
    __syncthreads();
    if ((int)threadIdx.x < KB && lds[threadIdx.x]) atomicMax(out + threadIdx.x, lds[threadIdx.x]);
}
template <int DT, int MODE> __global__ void __launch_bounds__(256) k_keys(KeyArgs a) {
    constexpr int H = MODE == kOfGated ? 2 : 1;
    __shared__ uint32_t lds[4][H][128];
    if (blockIdx.x >= a.e0) {
        int64_t i = blockIdx.x - a.e0;
        if (blockIdx.x < a.e1) return scale_keys(a.xs, a.sx, a.M, i * kKeyRows, a.KB, a.kx, lds[0][0]);
        i = blockIdx.x - a.e1;
        const int64_t per = (a.nb + kKeyRows - 1) / kKeyRows;
        if (i < per) scale_keys(a.ws0, a.sw, a.nb, i * kKeyRows, a.KB, a.kw, lds[0][0]);
        else scale_keys(a.ws1, a.sw + a.nb, a.nb, (i - per) * kKeyRows, a.KB, a.kw, lds[0][0]);
        return;
    }
    const int bx = (int)(blockIdx.x % a.cols), v = (int)threadIdx.x & 15, rl = (int)threadIdx.x >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / a.cols) * 128;
    const int c = bx * 128 + v * 8;
    int ew[H];
#pragma unroll
    for (int h = 0; h < H; ++h) ew[h] = exponent_of(a.sw[h * a.nb + bx]);   // 128 columns of dz: one block row of W
    uint32_t kc[H][8];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) kc[h][k] = 0;
    // Rows past the end are the last one again, which changes no maximum (but
    // atomics on one word take 8 ns each: only a row's own lanes make them).
    // The loads of R rows are in flight at once.
    auto rows = [&](auto FULL) {
        constexpr int R = MODE == kOfGated ? 2 : 4;
#pragma unroll 1
        for (int i = 0; i < 8; i += R) {
            float d[R][H][8];
            int64_t m[R];
            int ex[R];
            if constexpr (MODE == kOfUnary) {
                float z[R][8];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    m[r] = m0 + (i + r) * 16 + rl;
                    if (m[r] > a.M - 1) m[r] = a.M - 1;
                    ex[r] = exponent_of(a.sx[m[r]]);
                    ld8<DT, decltype(FULL)::value>(a.dy + m[r] * a.N, c, a.N, d[r][0]);
                    ld8<DT, decltype(FULL)::value>(a.z + m[r] * a.N, c, a.N, z[r]);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    // the keys of |dy| 2^e, none of zero and non-finite values (nor of those whose slope is 0)
                    int key[8], top = 0;
                    auto of = [&](int k, int e, bool ok) {
                        const uint32_t b = __float_as_uint(d[r][0][k]) & 0x7FFFFFFFu;
                        key[k] = ok && b - 1u < 0x7F7FFFFFu ? (int)(b >> 23) + e + kKeyBias : -(1 << 20);
                        top = max(top, key[k]);
                    };
                    if (a.act == kRelu)
#pragma unroll
                        for (int k = 0; k < 8; ++k) of(k, 0, !(z[r][k] <= 0.0f));
                    else
                        with_act(a.act, [&](auto A) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) of(k, slope_exponent<decltype(A)::value>(z[r][k]), true);
                        });
#pragma unroll
                    for (int k = 0; k < 8; ++k) kc[0][k] = (uint32_t)max((int)kc[0][k], key[k] + ex[r]);
                    const uint32_t kr = max_lanes<16>(top > 0 ? (uint32_t)max(top + ew[0], 0) : 0u);
                    if (v == 0 && a.krow && kr && m0 + (i + r) * 16 + rl < a.M) atomicMax(a.krow + m[r], kr);
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    m[r] = m0 + (i + r) * 16 + rl;
                    if (m[r] > a.M - 1) m[r] = a.M - 1;
                    ex[r] = exponent_of(a.sx[m[r]]);
                    dz_values<DT, MODE, decltype(FULL)::value, true>(a.dy, a.z, m[r], c, a.N, a.act, d[r][0], d[r][H - 1]);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    uint32_t kr = 0;
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        uint32_t top = 0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t b = finite_bits(d[r][h][k]);
                            top = umax(top, b);
                            kc[h][k] = umax(kc[h][k], key_of(b, ex[r]));
                        }
                        kr = umax(kr, key_of(top, ew[h]));
                    }
                    kr = max_lanes<16>(kr);
                    if (v == 0 && a.krow && kr && m0 + (i + r) * 16 + rl < a.M) atomicMax(a.krow + m[r], kr);
                }
            }
        }
    };
    if (bx * 128 + 128 <= a.N) rows(std::true_type{});
    else rows(std::false_type{});
    if (!a.kcol) return;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) {                       // the wave's four rows
            uint32_t m = kc[h][k];
            m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
            m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
            if ((rl & 3) == 0) lds[rl >> 2][h][v * 8 + k] = m;
        }
    __syncthreads();
    const int h = (int)threadIdx.x >> 7, cl = (int)threadIdx.x & 127;
    if (h < H && bx * 128 + cl < a.N) {
        const uint32_t m = umax(umax(lds[0][h][cl], lds[1][h][cl]), umax(lds[2][h][cl], lds[3][h][cl]));
        if (m) atomicMax(a.kcol + (int64_t)h * a.Np + bx * 128 + cl, m);
    }
}

struct DzArgs {
    const uint16_t* dy;
    const uint16_t* z;
    int64_t M, Mp;         // Mp: M padded to 64 (128 with REST)
    int N, Np;             // Np: N padded to 64
    int act;
    char* dz;              // [M, gated ? 2 Np : Np] f16, each row after its rest with REST; or nullptr
    char* dzt;             // [gated ? 2 Np : Np, Mp], likewise
    const float* sx;       // [M]
    const float* sw;       // [gated ? 2 nb : nb]
    int nb;
    const uint32_t* krow;  // [M]
    const uint32_t* kcol;  // [gated ? 2 Np : Np]
    float* bias;           // [Mp / 64][N] sums of 64 rows of dz each, or nullptr
};

// dz sw and the transpose of dz sx, each below its own exponents; 256
// threads, one 64 x 64 tile a workgroup; thread (i, v) takes 8 columns of the
// rows 2i and 2i + 1
template <int DT, int MODE, bool BIAS, bool REST>
__device__ __forceinline__ void dz_tile(const DzArgs& a, uint32_t bx, uint32_t by, TileT* lds, TileT8* lds8) {
    constexpr int H = MODE == kOfGated ? 2 : 1, E = REST ? 3 : 2;   // bytes an element takes of a row
    const int v = (int)threadIdx.x & 7, i = (int)threadIdx.x >> 3;
    const int64_t m = (int64_t)by * 64 + 2 * i;
    const int c = (int)bx * 64 + v * 8;
    const int64_t C = (int64_t)H * a.Np;
    float d[2][H][8];
    float sx[2] = {1.0f, 1.0f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (m + r >= a.M) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) d[r][h][k] = 0.0f;
            continue;
        }
        dz_values<DT, MODE, false, false>(a.dy, a.z, m + r, c, a.N, a.act, d[r][0], d[r][H - 1]);
        if (!BIAS || a.dzt) sx[r] = a.sx[m + r];
        if (a.dz) {
            const int e = exp_of(a.krow[m + r], 0);
            char* row = a.dz + (m + r) * C * E;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float sw = a.sw[h * a.nb + (bx >> 1)], f = mant_of(sw);
                const int s = e + exponent_of(sw);
                float t[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) t[k] = ldexpf(d[r][h][k] * f, s);
                const v4u o = pack_out16<kF16>(t);
                const int64_t at = (int64_t)h * a.Np + c;
                *(v4u*)(row + (E - 2) * C + 2 * at) = o;
                if constexpr (REST) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) t[k] = rest_of(t[k], o[k >> 1] >> (16 * (k & 1)));
                    *(v2u*)(row + at) = v2u{enc4<kE5M2>(t[0], t[1], t[2], t[3]), enc4<kE5M2>(t[4], t[5], t[6], t[7])};
                }
            }
        }
    }
    if constexpr (BIAS) {
        if (a.bias) {                                       // the wave's 16 rows, then the four waves
            float* sums = (float*)lds;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float s = d[0][0][k] + d[1][0][k];
                s += __shfl_xor(s, 8, 64);
                s += __shfl_xor(s, 16, 64);
                s += __shfl_xor(s, 32, 64);
                if ((i & 7) == 0) sums[(i >> 3) * 64 + v * 8 + k] = s;
            }
            __syncthreads();
            const int t = (int)threadIdx.x, col = (int)bx * 64 + t;
            if (t < 64 && col < a.N) a.bias[(int64_t)by * a.N + col] = (sums[t] + sums[64 + t]) + (sums[128 + t] + sums[192 + t]);
            __syncthreads();                                // the tiles are written there next
        }
    }
    if (!a.dzt) return;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int e = exp_of(a.kcol[(int64_t)h * a.Np + c + k], 0);
            const float p = ldexpf(d[0][h][k] * mant_of(sx[0]), e + exponent_of(sx[0]));
            const float q = ldexpf(d[1][h][k] * mant_of(sx[1]), e + exponent_of(sx[1]));
            const uint32_t o = pack_f16x2(p, q);
            lds[h].w[v * 8 + k][i] = o;
            if constexpr (REST)
                lds8[h].w[v * 8 + k][i] = (uint16_t)enc4<kE5M2>(rest_of(p, o & 0xFFFFu), rest_of(q, o >> 16), 0.0f, 0.0f);
        }
    __syncthreads();
    char* t = a.dzt + (int64_t)bx * 64 * a.Mp * E;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        char* th = t + (int64_t)h * a.Np * a.Mp * E;
        store_t(lds[h], th, a.Mp * E, (E - 2) * a.Mp + (int64_t)by * 128);
        if constexpr (REST) store_t(lds8[h], th, a.Mp * E, (int64_t)by * 64);
    }
}

struct DeqTArgs {
    const uint8_t* q;
    const float* s;        // s[(row >> sh) * KB + k / 128]
    int64_t R;             // rows
    int KB, sh;
    char* t;               // [K, C] f16 (each row after the e5m2 form with REST), this matrix from element `at` of a row
    int64_t C, at;
    const float* top;      // the top scale of row >> sh, which its scales are divided by
    const uint32_t* key;   // [KB]
    int qb;                // codes are below 2^qb
};

// The transposed dequantized matrix: 64 rows x 128 codes a workgroup; thread
// (i, v) takes 16 codes of the rows 2i and 2i + 1.  Rows past R are zero.
template <int FMT, bool REST>
__device__ __forceinline__ void deq_tile(const DeqTArgs& a, uint32_t bx, uint32_t by, TileT* t, TileT8* t8) {
    const int v = (int)threadIdx.x & 7, i = (int)threadIdx.x >> 3;
    const int64_t r0 = (int64_t)by * 64 + 2 * i;
    const int64_t K = (int64_t)a.KB * 128;
    const int ex = exp_of(a.key[bx], a.qb);
    float f[2][16];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (r0 + r < a.R) {
            const v4u c = *(const v4u*)(a.q + (r0 + r) * K + (int64_t)bx * 128 + v * 16);
            const float s = ldexpf(ratio_to(a.s[((r0 + r) >> a.sh) * a.KB + bx], a.top[(r0 + r) >> a.sh]), ex);
            dec4<FMT>(c.x, f[r]);
            dec4<FMT>(c.y, f[r] + 4);
            dec4<FMT>(c.z, f[r] + 8);
            dec4<FMT>(c.w, f[r] + 12);
#pragma unroll
            for (int k = 0; k < 16; ++k) f[r][k] *= s;
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) f[r][k] = 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint32_t o = pack_f16x2(f[0][k], f[1][k]);
        t[v >> 2].w[(v & 3) * 16 + k][i] = o;
        if constexpr (REST) t8[v >> 2].w[(v & 3) * 16 + k][i] = e5m2_pair(o);
    }
    __syncthreads();
    constexpr int E = REST ? 3 : 2;
    const int64_t at = a.at + (int64_t)by * 64;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        char* d = a.t + ((int64_t)bx * 128 + h * 64) * a.C * E;
        store_t(t[h], d, a.C * E, (E - 2) * a.C + 2 * at);
        if constexpr (REST) store_t(t8[h], d, a.C * E, at);
    }
}

// All of a call's layout passes in one launch: workgroups [0, e0) take tiles
// of dz, [e0, e1) of X, [e1, e2) of W (or the gate), the rest of the up
// projection.
struct PrepArgs {
    DzArgs dz;
    DeqTArgs x, w0, w1;
    uint32_t e0, e1, e2, dzx;
};
template <int DT, int MODE, bool BIAS, int XF, int WF> __global__ void __launch_bounds__(256) k_prep(PrepArgs a) {
    constexpr bool REST = has_rest(DT, MODE);
    __shared__ TileT lds[2];
    __shared__ __attribute__((aligned(16))) TileT8 lds8[REST ? 2 : 1];
    const uint32_t b = blockIdx.x;
    if (b < a.e0) {
        dz_tile<DT, MODE, BIAS, REST>(a.dz, b % a.dzx, b / a.dzx, lds, lds8);
    } else if (b < a.e1) {
        const uint32_t i = b - a.e0;
        deq_tile<XF, REST>(a.x, i % (uint32_t)a.x.KB, i / (uint32_t)a.x.KB, lds, lds8);
    } else if (b < a.e2) {
        const uint32_t i = b - a.e1;
        deq_tile<WF, REST>(a.w0, i % (uint32_t)a.w0.KB, i / (uint32_t)a.w0.KB, lds, lds8);
    } else {
        const uint32_t i = b - a.e2;
        deq_tile<WF, REST>(a.w1, i % (uint32_t)a.w1.KB, i / (uint32_t)a.w1.KB, lds, lds8);
    }
}

__global__ void __launch_bounds__(256) k_zero16(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}
void zero(void* p, int64_t n, int dt, hipStream_t st) {
    if (p && n > 0) launch_zero16(p, n * (dt == kF32 ? 2 : 1), st);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// c[m, n] = sum_k a[m, k] b[n, k]; rows [0, split) to c0, rows from gap to c1;
// N % 128 == 0; rest: each row's first K bytes are the rest; p: the plan of the
// product
Mm16Args mm16_args(const void* A, const void* B, int64_t M, int64_t N, int64_t K, bool rest, void* c0, void* c1,
                   int64_t split, int64_t gap, int cdt, const Plan16& p, const uint32_t* ka, const uint32_t* kb, int qb,
                   float* part) {
    const int K8 = rest ? (int)(K / 128) : 0;
    Mm16Args a{A, B, M, (int)N, (int)(K / 64) + K8, K8, 0, 0, c0, c1, split, gap, cdt, 0, ka, kb, qb, p.kper, p.splits, part};
    a.vec = al(c0, 16) && (!c1 || al(c1, 16));
    a.tn = (uint32_t)((N + 255) / 256);
    a.tm = (uint32_t)((M + p.bm - 1) / p.bm);
    return a;
}

template <typename F> void with_bool(bool b, F&& f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
}

// go(BM, REST)
template <typename F> void with_height(int bm, bool rest, F&& go) {
    with_bool(rest, [&](auto R) {
        if (bm == 256) go(KC<256>{}, R);
        else if (bm == 192) go(KC<192>{}, R);
        else if (bm == 128) go(KC<128>{}, R);
        else go(KC<64>{}, R);
    });
}

void mm16(const Mm16Args& a, int bm, bool rest, hipStream_t st) {
    const dim3 g(a.tm * a.tn, (unsigned)a.splits);
    with_height(bm, rest, [&](auto BMc, auto R) {
        constexpr int BM = decltype(BMc)::value;
        constexpr bool REST = decltype(R)::value;
        if (a.splits == 1) k_mm16<BM, false, REST><<<g, kMmThreads, 0, st>>>(a);
        else if constexpr (BM != 192) k_mm16<BM, true, REST><<<g, kMmThreads, 0, st>>>(a);   // 192 is never split
    });
    if (a.splits > 1)
        k_mm16_join<<<(unsigned)std::min<int64_t>((a.M * (a.N / 8) + 255) / 256, 4096), 256, 0, st>>>(a);
}

// both, the longer tiles first
void mm16_two(const Mm16Args& a, const Mm16Args& b, int bm, bool rest, hipStream_t st) {
    if (a.KB < b.KB) return mm16_two(b, a, bm, rest, st);
    const unsigned g = a.tm * a.tn + b.tm * b.tn;
    with_height(bm, rest, [&](auto BMc, auto R) {
        constexpr int BM = decltype(BMc)::value;
        if constexpr (BM != 64) k_mm16_two<BM, decltype(R)::value><<<g, kMmThreads, 0, st>>>(a, b);
    });
}

template <typename F> void with_fmt(int f, F&& go) {
    if (f == kE4M3) go(KC<kE4M3>{});
    else go(KC<kE5M2>{});
}

// go(DT, MODE)
template <typename F> void with_dt(int dt, int mode, F&& go) {
    auto of = [&](auto DT) {
        if (mode == kOfLinear) go(DT, KC<kOfLinear>{});
        else if (mode == kOfGated) go(DT, KC<kOfGated>{});
        else go(DT, KC<kOfUnary>{});
    };
    if (dt == kBF16) of(KC<kBF16>{});
    else of(KC<kF16>{});
}

struct BwdLayout {
    int64_t Mp, Np, C;     // padded rows and columns; C: columns of dz
    int64_t dz, dzt, wt, xt;
    int64_t sx, sw;        // top scales of the rows of X and of the block rows of W
    int64_t krow, kcol, kx, kw, nkeys;   // keys: M, C and twice K / 128, nkeys in all
    int64_t part;          // the products' partial sums
    int64_t bytes;
};
BwdLayout layout(int64_t M, int64_t N, int64_t K, bool gated, bool rest, const PlanBwd& p) {
    BwdLayout l;
    l.Mp = rows_padded(M, rest);
    l.C = dz_columns(N, gated, rest);
    l.Np = gated ? l.C / 2 : l.C;
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t p = at; at += up256(bytes); return p; };
    const int e = rest ? 3 : 2;                             // bytes an element
    l.dz = take(e * M * l.C);
    l.dzt = take(e * l.C * l.Mp);
    l.wt = take(e * K * l.C);
    l.xt = take(e * K * l.Mp);
    l.sx = take(4 * M);
    l.sw = take(8 * ((N + 127) / 128));
    l.nkeys = M + l.C + K / 64;
    l.krow = take(4 * l.nkeys);
    l.kcol = l.krow + 4 * M;
    l.kx = l.kcol + 4 * l.C;
    l.kw = l.kx + 4 * (K / 128);
    l.part = take(std::max(p.dx.part, p.dw.part));
    l.bytes = at;
    return l;
}

}  // namespace

void launch_zero16(void* p, int64_t n, hipStream_t st) {
    k_zero16<<<(unsigned)std::min<int64_t>((n + 255) / 256, 65536), 256, 0, st>>>((uint16_t*)p, n);
}

namespace {

PlanBwd plan_of(int64_t M, int64_t N, int64_t K, bool gated, bool rest, bool act) {
    if (act) return plan_bwd_act(M, N, K, rest);
    return PlanBwd{plan_dx(M, N, K, gated, rest), plan_dw(M, N, K, gated, rest), false};
}
int64_t layout_bytes(int64_t M, int64_t N, int64_t K, bool gated, bool rest, bool act) {
    return layout(M, N, K, gated, rest, plan_of(M, N, K, gated, rest, act)).bytes;
}

int64_t bias_rows(int64_t M) { return (M + 127) / 128 * 2; }  // sums of 64 rows, padded as M is with a rest

// dx, the weight gradients and, of a projection with an epilogue (act), the
// partial sums of dbias (bias: [bias_rows(M)][N] floats, or nullptr); sizes > 0
void run_bwd(const MmBwd& f, int mode, bool act, float* bias, hipStream_t st) {
    const bool gated = mode == kOfGated, rest = has_rest(f.dt, mode);
    PlanBwd plan = plan_of(f.M, f.N, f.K, gated, rest, act);
    const BwdLayout l = layout(f.M, f.N, f.K, gated, rest, plan);
    char* ws = (char*)f.ws;
    char *dz = ws + l.dz, *dzt = ws + l.dzt, *wt = ws + l.wt, *xt = ws + l.xt;
    float* part = (float*)(ws + l.part);
    const int KB = f.K / 128;
    const bool wdx = f.dx != nullptr, wdw = f.dw0 != nullptr;
    if (plan.both && !(wdx && wdw)) {
        plan.dx = alone16(f.M, f.K, plan.dx.kper);
        plan.dw = alone16(f.N, f.K, plan.dw.kper);
        plan.both = false;
    }
    const int nb = (f.N + 127) / 128;
    float *sx = (float*)(ws + l.sx), *sw = (float*)(ws + l.sw);
    uint32_t *krow = (uint32_t*)(ws + l.krow), *kcol = (uint32_t*)(ws + l.kcol), *kx = (uint32_t*)(ws + l.kx),
             *kw = (uint32_t*)(ws + l.kw);
    const float* ws1 = gated ? f.ws1 : nullptr;
    const ScaleArgs sa{f.xs, f.M, f.ws0, ws1, nb, KB, sx, sw, krow, l.nkeys, mode != kOfLinear};
    k_scales<<<(unsigned)std::min<int64_t>((f.M + (gated ? 2 : 1) * nb + 15) / 16, 4096), 256, 0, st>>>(sa);
    KeyArgs ka{(const uint16_t*)f.dy, (const uint16_t*)f.z, f.M, f.N, f.act, sx, sw, wdx ? krow : nullptr,
               wdw ? kcol : nullptr, (int)l.Np, f.xs, f.ws0, ws1, nb, KB, kx, kw, 0, 0, (uint32_t)nb};
    ka.e0 = (uint32_t)nb * (uint32_t)((f.M + 127) / 128);
    ka.e1 = ka.e0 + (uint32_t)((f.M + kKeyRows - 1) / kKeyRows);
    const unsigned gk = ka.e1 + (gated ? 2 : 1) * (uint32_t)((nb + kKeyRows - 1) / kKeyRows);
    with_dt(f.dt, mode, [&](auto DT, auto MD) { k_keys<decltype(DT)::value, decltype(MD)::value><<<gk, 256, 0, st>>>(ka); });
    PrepArgs p{};
    const int qx = f.xfmt == kE4M3 ? 9 : 16, qw = f.wfmt == kE4M3 ? 9 : 16;   // 448 < 2^9, 57344 < 2^16
    p.dz = DzArgs{(const uint16_t*)f.dy, (const uint16_t*)f.z, f.M, l.Mp, f.N, (int)l.Np, f.act,
                  wdx ? dz : nullptr, wdw ? dzt : nullptr, sx, sw, nb, krow, kcol, bias};
    p.x = DeqTArgs{f.x, f.xs, f.M, KB, 0, xt, l.Mp, 0, sx, kx, qx};
    p.w0 = DeqTArgs{f.w0, f.ws0, f.N, KB, 7, wt, l.C, 0, sw, kw, qw};
    p.w1 = DeqTArgs{f.w1, f.ws1, f.N, KB, 7, wt, l.C, l.Np, sw + nb, kw, qw};
    p.dzx = (uint32_t)(l.Np / 64);
    const uint32_t row_tiles = (uint32_t)(l.Mp / 64), w_tiles = wdx ? (uint32_t)KB * p.dzx : 0;
    p.e0 = p.dzx * row_tiles;
    p.e1 = p.e0 + (wdw ? (uint32_t)KB * row_tiles : 0);
    p.e2 = p.e1 + w_tiles;
    const unsigned g = p.e2 + (gated ? w_tiles : 0);
    with_fmt(f.xfmt, [&](auto X) {
        with_fmt(f.wfmt, [&](auto W) {
            constexpr int XF = decltype(X)::value, WF = decltype(W)::value;
            with_dt(f.dt, mode, [&](auto DT, auto MD) {
                constexpr int T = decltype(DT)::value, MODE = decltype(MD)::value;
                // an activation without a gate comes with a bias more often than not: one instance serves both
                if constexpr (MODE == kOfUnary) k_prep<T, MODE, true, XF, WF><<<g, 256, 0, st>>>(p);
                else if (MODE == kOfLinear && bias) k_prep<T, kOfLinear, true, XF, WF><<<g, 256, 0, st>>>(p);
                else k_prep<T, MODE, false, XF, WF><<<g, 256, 0, st>>>(p);
            });
        });
    });
    const Mm16Args ax = mm16_args(dz, wt, f.M, f.K, l.C, rest, f.dx, nullptr, f.M, f.M, f.dt, plan.dx, krow, kw, qw, part);
    const Mm16Args aw = mm16_args(dzt, xt, gated ? l.Np + f.N : f.N, f.K, l.Mp, rest, f.dw0, gated ? f.dw1 : nullptr, f.N,
                                  gated ? l.Np : f.N, f.dwdt, plan.dw, kcol, kx, qx, part);
    if (plan.both) return mm16_two(ax, aw, plan.dx.bm, rest, st);
    if (wdx) mm16(ax, plan.dx.bm, rest, st);
    if (wdw) mm16(aw, plan.dw.bm, rest, st);
}

}  // namespace

int64_t mm_bwd_workspace(int64_t M, int64_t N, int64_t K, bool gated) {
    if (M == 0 || N == 0 || K == 0) return 0;
    // enough for either type of gradient, which is not known here
    return std::max(layout_bytes(M, N, K, gated, false, false), layout_bytes(M, N, K, gated, gated, false));
}

void launch_mm_bwd(const MmBwd& f, hipStream_t st) {
    if (f.M == 0 || f.N == 0 || f.K == 0) {
        zero(f.dx, f.M * f.K, f.dt, st);
        zero(f.dw0, (int64_t)f.N * f.K, f.dwdt, st);
        zero(f.dw1, (int64_t)f.N * f.K, f.dwdt, st);
        return;
    }
    run_bwd(f, f.gated ? kOfGated : kOfLinear, false, nullptr, st);
}

int64_t mm_act_bwd_workspace(int64_t M, int64_t N, int64_t K) {
    if (M == 0 || N == 0) return 0;
    const int64_t products = K == 0 ? 0 : std::max(layout_bytes(M, N, K, false, false, true), layout_bytes(M, N, K, false, true, true));
    return products + bias_rows(M) * N * 4;
}

void launch_mm_act_bwd(const MmActBwd& e, hipStream_t st) {
    const MmBwd& f = e.f;
    if (f.M == 0 || f.N == 0) {
        zero(f.dx, f.M * f.K, f.dt, st);
        zero(f.dw0, (int64_t)f.N * f.K, f.dwdt, st);
        zero(e.db, f.N, f.dwdt, st);
        return;
    }
    const int mode = f.act == kIdentity ? kOfLinear : kOfUnary;
    const bool products = f.K > 0 && (f.dx || f.dw0), rest = has_rest(f.dt, mode);
    float* bias = e.db ? (float*)((char*)f.ws + (products ? layout_bytes(f.M, f.N, f.K, false, rest, true) : 0)) : nullptr;
    const int64_t tiles = (products ? rows_padded(f.M, rest) : up64(f.M)) / 64;
    if (products) {
        run_bwd(f, mode, true, bias, st);
    } else {                                                // dbias alone: the tiles of dz, none laid out
        PrepArgs p{};
        p.dz.dy = (const uint16_t*)f.dy;
        p.dz.z = (const uint16_t*)f.z;
        p.dz.M = f.M;
        p.dz.N = f.N;
        p.dz.act = f.act;
        p.dz.bias = bias;
        p.dzx = (uint32_t)(up64(f.N) / 64);
        p.e0 = p.e1 = p.e2 = p.dzx * (uint32_t)tiles;
        with_dt(f.dt, mode, [&](auto DT, auto MD) {
            if constexpr (decltype(MD)::value != kOfGated)
                k_prep<decltype(DT)::value, decltype(MD)::value, true, kE4M3, kE4M3><<<p.e0, 256, 0, st>>>(p);
        });
    }
    if (e.db) launch_column_sums(bias, tiles, f.N, e.db, nullptr, f.dwdt, st);
}

}  // namespace fp8q
