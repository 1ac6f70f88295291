// fp8q_mm.h -- the tiled matrix products of the feed-forward operators.
//
// One loader serves the fp8 forward products and the f16 backward ones.
// Both are C[m, n] = sum_k A[m, k] B[n, k] with rows of A ("tokens") and of B
// ("columns") contiguous in k, and both move 128 bytes of every row per step:
// 128 fp8 codes or 64 f16 values.
//
//  - A workgroup of 8 waves owns BM rows of A by 256 rows of B.  Wave (wm, wn)
//    of the 2 x 4 grid owns BM/2 rows of A and 64 of B: 32 from each half of
//    the 256, so that the gate and the up projection of one output column
//    (the two halves of a gated tile) end in the same lane.
//  - B is the first MFMA operand, so a result register block holds 4
//    consecutive n of one m per lane; B's rows are dealt to the MFMA tiles so
//    that a lane's two blocks are 8 consecutive n: 16-byte stores.
//  - Tiles go from memory to LDS directly (global_load_lds, 16 bytes a lane),
//    16-byte chunk c of row r at chunk c ^ (r & 7): the fragment reads of 16
//    rows then spread over all banks.
//  - The sum over 128 codes times the two scales of that block goes to a
//    binary32 accumulator, one FMA per element.
//
// Two matrix instructions sum the 128 codes.  v_mfma_f32_16x16x128_f8f6f4
// takes codes directly (4.9 PFLOP/s measured), but it aligns the products of a
// step to the largest before adding them: 1.5e-5 of the sum's rms on normal
// data, 4e-5 where one code of the block is 20 times the rest (measured; the
// older 16x16x32 fp8 form gives the same bits).  That is 1/5 of f16's and 1/40
// of bf16's own rounding, so it serves 16-bit results.  Results that are
// binary32, and scales computed from the sums, take the codes as bf16 (exact)
// through v_mfma_f32_16x16x32_bf16 (2.3 PFLOP/s, 1e-8).
#pragma once

#include "fp8q_device.h"
#include "fp8q_ffn_launch.h"

namespace fp8q {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kMmThreads = 512;
constexpr int kMmBN = 256;

// 16 bytes a lane from base + voff to LDS at lds + lane * 16 (lds_dma4_at: 4
// bytes from the lane's own address).  base and lds are wave-uniform.  Written
// as asm because the compiler would otherwise wait for every load in flight
// before each LDS read; nothing is returned in registers, and the pipeline
// waits with dma_wait.  The LDS address goes through m0, which is named as
// clobbered: the compiler writes m0 for uses of its own, and would keep such a
// value across the asm.  It warns that m0 is a reserved register, which is that
// it never allocates m0 to a value.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma16(uint32_t lds, uint32_t voff, const void* base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base)
                 : "memory", "m0");
}
__device__ __forceinline__ void lds_dma4_at(uint32_t lds, const void* addr) {   // a lane's own address
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(addr)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
// all but this wave's N newest LDS loads have landed, and its LDS reads have returned
template <int N = 0> __device__ __forceinline__ void dma_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wg_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
// Workgroup -> tile.  Workgroup i runs on XCD i mod 8; each XCD takes one
// contiguous run of the tile order, which walks groups of 8 row tiles column
// by column, so the 32 workgroups an XCD runs at once share 8 A tiles and 4 B
// tiles in its L2.
__device__ __forceinline__ void tile_of(uint32_t bid, uint32_t tm, uint32_t tn, uint32_t* im, uint32_t* in) {
    const uint32_t total = tm * tn;
    const uint32_t q = total / 8, r = total % 8, x = bid % 8, i = bid / 8;
    const uint32_t id = x * q + (x < r ? x : r) + i;
    const uint32_t per = 8 * tn, g = id / per, first = g * 8;
    const uint32_t gm = tm - first < 8 ? tm - first : 8;
    const uint32_t l = id - g * per;
    *im = first + l % gm;
    *in = l / gm;
}

// the row of B (within its half of 128) that LDS row p of the half holds:
// row r of MFMA tile j of a 32-row block is column 8 (r / 4) + 4 j + r % 4
__device__ __forceinline__ int b_row_of(int p) {
    const int q = p & 31, j = q >> 4, r = q & 15;
    return (p & ~31) + 8 * (r >> 2) + 4 * j + (r & 3);
}

// Tile loader: the rows of one stage, [BM rows of A][256 rows of B], 128 bytes
// each.  Every wave loads 8 rows per instruction; offsets within a row do not
// change from step to step, only the three bases move.
template <int BM> struct TileLoad {
    static constexpr int JA = BM / 64, JB = 4;
    const char* a;
    const char* b0;
    const char* b1;
    uint32_t va[JA], vb[JB];
    uint32_t lds;      // this wave's first LDS byte of a stage, relative to the stage

    // rows past the end of A or B read the last row instead; their results
    // are not stored
    __device__ __forceinline__ void init(const void* A, int64_t m0, int64_t M, const void* B0, const void* B1,
                                         int64_t n0, int64_t n1, int64_t N0, int64_t N1, int64_t row_bytes, int wave,
                                         int lane) {
        a = (const char*)A + m0 * row_bytes;
        b0 = (const char*)B0 + n0 * row_bytes;
        b1 = (const char*)B1 + n1 * row_bytes;
        const int sub = lane >> 3, ch = lane & 7;
        const uint32_t off = (uint32_t)((ch ^ sub) * 16);    // LDS rows of a wave start at a multiple of 8
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            int64_t r = j * 64 + wave * 8 + sub;
            if (r > M - 1 - m0) r = M - 1 - m0;
            va[j] = (uint32_t)(r * row_bytes) + off;
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int p = (j * 64 + wave * 8 + sub) & 127;
            int64_t r = b_row_of(p);
            const int64_t last = j < 2 ? N0 - 1 - n0 : N1 - 1 - n1;
            if (r > last) r = last;
            // a half that lies wholly past the end reads the last row before its base
            vb[j] = (uint32_t)((r < 0 ? 0 : r) * row_bytes) + off;
        }
        if (n1 > N1 - 1) b1 = (const char*)B1 + (N1 - 1) * row_bytes;
        lds = (uint32_t)(wave * 1024);
    }
    __device__ __forceinline__ void issue(uint32_t stage_lds, int64_t k) const {
        const char* ak = a + k * 128;
        const char* b0k = b0 + k * 128;
        const char* b1k = b1 + k * 128;
#pragma unroll
        for (int j = 0; j < JA; ++j) lds_dma16(stage_lds + lds + j * 8192, va[j], ak);
#pragma unroll
        for (int j = 0; j < JB; ++j) lds_dma16(stage_lds + lds + (JA + j) * 8192, vb[j], j < 2 ? b0k : b1k);
    }
};

// two 16-byte chunks of LDS as one fragment
__device__ __forceinline__ v8i frag(const char* p0, const char* p1) {
    const v4i a = *(const v4i*)p0, b = *(const v4i*)p1;
    return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// c + the sum over 128 codes; FA, FB: formats of the first and second operand
template <int FA, int FB> __device__ __forceinline__ v4f mfma_fp8(v8i a, v8i b, v4f c = {0.0f, 0.0f, 0.0f, 0.0f}) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, FA, FB, 0, 0, 0, 0);
}

__device__ __forceinline__ v4f mfma_bf16(v4i a, v4i b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
__device__ __forceinline__ v4f mfma_f16(v4i a, v4i b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16 fp8 codes of each chunk as bf16, 8 at a time: exact for every code
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
template <int FMT> __device__ __forceinline__ void widen_codes(v8i c, v4i (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v2bf lo, hi;
        if constexpr (FMT == kE4M3) {
            lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[i], 1.0f, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[i], 1.0f, true);
        } else {
            lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)c[i], 1.0f, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)c[i], 1.0f, true);
        }
        o[i >> 1][2 * (i & 1)] = __builtin_bit_cast(int, lo);
        o[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(int, hi);
    }
}

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
// Each is g times a probability that vanishes for negative g: the logistic
// function of w = g (SiLU) or of w = 2 sqrt(2 / pi) (g + 0.044715 g^3) (tanh GELU:
// 1 + tanh would cancel, and leaves nothing from g = -5.5 on), or the normal
// distribution, from erfc for the same reason.  Far out, where exp(-w) or erfc
// leave binary32 before their product with another factor does, the value and
// the slope are kept with a factor e, a square root of what vanishes, still to
// be multiplied: act(g) u = (a u) e.
struct Act {
    float a, d, e;         // act(g) = a e, act'(g) = d e
};

// QUICK: the logistic function to 2^-16 only, and never less than exp's smallest
// normal value, where no more than its exponent counts
template <int ACT, bool SLOPE, bool QUICK = false> __device__ __forceinline__ Act act_at(float g) {
    Act r;
    r.d = 0.0f;
    if constexpr (ACT == kGelu) {
        if (g < -10.0f) {
            // Phi(g) = phi(g) / -g (1 - 1/g^2 + 3/g^4 - 15/g^6 + 105/g^8 - ...), the next term under 1e-7
            const float x = g * g, q = 1.0f / x, h = 0.39894228040143268f;
            const float c = h * (1.0f - q * (1.0f - 3.0f * q * (1.0f - 5.0f * q * (1.0f - 7.0f * q)))) / -g;
            r.e = expf(-0.25f * x);
            r.a = g * r.e * c;
            if (SLOPE) r.d = r.e * (c + h * g);
        } else {
            const float c = 0.5f * erfcf(g * -0.70710678118654752f);
            r.e = 1.0f;
            r.a = g * c;
            if (SLOPE) r.d = c + g * (0.39894228040143268f * expf(-0.5f * g * g));
        }
        return r;
    } else {
        // w and its derivative w1; beyond |g| = 64 the logistic function of the tanh
        // form's w is 0 or 1, and is taken at 64, where g^3 is finite (a NaN passes)
        float w = g, w1 = 1.0f, h = g;
        if constexpr (ACT == kGeluTanh) {
            const float k = 1.5957691216057308f;
            h = g > 64.0f ? 64.0f : g < -64.0f ? -64.0f : g;
            w = k * (h + 0.044715f * h * h * h);
            w1 = k * (1.0f + 0.134145f * h * h);
        }
        const bool tail = w < -60.0f;
        const float x = tail ? 0.5f * w : -w;
        const float t = QUICK ? fmaxf(__expf(x), 0x1p-126f) : expf(x);   // __expf has no subnormal values
        r.e = tail ? t : 1.0f;
        if (!SLOPE) {
            r.a = tail ? g * t : g / (1.0f + t);
            return r;
        }
        const float s = tail ? t : QUICK ? __builtin_amdgcn_rcpf(1.0f + t) : 1.0f / (1.0f + t);
        r.a = g * s;
        r.d = s * (1.0f + h * ((tail ? 1.0f : 1.0f - s) * w1));
        return r;
    }
}

// act(g) * u
template <int ACT> __device__ __forceinline__ float gated_value(float g, float u) {
    const Act r = act_at<ACT, false>(g);
    return r.a * u * r.e;
}

// f(integral_constant) over a runtime activation
template <typename F> __device__ __forceinline__ void with_act(int act, F&& f) {
    if (act == kSilu) f(std::integral_constant<int, kSilu>{});
    else if (act == kGelu) f(std::integral_constant<int, kGelu>{});
    else f(std::integral_constant<int, kGeluTanh>{});
}

// ---------------------------------------------------------------------------
// output of 8 consecutive columns n .. n+7 of row m (row pitch N), rounded
// once; vec: 16-byte aligned rows (N % 8 == 0 and an aligned base)
// ---------------------------------------------------------------------------

__device__ __forceinline__ void put8(void* y, int ydt, int64_t m, int64_t pitch, int n, int N, bool vec, const float* v) {
    const int64_t e = m * pitch + n;
    if (vec && n + 8 <= N) {
        if (ydt == kF32) {
            *(v4f*)((float*)y + e) = v4f{v[0], v[1], v[2], v[3]};
            *(v4f*)((float*)y + e + 4) = v4f{v[4], v[5], v[6], v[7]};
        } else if (ydt == kBF16) {
            *(v4u*)((uint16_t*)y + e) = pack_out16<kBF16>(v);
        } else {
            *(v4u*)((uint16_t*)y + e) = pack_out16<kF16>(v);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (n + k < N) {
            if (ydt == kF32) store1<kF32>(y, e + k, v[k]);
            else if (ydt == kBF16) store1<kBF16>(y, e + k, v[k]);
            else store1<kF16>(y, e + k, v[k]);
        }
}

}  // namespace fp8q
