// fp8q_rows.h -- device helpers of the kernels that hold rows in registers
// (fp8q_norm.hip, fp8q_layernorm.hip): loads and stores of lane vectors of rows
// of any width, sums and maxima over a row's lanes, and the casts of a row.
#pragma once

#include "fp8q_host.h"

namespace fp8q {

namespace {

// 16 bytes at an address aligned to the element only: gfx950 executes it as
// one global_load/store_dwordx4 (unaligned access mode is on), so rows of any
// width take the same path as aligned ones.
typedef unsigned int v4u_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int v2u_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned int u32_a1 __attribute__((aligned(1)));

// the lane vector of VE elements of row `row` that starts at column c; the
// last vector of a row may hold fewer than VE (the rest read as zero).  NT: a
// stream read once.  Rows of whole 128-element groups are streamed past the
// caches (16384 x 7168 bf16: 158.6 us against 166.6); rows that may end inside
// a line are not, because the line's other half is the next row's (1999 x 5001
// f32: 21.4 us streamed, 19.1 cached).
template <int DT, bool NT = true> __device__ __forceinline__ v4u ld_row(const void* row, int c, int cols) {
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    if (c + VE <= cols) {
        const v4u_a2* p = (const v4u_a2*)((const char*)row + (int64_t)c * ES);
        const v4u_a2 t = NT ? __builtin_nontemporal_load(p) : *p;
        return v4u{t.x, t.y, t.z, t.w};
    }
    union { v4u v; uint32_t w[4]; uint16_t e[8]; } t;
    t.v = v4u{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < VE; ++k)
        if (c + k < cols) {
            if constexpr (DT == kF32) t.w[k] = ((const uint32_t*)row)[c + k];
            else t.e[k] = ((const uint16_t*)row)[c + k];
        }
    return t.v;
}

template <int DT, bool NT = true> __device__ __forceinline__ void st_row(void* row, int c, int cols, const float* p) {
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    const v4u t = pack_out16<DT>(p);
    if (c + VE <= cols) {
        v4u_a2* d = (v4u_a2*)((char*)row + (int64_t)c * ES);
        if constexpr (NT) __builtin_nontemporal_store(v4u_a2{t.x, t.y, t.z, t.w}, d);
        else *d = v4u_a2{t.x, t.y, t.z, t.w};
        return;
    }
#pragma unroll
    for (int k = 0; k < VE; ++k)
        if (c + k < cols) store1<DT>(row, c + k, p[k]);
}

template <int FMT, int VE, bool NT> __device__ __forceinline__ void st_codes(uint8_t* row, int c, int cols, const float* p) {
    uint32_t w[VE / 4];
#pragma unroll
    for (int k = 0; k < VE / 4; ++k) w[k] = enc4<FMT>(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
    if (c + VE <= cols) {
        if constexpr (VE == 8 && NT) __builtin_nontemporal_store(v2u_a1{w[0], w[1]}, (v2u_a1*)(row + c));
        else if constexpr (VE == 8) *(v2u_a1*)(row + c) = v2u_a1{w[0], w[1]};
        else if constexpr (NT) __builtin_nontemporal_store((u32_a1)w[0], (u32_a1*)(row + c));
        else *(u32_a1*)(row + c) = w[0];
        return;
    }
#pragma unroll
    for (int k = 0; k < VE; ++k)
        if (c + k < cols) row[c + k] = (uint8_t)(w[k / 4] >> (8 * (k & 3)));
}

template <int DT> __device__ __forceinline__ void widen16(v4u r, float* v) {
    HpVec<DT> t;
    t.r = r;
    t.widen(v);
}

// VE weights from column c (zero past the row's end), kept as loaded; WF32: the
// weight is binary32 whatever the activations are
template <int DT, bool WF32> struct Weights {
    static constexpr bool kWide = WF32 && DT != kF32;
    v4u r[kWide ? 2 : 1];
    __device__ __forceinline__ void load(const void* w, int c, int cols) {
        if constexpr (!kWide) {
            r[0] = ld_row<DT, false>(w, c, cols);
        } else {
            r[0] = ld_row<kF32, false>(w, c, cols);
            r[1] = ld_row<kF32, false>(w, c + 4, cols);
        }
    }
    // the asm keeps the compiler from widening once for all rows: that holds
    // twice the registers, and spills beside the next row's loads
    __device__ __forceinline__ void widen(float* v) {
        asm volatile("" : "+v"(r[0]));
        if constexpr (kWide) asm volatile("" : "+v"(r[1]));
        if constexpr (!kWide) {
            widen16<DT>(r[0], v);
        } else {
            widen16<kF32>(r[0], v);
            widen16<kF32>(r[1], v + 4);
        }
    }
};
template <int DT, bool WF32> __device__ __forceinline__ void ld_weight(const void* w, int c, int cols, float* v) {
    Weights<DT, WF32> t;
    t.load(w, c, cols);
    t.widen(v);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// LDS writes of every wave are visible after it; loads in flight stay in
// flight (the next row's are)
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// sum and max over the lanes of a row: one wave (WAVE), or the whole
// workgroup through lds, whose 16 words may be written again after the
// workgroup's next barrier
template <bool WAVE> __device__ __forceinline__ float row_sum(float v, float* lds) {
    v = wave_sum(v);
    if constexpr (WAVE) return v;
    const int nw = (int)blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    lds_barrier();
    float s = lds[0];
    for (int i = 1; i < nw; ++i) s += lds[i];
    return s;
}

template <bool WAVE> __device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* lds) {
    v = max_lanes<64>(v);
    if constexpr (WAVE) return v;
    const int nw = (int)blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    lds_barrier();
    uint32_t m = lds[0];
    for (int i = 1; i < nw; ++i) m = umax(m, lds[i]);
    return m;
}

// h of one lane vector, in binary32, from the loaded vectors
template <int DT> __device__ __forceinline__ void sum_h(v4u x, v4u r, bool res, float* h) {
    constexpr int VE = LaneVE<DT>::value;
    widen16<DT>(x, h);
    if (res) {
        float t[VE];
        widen16<DT>(r, t);
#pragma unroll
        for (int k = 0; k < VE; ++k) h[k] += t[k];
    }
}
template <int DT> __device__ __forceinline__ void load_h(const void* xr, const void* rr, int c, int cols, float* h) {
    sum_h<DT>(ld_row<DT>(xr, c, cols), rr ? ld_row<DT>(rr, c, cols) : v4u{0, 0, 0, 0}, rr != nullptr, h);
}

// scale and encode one lane vector of y; group: every 128 / VE lanes hold one
// group, whose scale comes from their max; else (scale, sat) are the row's
template <int DT, int FMT, bool GROUP>
__device__ __forceinline__ void cast_vec(const float* y, int c, int cols, uint8_t* qr, float* sr, float scale,
                                         bool satur) {
    constexpr int VE = LaneVE<DT>::value;
    float p[VE];
    if constexpr (GROUP) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < VE; ++k) m = umax(m, __float_as_uint(y[k]) & 0x7FFFFFFFu);
        m = max_lanes<128 / VE>(m);
        m = umax(m, 0x38D1B717u);                           // the 1e-4 clamp; a NaN stays above it
        const float a = __uint_as_float(m), sc = Fp8Fmt<FMT>::max / a;
        if (c < cols && (c & 127) == 0) sr[c >> 7] = a / Fp8Fmt<FMT>::max;
#pragma unroll
        for (int k = 0; k < VE; ++k) p[k] = y[k] * sc;
    } else {
#pragma unroll
        for (int k = 0; k < VE; ++k) p[k] = satur ? sat<FMT>(y[k] * scale) : y[k] * scale;
    }
    if (c < cols) st_codes<FMT, VE, GROUP>(qr, c, cols, p);
}

// the per-row scale from the row's amax bits (the per-channel cast's guard)
template <int FMT> __device__ __forceinline__ float row_scale(uint32_t m, float* sinv, bool first, bool* satur) {
    const float amax = __uint_as_float(m);
    const float a = amax > 0.0f ? amax : 1.0f;
    const float scale = Fp8Fmt<FMT>::max / a;
    if (first) *sinv = a / Fp8Fmt<FMT>::max;
    *satur = needs_saturation(m, scale);
    return scale;
}

// f(bool_constant) over a runtime flag
template <typename F> void with_bool(bool b, F&& f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
}

}  // namespace

}  // namespace fp8q
