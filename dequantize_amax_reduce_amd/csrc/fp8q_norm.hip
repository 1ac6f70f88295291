// fp8q_norm.hip -- residual addition, root-mean-square norm and the cast of
// its result to fp8, and the norm's backward pass.
//
//   h = x + r;  rstd = 1 / sqrt(mean(h^2) + eps);  y = (h * rstd) * w;
//   q, scale_inv = cast(y), per 128 columns or per row.
//
// Bound by HBM: x and r are read once, h, q and the scales written once.  A
// row stays in registers between its two reductions (the sum of squares, and
// the amax of the cast), as binary32, so that y comes from the sum before its
// rounding to the element type.
#include "fp8q_ffn_launch.h"
#include "fp8q_ffn_plan.h"
#include "fp8q_host.h"
#include "fp8q_rows.h"

namespace fp8q {

namespace {

struct NormArgs {
    const void* x;
    const void* res;
    const void* w;
    int64_t rows;
    int cols;
    float eps;
    uint8_t* q;
    float* sinv;
    void* h;
    float* rstd;
};

__device__ __forceinline__ float rstd_of(float ss, int cols, float eps) {
    return 1.0f / sqrtf(ss / (float)cols + eps);
}

// One row per workgroup (or, WAVE, per wave) at a time, V lane vectors a
// thread.  A workgroup takes several rows, so that the weight is read once and
// the next row's loads are in flight through the reductions and stores of this
// one: 16384 x 7168 bf16 with residual 158.6 us with one row a workgroup.
// TB: the most threads; up to 512 leave the registers for the next row's loads.
template <int DT, bool WF32, int FMT, bool GROUP, bool WAVE, int V, int TB>
__global__ void __launch_bounds__(TB) k_norm_rows(NormArgs a) {
    constexpr bool PF = TB <= 512;
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    __shared__ float lds_s[2][16];
    __shared__ uint32_t lds_m[2][16];
    const int lanes = WAVE ? 64 : (int)blockDim.x;
    const int t = WAVE ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
    const int per = WAVE ? (int)blockDim.x >> 6 : 1;        // rows a workgroup takes at once
    const int64_t first = (int64_t)blockIdx.x * per + (WAVE ? threadIdx.x >> 6 : 0), next = (int64_t)gridDim.x * per;
    if (first >= a.rows) return;                            // whole waves; whole workgroups unless WAVE
    v4u xv[V], rv[V];
    auto load = [&](int64_t row) {
        const int64_t off = row * (int64_t)a.cols * ES;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * lanes + t) * VE;
            xv[v] = ld_row<DT, GROUP>((const char*)a.x + off, c, a.cols);
            if (a.res) rv[v] = ld_row<DT, GROUP>((const char*)a.res + off, c, a.cols);
        }
    };
    load(first);
    Weights<DT, WF32> w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) w[v].load(a.w, (v * lanes + t) * VE, a.cols);
    int flip = 0;
    for (int64_t row = first; row < a.rows; row += next, flip ^= 1) {
        float h[V][VE];
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sum_h<DT>(xv[v], rv[v], a.res != nullptr, h[v]);
#pragma unroll
            for (int k = 0; k < VE; ++k) ss = __builtin_fmaf(h[v][k], h[v][k], ss);
        }
        if (PF && row + next < a.rows) load(row + next);
        const float rs = rstd_of(row_sum<WAVE>(ss, lds_s[flip]), a.cols, a.eps);
        if (t == 0 && a.rstd) a.rstd[row] = rs;
        if (a.h) {
            void* hr = (char*)a.h + row * (int64_t)a.cols * ES;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (v * lanes + t) * VE;
                if (c < a.cols) st_row<DT, GROUP>(hr, c, a.cols, h[v]);
            }
        }
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float wv[VE];
            w[v].widen(wv);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                h[v][k] = (h[v][k] * rs) * wv[k];
                if constexpr (!GROUP) {
                    const int c = (v * lanes + t) * VE + k;     // columns past the row's end do not count
                    m = umax(m, c < a.cols ? __float_as_uint(h[v][k]) & 0x7FFFFFFFu : 0u);
                }
            }
        }
        float scale = 0.0f;
        bool satur = false;
        if constexpr (!GROUP) scale = row_scale<FMT>(row_max<WAVE>(m, lds_m[flip]), a.sinv + row, t == 0, &satur);
        uint8_t* qr = a.q + row * (int64_t)a.cols;
        float* sr = GROUP ? a.sinv + row * (int64_t)(a.cols >> 7) : nullptr;
#pragma unroll
        for (int v = 0; v < V; ++v)
            cast_vec<DT, FMT, GROUP>(h[v], (v * lanes + t) * VE, a.cols, qr, sr, scale, satur);
        if (!PF && row + next < a.rows) load(row + next);
    }
}

// Rows too long for registers: three passes over the row, the later ones
// mostly from cache.  h is written in the last pass, after a lane's own reads
// of the same columns, so that it may be x or the residual itself.
template <int DT, bool WF32, int FMT, bool GROUP> __global__ void __launch_bounds__(1024) k_norm_long(NormArgs a) {
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    __shared__ float lds_s[16];
    __shared__ uint32_t lds_m[16];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t off = row * (int64_t)a.cols * ES;
        const void* xr = (const char*)a.x + off;
        const void* rr = a.res ? (const char*)a.res + off : nullptr;
        const int step = (int)blockDim.x * VE;
        const int c0 = (int)threadIdx.x * VE;
        float ss = 0.0f;
        for (int64_t c = c0; c < a.cols; c += step) {
            float h[VE];
            load_h<DT>(xr, rr, (int)c, a.cols, h);
#pragma unroll
            for (int k = 0; k < VE; ++k) ss = __builtin_fmaf(h[k], h[k], ss);
        }
        const float rs = rstd_of(row_sum<false>(ss, lds_s), a.cols, a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rs;
        float scale = 0.0f;
        bool satur = false;
        if constexpr (!GROUP) {
            uint32_t m = 0;
            for (int64_t c = c0; c < a.cols; c += step) {
                float h[VE], w[VE];
                load_h<DT>(xr, rr, (int)c, a.cols, h);
                ld_weight<DT, WF32>(a.w, (int)c, a.cols, w);
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    m = umax(m, c + k < a.cols ? __float_as_uint((h[k] * rs) * w[k]) & 0x7FFFFFFFu : 0u);
            }
            scale = row_scale<FMT>(row_max<false>(m, lds_m), a.sinv + row, threadIdx.x == 0, &satur);
        }
        uint8_t* qr = a.q + row * (int64_t)a.cols;
        float* sr = GROUP ? a.sinv + row * (int64_t)(a.cols >> 7) : nullptr;
        void* hr = a.h ? (char*)a.h + off : nullptr;
        const int64_t end = ((int64_t)a.cols + step - 1) / step * step;   // whole waves stay in the group max
        for (int64_t c = c0; c < end; c += step) {
            float h[VE], w[VE];
            load_h<DT>(xr, rr, (int)(c < a.cols ? c : a.cols), a.cols, h);
            ld_weight<DT, WF32>(a.w, (int)(c < a.cols ? c : a.cols), a.cols, w);
            if (hr && c < a.cols) st_row<DT>(hr, (int)c, a.cols, h);
#pragma unroll
            for (int k = 0; k < VE; ++k) h[k] = (h[k] * rs) * w[k];
            cast_vec<DT, FMT, GROUP>(h, (int)(c < a.cols ? c : a.cols), a.cols, qr, sr, scale, satur);
        }
        __syncthreads();                                        // the reductions' LDS is used again
    }
}

// ---------------------------------------------------------------------------
// backward: n = h rstd, dn = dy w, dx = (dn - n mean(dn n)) rstd + dh, and
// dweight = sum over rows of dy n.  Each workgroup takes every G-th row and
// keeps its columns' dweight sums in registers; the G partial rows are summed
// in order by a second kernel, so the result does not depend on timing.
// ---------------------------------------------------------------------------

struct NormBwdArgs {
    const void* dy;
    const void* h;
    const void* w;
    const float* rstd;
    const void* dh;
    int64_t rows;
    int cols;
    void* dx;
    float* part;   // [gridDim.x][cols], or nullptr
};

// Waves of up to 512 threads hold the next row's dy and h meanwhile (8192 x
// 7168 bf16: 91.8 us against 95.5 without; dh too spilled registers, 101 us).
template <int DT, bool WF32, int V, int TB> __global__ void __launch_bounds__(TB, 4) k_norm_bwd(NormBwdArgs a) {
    constexpr bool PF = TB <= 512 && !Weights<DT, WF32>::kWide;
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    __shared__ float lds[2][16];
    const int T = (int)blockDim.x, t = (int)threadIdx.x;
    Weights<DT, WF32> w[V];
    float acc[V][VE];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v].load(a.w, (v * T + t) * VE, a.cols);
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[v][k] = 0.0f;
    }
    int flip = 0;
    v4u dyr[V], hr[V], dhr[V];
    float rsn;
    auto load = [&](int64_t row) {
        const int64_t off = row * (int64_t)a.cols * ES;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * VE;
            dyr[v] = ld_row<DT>((const char*)a.dy + off, c, a.cols);
            hr[v] = ld_row<DT>((const char*)a.h + off, c, a.cols);
        }
        rsn = a.rstd[row];
    };
    if ((int64_t)blockIdx.x < a.rows) load(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const int64_t off = row * (int64_t)a.cols * ES;
        const float rs = rsn;
        float s = 0.0f;
        float n[V][VE], dn[V][VE];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float wv[VE];
            w[v].widen(wv);
            widen16<DT>(dyr[v], dn[v]);
            widen16<DT>(hr[v], n[v]);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                n[v][k] *= rs;
                acc[v][k] = __builtin_fmaf(dn[v][k], n[v][k], acc[v][k]);
                dn[v][k] *= wv[k];
                s = __builtin_fmaf(dn[v][k], n[v][k], s);
            }
        }
        if (a.dh)
#pragma unroll
            for (int v = 0; v < V; ++v) dhr[v] = ld_row<DT>((const char*)a.dh + off, (v * T + t) * VE, a.cols);
        if (PF && row + gridDim.x < a.rows) load(row + gridDim.x);   // in flight through the reduction and the stores
        const float mean = row_sum<false>(s, lds[flip]) / (float)a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * VE;
            float o[VE];
#pragma unroll
            for (int k = 0; k < VE; ++k) o[k] = (dn[v][k] - n[v][k] * mean) * rs;
            if (a.dh) {
                float d[VE];
                widen16<DT>(dhr[v], d);
#pragma unroll
                for (int k = 0; k < VE; ++k) o[k] += d[k];
            }
            if (c < a.cols) st_row<DT>((char*)a.dx + off, c, a.cols, o);
        }
        if (!PF && row + gridDim.x < a.rows) load(row + gridDim.x);
    }
    if (a.part) {
        float* p = a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const int c = (v * T + t) * VE + k;
                if (c < a.cols) p[c] = acc[v][k];
            }
    }
}

// Rows too long for registers: the row is read twice, and the dweight sums
// live in the workgroup's own partial row (zeroed first; each word is touched
// by one thread only).
template <int DT, bool WF32> __global__ void __launch_bounds__(1024) k_norm_bwd_long(NormBwdArgs a) {
    constexpr int VE = LaneVE<DT>::value, ES = ESize<DT>::value;
    __shared__ float lds[2][16];
    const int step = (int)blockDim.x * VE;
    const int c0 = (int)threadIdx.x * VE;
    float* part = a.part ? a.part + (int64_t)blockIdx.x * a.cols : nullptr;
    if (part)
        for (int64_t c = c0; c < a.cols; c += step)
            for (int k = 0; k < VE; ++k)
                if (c + k < a.cols) part[c + k] = 0.0f;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const int64_t off = row * (int64_t)a.cols * ES;
        const float rs = a.rstd[row];
        float s = 0.0f;
        for (int64_t c = c0; c < a.cols; c += step) {
            float dy[VE], n[VE], w[VE];
            widen16<DT>(ld_row<DT>((const char*)a.dy + off, (int)c, a.cols), dy);
            widen16<DT>(ld_row<DT>((const char*)a.h + off, (int)c, a.cols), n);
            ld_weight<DT, WF32>(a.w, (int)c, a.cols, w);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                n[k] *= rs;
                s = __builtin_fmaf(dy[k] * w[k], n[k], s);
                if (part && c + k < a.cols) part[c + k] = __builtin_fmaf(dy[k], n[k], part[c + k]);
            }
        }
        const float mean = row_sum<false>(s, lds[flip]) / (float)a.cols;
        for (int64_t c = c0; c < a.cols; c += step) {
            float dy[VE], n[VE], w[VE], o[VE];
            widen16<DT>(ld_row<DT>((const char*)a.dy + off, (int)c, a.cols), dy);
            widen16<DT>(ld_row<DT>((const char*)a.h + off, (int)c, a.cols), n);
            ld_weight<DT, WF32>(a.w, (int)c, a.cols, w);
#pragma unroll
            for (int k = 0; k < VE; ++k) o[k] = (dy[k] * w[k] - (n[k] * rs) * mean) * rs;
            if (a.dh) {
                float d[VE];
                widen16<DT>(ld_row<DT>((const char*)a.dh + off, (int)c, a.cols), d);
#pragma unroll
                for (int k = 0; k < VE; ++k) o[k] += d[k];
            }
            st_row<DT>((char*)a.dx + off, (int)c, a.cols, o);
        }
    }
}

// dweight[c] = sum of part[0 .. parts)[c] in a fixed order: 32 columns a
// workgroup at a time, 32 row lanes, then a tree over the row lanes in LDS
// (each word of its first row is read by the thread that writes it next)
template <int WDT> __global__ void __launch_bounds__(1024) k_norm_dw(const float* part, int64_t parts, int cols, void* dw) {
    __shared__ float lds[32][33];
    const int cl = (int)threadIdx.x & 31, rl = (int)threadIdx.x >> 5;
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < cols; c0 += (int64_t)gridDim.x * 32) {
        const int64_t c = c0 + cl;
        float s = 0.0f;
        if (c < cols)
            for (int64_t p = rl; p < parts; p += 32) s += part[p * cols + c];
        lds[rl][cl] = s;
        __syncthreads();
        for (int o = 16; o > 0; o >>= 1) {
            if (rl < o) lds[rl][cl] += lds[rl + o][cl];
            __syncthreads();
        }
        if (rl == 0 && c < cols) store1<WDT>(dw, c, lds[0][cl]);
    }
}

template <int DT, int FMT> struct NormCast {
    static void run(bool group, bool wf32, const NormArgs& a, hipStream_t st) {
        constexpr int VE = LaneVE<DT>::value;
        const NormPlan p = norm_plan(a.rows, ((int64_t)a.cols + VE - 1) / VE);
        const unsigned g = (unsigned)p.groups;
        with_bool(group, [&](auto G) {
            with_bool(wf32 && DT != kF32, [&](auto W) {
                constexpr bool GR = decltype(G)::value, WF = decltype(W)::value;
                const int T = p.threads;
                if (p.V == 0) k_norm_long<DT, WF, FMT, GR><<<g, T, 0, st>>>(a);
                else if (p.wave && p.V == 1) k_norm_rows<DT, WF, FMT, GR, true, 1, 256><<<g, T, 0, st>>>(a);
                else if (p.wave) k_norm_rows<DT, WF, FMT, GR, true, 2, 256><<<g, T, 0, st>>>(a);
                else if (p.V == 1) k_norm_rows<DT, WF, FMT, GR, false, 1, 256><<<g, T, 0, st>>>(a);
                else if (p.V == 2 && T <= 512) k_norm_rows<DT, WF, FMT, GR, false, 2, 512><<<g, T, 0, st>>>(a);
                else if (p.V == 2) k_norm_rows<DT, WF, FMT, GR, false, 2, 1024><<<g, T, 0, st>>>(a);
                else k_norm_rows<DT, WF, FMT, GR, false, 4, 1024><<<g, T, 0, st>>>(a);
            });
        });
    }
};

template <int DT> void norm_bwd(bool wf32, const NormBwdArgs& a, hipStream_t st) {
    constexpr int VE = LaneVE<DT>::value;
    const NormPlan p = norm_bwd_plan(a.rows, ((int64_t)a.cols + VE - 1) / VE);
    const unsigned g = (unsigned)p.groups;
    with_bool(wf32 && DT != kF32, [&](auto W) {
        constexpr bool WF = decltype(W)::value;
        const int T = p.threads;
        if (p.V == 0) k_norm_bwd_long<DT, WF><<<g, T, 0, st>>>(a);
        else if (p.V == 1) k_norm_bwd<DT, WF, 1, 256><<<g, T, 0, st>>>(a);
        else if (T <= 512) k_norm_bwd<DT, WF, 2, 512><<<g, T, 0, st>>>(a);
        else k_norm_bwd<DT, WF, 2, 1024><<<g, T, 0, st>>>(a);
    });
}

}  // namespace

void launch_rmsnorm_cast(bool group, const void* x, int dt, const void* res, const void* w, int wdt, int64_t rows,
                         int64_t cols, float eps, int fmt, uint8_t* q, float* sinv, void* h, float* rstd,
                         hipStream_t st) {
    const NormArgs a{x, res, w, rows, (int)cols, eps, q, sinv, h, rstd};
    dispatch_dt_fmt<NormCast>(dt, fmt, group, wdt == kF32, a, st);
}

int64_t rmsnorm_bwd_parts(int64_t rows) { return norm_bwd_parts(rows); }

void launch_rmsnorm_bwd(const void* dy, const void* h, int dt, const void* w, int wdt, const float* rstd,
                        const void* dh, int64_t rows, int64_t cols, void* dx, void* dw, float* ws, hipStream_t st) {
    const int64_t parts = rmsnorm_bwd_parts(rows);
    const NormBwdArgs a{dy, h, w, rstd, dh, rows, (int)cols, dx, dw ? ws : nullptr};
    if (dt == kF32) norm_bwd<kF32>(wdt == kF32, a, st);
    else if (dt == kBF16) norm_bwd<kBF16>(wdt == kF32, a, st);
    else norm_bwd<kF16>(wdt == kF32, a, st);
    if (!dw) return;
    const unsigned gc = grid((cols + 31) / 32);            // 1024 threads each: a grid holds fewer than 2^32
    if (wdt == kF32) k_norm_dw<kF32><<<gc, 1024, 0, st>>>(ws, parts, (int)cols, dw);
    else if (wdt == kBF16) k_norm_dw<kBF16><<<gc, 1024, 0, st>>>(ws, parts, (int)cols, dw);
    else k_norm_dw<kF16><<<gc, 1024, 0, st>>>(ws, parts, (int)cols, dw);
}

}  // namespace fp8q
