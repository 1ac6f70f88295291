// fp8q_mm_fwd.hip -- the forward products on fp8 operands: one projection, or
// the gate and up projections with the activation and their product (and the
// group cast of it) in the same kernel.
//
//   y[m, n] = sum_kb xs[m, kb] ws[n/128, kb] sum_{k in kb} x[m, k] w[n, k]
//
// Many rows: bound by the matrix cores (k_mm).  Few rows: bound by the
// weights' bytes (k_mm_rows), whose sums are binary32 throughout.
#include "fp8q_ffn_plan.h"
#include "fp8q_host.h"
#include "fp8q_mm.h"

namespace fp8q {

namespace {

enum { kOutLinear = 0, kOutGated = 1, kOutPartial = 2 };

struct FwdArgs {
    const uint8_t* x;
    const float* xs;
    const uint8_t* w0;
    const float* ws0;
    const uint8_t* w1;
    const float* ws1;
    int64_t M;
    int N, KB;             // KB = K / 128
    uint32_t tm, tn;
    int act;
    void* y;
    int ydt;
    uint8_t* q;
    int qfmt;
    float* sinv;
    void* z;
    int zdt;
    int vec_y, vec_z, gated, kper;
    float* part;           // [splits][M][gated ? 2 N : N]
};

// LDS of one step: the tiles, then 64 floats a wave: the scales of BM / 8
// rows of A and, in the last two, of the halves of B
template <int BM> struct FwdLds {
    static constexpr int kS = (BM + kMmBN) * 128;
    static constexpr int kStage = kS + 8 * 256;
    static constexpr int kStages = BM == 256 ? 2 : 3;
    static constexpr int kPer = BM / 64 + 4 + 1;            // loads a wave issues for a step
};

// group-cast epilogue: the amax of a token's 128 columns is over a lane's 8
// values, the 4 lane rows and the 4 waves of the token's wave row
template <int BM, int MT> __device__ __forceinline__ void cast_tile(const FwdArgs& a, float (&p)[MT][8], uint32_t* lds,
                                                                    int64_t m0, int n0, int wm, int wn, int lane) {
    const int col = lane & 15, lr = lane >> 4;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = umax(m, __float_as_uint(p[t][k]) & 0x7FFFFFFFu);
        m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (lr == 0) lds[wn * BM + wm * (BM / 2) + t * 16 + col] = m;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int r = wm * (BM / 2) + t * 16 + col;
        uint32_t m = umax(umax(lds[r], lds[BM + r]), umax(lds[2 * BM + r], lds[3 * BM + r]));
        m = umax(m, 0x38D1B717u);                           // the group cast's 1e-4 clamp
        const float am = __uint_as_float(m);
        const int64_t row = m0 + r;
        if (row >= a.M) continue;
        const float mx = a.qfmt == kE4M3 ? Fp8Fmt<kE4M3>::max : Fp8Fmt<kE5M2>::max;
        const float sc = mx / am;
        if (wn == 0 && lr == 0) a.sinv[row * (a.N >> 7) + (n0 >> 7)] = am / mx;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p[t][k] * sc;
        v2u o;
        if (a.qfmt == kE4M3) o = v2u{enc4<kE4M3>(v[0], v[1], v[2], v[3]), enc4<kE4M3>(v[4], v[5], v[6], v[7])};
        else o = v2u{enc4<kE5M2>(v[0], v[1], v[2], v[3]), enc4<kE5M2>(v[4], v[5], v[6], v[7])};
        uint8_t* d = a.q + row * a.N + n0 + wn * 32 + lr * 8;
        if (((uintptr_t)a.q & 3) == 0) st8<false>(d, o);
        else
            for (int k = 0; k < 8; ++k) d[k] = (uint8_t)((k < 4 ? o.x : o.y) >> (8 * (k & 3)));
    }
}

// EX: binary32 sums of the codes as bf16; else the fp8 instruction
template <int XF, int WF, int BM, int OUT, bool EX> __global__ void __launch_bounds__(kMmThreads, 2) k_mm(FwdArgs a) {
    using L = FwdLds<BM>;
    constexpr int MT = BM / 32;
    __shared__ __attribute__((aligned(1024))) char smem[L::kStages * L::kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    uint32_t im, in;
    tile_of(blockIdx.x, a.tm, a.tn, &im, &in);
    const int64_t m0 = (int64_t)im * BM;
    const bool gated = OUT == kOutGated || (OUT == kOutPartial && a.gated);
    const int n0 = (int)in * (gated ? 128 : 256);
    const int n1 = gated ? n0 : n0 + 128;

    const int kb0 = OUT == kOutPartial ? (int)blockIdx.y * a.kper : 0;
    const int kb1 = OUT == kOutPartial ? min(a.KB, kb0 + a.kper) : a.KB;

    TileLoad<BM> ld;
    ld.init(a.x, m0, a.M, a.w0, gated ? a.w1 : a.w0, n0, n1, a.N, a.N, (int64_t)a.KB * 128, wave, lane);
    const uint32_t lds0 = lds_offset(smem);
    // Scales through LDS like the tiles (a load into a register inside the
    // loop would wait for every tile load issued before it): lanes below BM / 8
    // bring the wave's rows of A, the last two the halves of B.
    const float* sp;
    if (lane < 62) {
        int64_t r = wave * (BM / 8) + (lane < BM / 8 ? lane : 0);
        if (r > a.M - 1 - m0) r = a.M - 1 - m0;
        sp = a.xs + (m0 + r) * a.KB;
    } else {
        sp = lane == 62 ? a.ws0 + (int64_t)(n0 >> 7) * a.KB
                        : (gated ? a.ws1 : a.ws0) + (int64_t)(min(n1, a.N - 1) >> 7) * a.KB;
    }
    auto issue = [&](int kb, int buf) {
        const uint32_t s = lds0 + buf * L::kStage;
        ld.issue(s, kb);
        lds_dma4_at(s + L::kS + wave * 256, sp + kb);
    };

    v4f acc[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[t][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const int col = lane & 15, lr = lane >> 4;
    const uint32_t c0 = (uint32_t)((lr ^ (col & 7)) * 16), c1 = (uint32_t)(((lr + 4) ^ (col & 7)) * 16);
    const uint32_t ra = (uint32_t)((wm * (BM / 2) + col) * 128), rb = (uint32_t)((BM + wn * 32 + col) * 128);
    // row r of A: scale r % (BM / 8) of wave r / (BM / 8)
    const uint32_t rs = (uint32_t)(L::kS + wm * 1024 + (BM == 64 ? (col >> 3) * 256 + (col & 7) * 4 : col * 4));
    auto scale_at = [&](int t) { return rs + (BM == 256 ? (t >> 1) * 256 + (t & 1) * 64 : t * (BM == 128 ? 256 : 512)); };

    // A step reads its fragments PF row tiles ahead of their MFMAs.  Its
    // barrier comes when the last of them are in registers: the step's buffer
    // is free then and takes the tiles of the step ST later, and the first
    // fragments of the next step are read behind the step's last MFMAs.
    // The tallest tile has no registers for the next B beside its own, and reads
    // it after the step's last MFMA.
    constexpr int ST = L::kStages, PF = MT >= 4 ? 2 : 1;
    constexpr bool BLATE = BM == 256;
    v8i b[4], bn[4], x[MT + PF];                            // x[MT ..): the next step's first
    auto read_b = [&](v8i (&d)[4], const char* s) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const char* p = s + rb + (n >> 1) * (128 * 128) + (n & 1) * (16 * 128);
            d[n] = frag(p + c0, p + c1);
        }
    };
    auto read_x = [&](const char* s, int t) { return frag(s + ra + t * (16 * 128) + c0, s + ra + t * (16 * 128) + c1); };
    int buf = 0;
    auto step = [&](int kb, auto NEXT, auto LOAD) {
        const char* s = smem + buf * L::kStage;
        const int nbuf = buf + 1 == ST ? 0 : buf + 1;
        float sx[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) sx[t] = *(const float*)(s + scale_at(t));
        const float s0 = *(const float*)(s + L::kS + 62 * 4), s1 = *(const float*)(s + L::kS + 63 * 4);
        v4i bw[4][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (t + PF < MT) x[t + PF] = read_x(s, t + PF);
            if (t == MT - PF) {
                if constexpr (decltype(LOAD)::value) dma_wait<(ST - 2) * L::kPer>();
                else dma_wait<0>();
                wg_barrier();
                if constexpr (decltype(LOAD)::value) issue(kb + ST, buf);
                if constexpr (decltype(NEXT)::value && !BLATE) read_b(bn, smem + nbuf * L::kStage);
            }
            if constexpr (decltype(NEXT)::value)
                if (t >= MT - PF) x[t + PF] = read_x(smem + nbuf * L::kStage, t + PF - MT);
            const float f0 = sx[t] * s0, f1 = sx[t] * s1;
            v4f r[4];
            auto add = [&](int n) {
                const float f = n < 2 ? f0 : f1;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][n][i] = __builtin_fmaf(r[n][i], f, acc[t][n][i]);
            };
            if constexpr (EX) {
                v4i xw[4];
                widen_codes<XF>(x[t], xw);
#pragma unroll
                for (int n = 0; n < 4; ++n) r[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                if (t == 0) {
                    // each column tile is widened when its MFMAs come, so that
                    // they start before all four are
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        widen_codes<WF>(b[n], bw[n]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) r[n] = mfma_bf16(bw[n][k], xw[k], r[n]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int n = 0; n < 4; ++n) r[n] = mfma_bf16(bw[n][k], xw[k], r[n]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) r[n] = mfma_fp8<WF, XF>(b[n], x[t]);
            }
            if constexpr (decltype(NEXT)::value && BLATE)
                if (t == MT - 1) read_b(b, smem + nbuf * L::kStage);
#pragma unroll
            for (int n = 0; n < 4; ++n) add(n);
        }
        if constexpr (decltype(NEXT)::value) {
            if constexpr (!BLATE)
#pragma unroll
                for (int n = 0; n < 4; ++n) b[n] = bn[n];
#pragma unroll
            for (int t = 0; t < PF; ++t) x[t] = x[MT + t];
        }
        buf = nbuf;
    };
    if (kb0 < kb1) {
        const int first = min(ST, kb1 - kb0);
        for (int i = 0; i < first; ++i) issue(kb0 + i, i);
        if (first == ST) dma_wait<(ST - 1) * L::kPer>();
        else dma_wait<0>();
        wg_barrier();
        read_b(b, smem);
#pragma unroll
        for (int t = 0; t < PF; ++t) x[t] = read_x(smem, t);
        int kb = kb0;
        for (; kb < kb1 - ST; ++kb) step(kb, std::true_type{}, std::true_type{});
        for (; kb < kb1 - 1; ++kb) step(kb, std::true_type{}, std::false_type{});
        step(kb, std::false_type{}, std::false_type{});
    }

    const int nc = n0 + wn * 32 + lr * 8;                  // this lane's 8 columns of the first half
    if constexpr (OUT == kOutGated) {
        if (a.z) {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t row = m0 + wm * (BM / 2) + t * 16 + col;
                if (row >= a.M) continue;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = acc[t][2 * half + (k >> 2)][k & 3];
                    put8((char*)a.z + half * (int64_t)a.N * (a.zdt == kF32 ? 4 : 2), a.zdt, row, 2 * (int64_t)a.N, nc,
                         a.N, a.vec_z, v);
                }
            }
        }
        // A loop for each activation: one body of all three is past what is unrolled.
        // The 256-row tile spills 33 registers around it, to the GELU's constants,
        // and none inside the loop above.
        with_act(a.act, [&](auto A) {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float g = acc[t][k >> 2][k & 3], u = acc[t][2 + (k >> 2)][k & 3];
                    acc[t][k >> 2][k & 3] = gated_value<decltype(A)::value>(g, u);
                }
                __builtin_amdgcn_sched_barrier(0);         // no registers for more than one row tile's exps at once
            }
        });
        float p[MT][8];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k) p[t][k] = acc[t][k >> 2][k & 3];
        if (a.y) {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t row = m0 + wm * (BM / 2) + t * 16 + col;
                if (row < a.M) put8(a.y, a.ydt, row, a.N, nc, a.N, a.vec_y, p[t]);
            }
        }
        if constexpr (EX) {                                // a cast's sums are binary32
            if (a.q) {
                __syncthreads();                           // the last stage's reads are done; LDS is free
                cast_tile<BM, MT>(a, p, (uint32_t*)smem, m0, n0, wm, wn, lane);
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int64_t row = m0 + wm * (BM / 2) + t * 16 + col;
            if (row >= a.M) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = acc[t][2 * half + (k >> 2)][k & 3];
                if constexpr (OUT == kOutLinear) {
                    put8(a.y, a.ydt, row, a.N, nc + half * 128, a.N, a.vec_y, v);
                } else {
                    const int64_t W = a.gated ? 2 * (int64_t)a.N : a.N;
                    float* pt = a.part + (int64_t)blockIdx.y * a.M * W;
                    if (a.gated) put8(pt + half * (int64_t)a.N, kF32, row, W, nc, a.N, a.vec_y, v);
                    else put8(pt, kF32, row, W, nc + half * 128, a.N, a.vec_y, v);
                }
            }
        }
    }
}

// The end of a split product: the partial sums of every output, in order,
// then the epilogue.  A thread takes V columns of a row (4 where the rows are
// whole vectors); with CAST, the 32 threads of a 128-group find its amax.
struct JoinArgs {
    const float* part;
    int splits;
    int64_t M;
    int N, gated, act;
    void* y;
    int ydt;
    void* z;
    int zdt;
    uint8_t* q;
    int qfmt;
    float* sinv;
};

__device__ __forceinline__ void put1(void* y, int dt, int64_t e, float v) {
    if (dt == kF32) store1<kF32>(y, e, v);
    else if (dt == kBF16) store1<kBF16>(y, e, v);
    else store1<kF16>(y, e, v);
}

template <int V, bool CAST> __global__ void __launch_bounds__(256) k_mm_join(JoinArgs a) {
    const int64_t W = a.gated ? 2 * (int64_t)a.N : a.N, per = a.N / V, total = a.M * per;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
        const int64_t m = i / per, n = (i - m * per) * V;
        const float* p = a.part + m * W + n;
        float g[V], u[V], v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = u[k] = 0.0f;
        for (int s = 0; s < a.splits; ++s, p += a.M * W) {
            if constexpr (V == 4) {
                const v4f x = *(const v4f*)p;
#pragma unroll
                for (int k = 0; k < 4; ++k) g[k] += x[k];
                if (a.gated) {
                    const v4f y = *(const v4f*)(p + a.N);
#pragma unroll
                    for (int k = 0; k < 4; ++k) u[k] += y[k];
                }
            } else {
                g[0] += p[0];
                if (a.gated) u[0] += p[a.N];
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = g[k];
        if (a.gated)
            with_act(a.act, [&](auto A) {
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = gated_value<decltype(A)::value>(g[k], u[k]);
            });
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (a.z) {
                put1(a.z, a.zdt, m * W + n + k, g[k]);
                put1(a.z, a.zdt, m * W + a.N + n + k, u[k]);
            }
            if (!CAST) put1(a.y, a.ydt, m * a.N + n + k, v[k]);
        }
        if constexpr (CAST) {                              // N % 128 == 0: whole groups of 32 threads
            uint32_t mx = 0;
#pragma unroll
            for (int k = 0; k < V; ++k) mx = umax(mx, __float_as_uint(v[k]) & 0x7FFFFFFFu);
            mx = umax(max_lanes<32>(mx), 0x38D1B717u);      // the group cast's 1e-4 clamp
            const float top = a.qfmt == kE4M3 ? Fp8Fmt<kE4M3>::max : Fp8Fmt<kE5M2>::max;
            const float sc = top / __uint_as_float(mx);
            if ((threadIdx.x & 31) == 0) a.sinv[i >> 5] = __uint_as_float(mx) / top;
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] *= sc;
            const uint32_t w = a.qfmt == kE4M3 ? enc4<kE4M3>(v[0], v[1 % V], v[2 % V], v[3 % V])
                                               : enc4<kE5M2>(v[0], v[1 % V], v[2 % V], v[3 % V]);
#pragma unroll
            for (int k = 0; k < V; ++k) a.q[m * a.N + n + k] = (uint8_t)(w >> (8 * k));
        }
    }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// Up to 16 rows of X: bound by the weights' bytes.  A workgroup takes tiles of
// 16 BT weight rows (8 BT columns of each projection of a gated pair: the gate
// in the first 8 rows of an MFMA tile, the up projection in the other 8), and
// its 8 waves every 8th block of K.  Each wave streams its blocks through a
// ring of D stages in LDS that is its own: whole 128-byte lines of each row,
// D - 1 stages in flight, no registers held and no barrier.  The ring runs on
// across tiles, so that the loads of the next tile are in flight while the
// waves' sums of this one meet in LDS, in a fixed order.
template <int MP, int BT> struct RowsLds {
    static constexpr int kX = BT * 2048, kS = kX + MP * 1024, kStage = kS + 256;
    static constexpr int kRed = 8 * BT * 1024;
    static constexpr int kStages = (160 * 1024 - kRed) / (8 * kStage) < 6 ? (160 * 1024 - kRed) / (8 * kStage) : 6;
    static constexpr int kPer = 2 * BT + MP + 1;
};

// MP: 8-row pieces of X (1 or 2)
template <int XF, int WF, int MP, int BT, bool GATED>
__global__ void __launch_bounds__(512) k_mm_rows(FwdArgs a, float* pbuf) {
    using L = RowsLds<MP, BT>;
    constexpr int D = L::kStages, C = GATED ? 8 * BT : 16 * BT;   // columns a tile
    __shared__ __attribute__((aligned(1024))) char smem[8 * D * L::kStage + L::kRed];
    float* red = (float*)(smem + 8 * D * L::kStage);              // [wave][tile][lane][4]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, lr = lane >> 4, sub = lane >> 3;
    const int64_t pitch = (int64_t)a.KB * 128;
    const int tiles = (a.N + C - 1) / C, nb = (a.KB + 7) / 8;
    char* ring = smem + wave * D * L::kStage;
    const uint32_t ring_lds = lds_offset(ring), off = (uint32_t)(((lane & 7) ^ sub) * 16);

    uint32_t vx[MP];
#pragma unroll
    for (int p = 0; p < MP; ++p) vx[p] = (uint32_t)(min((int64_t)(p * 8 + sub), a.M - 1) * pitch) + off;
    const float* sx = a.xs + min((int64_t)col, a.M - 1) * a.KB;

    // the next block to load: block `li` of tile `lt`.  A wave's blocks past
    // the end of K (and of the last tile) are loads of the last one again, so
    // that the count in flight is the same for all; they are not multiplied.
    int lt = blockIdx.x, li = 0;
    auto issue = [&](int stage) {
        const int n0 = lt * C, kb = min(wave + 8 * li, a.KB - 1);
        const uint32_t s = ring_lds + stage * L::kStage;
#pragma unroll
        for (int j = 0; j < BT; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int r = GATED ? 8 * j + sub : 16 * j + 8 * p + sub;
                const uint32_t v = (uint32_t)(min(r, a.N - 1 - n0) * pitch) + off;
                lds_dma16(s + j * 2048 + p * 1024, v, (GATED && p ? a.w1 : a.w0) + n0 * pitch + kb * 128);
            }
#pragma unroll
        for (int p = 0; p < MP; ++p) lds_dma16(s + L::kX + p * 1024, vx[p], a.x + kb * 128);
        const float* sp = lane < 62 ? sx : (GATED && lane == 63 ? a.ws1 : a.ws0) + (int64_t)(n0 >> 7) * a.KB;
        lds_dma4_at(s + L::kS, sp + kb);
        if (++li == nb) {
            li = 0;
            if (lt + (int)gridDim.x < tiles) lt += gridDim.x;
        }
    };
    if (a.KB > 0)
        for (int i = 0; i < D - 1; ++i) issue(i);
    int stage = 0;
    const uint32_t c0 = (uint32_t)((lr ^ (col & 7)) * 16), c1 = (uint32_t)(((lr + 4) ^ (col & 7)) * 16);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        v4f acc[BT];
#pragma unroll
        for (int j = 0; j < BT; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < nb; ++i) {
            issue(stage == 0 ? D - 1 : stage - 1);
            dma_wait<(D - 1) * L::kPer>();
            const char* s = ring + stage * L::kStage;
            v8i w[BT];
#pragma unroll
            for (int j = 0; j < BT; ++j) w[j] = frag(s + j * 2048 + col * 128 + c0, s + j * 2048 + col * 128 + c1);
            const char* px = s + L::kX + (MP == 1 ? col & 7 : col) * 128;
            const v8i x = frag(px + c0, px + c1);
            const float f = *(const float*)(s + L::kS + col * 4);
            const float f0 = f * *(const float*)(s + L::kS + 62 * 4), f1 = f * *(const float*)(s + L::kS + 63 * 4);
            v4i xw[4];
            widen_codes<XF>(x, xw);
            v4f r[BT];
#pragma unroll
            for (int j = 0; j < BT; ++j) {
                v4i ww[4];
                widen_codes<WF>(w[j], ww);
                r[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 4; ++k) r[j] = mfma_bf16(ww[k], xw[k], r[j]);
            }
            // rows 8 to 15 of a gated tile, the up projection's, are in the lanes from 32 on
            const float fl = GATED && lr >= 2 ? f1 : f0;
            if (wave + 8 * i < a.KB)
#pragma unroll
                for (int j = 0; j < BT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(r[j][e], fl, acc[j][e]);
            // this stage's reads are done before its next loads are issued
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            stage = stage + 1 == D ? 0 : stage + 1;
        }
#pragma unroll
        for (int j = 0; j < BT; ++j) *(v4f*)(red + ((wave * BT + j) * 64 + lane) * 4) = acc[j];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wg_barrier();
        for (int i = threadIdx.x; i < C * 16; i += 512) {
            const int nl = i % C, m = i / C, n = tile * C + nl;
            if (m >= a.M || n >= a.N) continue;
            const int j = GATED ? nl >> 3 : nl >> 4, row = GATED ? nl & 7 : nl & 15;
            const float* p = red + (j * 64 + m + (row >> 2) * 16) * 4 + (row & 3);
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                g += p[w * BT * 256];
                if constexpr (GATED) u += p[w * BT * 256 + 32 * 4];
            }
            float v = g;
            if constexpr (GATED) {
                if (a.z) {
                    const int64_t at = m * 2 * (int64_t)a.N + n;
                    put1(a.z, a.zdt, at, g);
                    put1(a.z, a.zdt, at + a.N, u);
                }
                with_act(a.act, [&](auto A) { v = gated_value<decltype(A)::value>(g, u); });
            }
            const int64_t at = m * (int64_t)a.N + n;
            if (pbuf) pbuf[at] = v;
            else put1(a.y, a.ydt, at, v);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wg_barrier();                                      // red is free for the next tile
    }
    dma_wait<0>();                                         // no load may land in LDS that is no longer ours
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

template <int XF, int WF> void run_rows(const FwdArgs& a, float* pbuf, bool gated, hipStream_t st) {
    // One or two MFMA tiles a workgroup tile: whichever spreads the weights
    // more evenly over 256 workgroups, and two where they are level (the rows
    // of X are read half as often).  One token through 18432 gated columns:
    // 45.1 us with one (9 rounds of 8 columns), 46.6 with two (5 of 16, the
    // last half empty); 16 rows through 7168 columns: 34.8 and 27.9.
    const int per = gated ? 8 : 16;
    auto rounds = [&](int bt) { return (((a.N + per * bt - 1) / (per * bt) + 255) / 256) * bt; };
    auto go = [&](auto MPc, auto BTc) {
        constexpr int MP = decltype(MPc)::value, BT = decltype(BTc)::value;
        const unsigned g = (unsigned)std::min((a.N + per * BT - 1) / (per * BT), 256);
        if (gated) k_mm_rows<XF, WF, MP, BT, true><<<g, 512, 0, st>>>(a, pbuf);
        else k_mm_rows<XF, WF, MP, BT, false><<<g, 512, 0, st>>>(a, pbuf);
    };
    auto rows = [&](auto MPc) {
        if (rounds(1) < rounds(2)) go(MPc, KC<1>{});
        else go(MPc, KC<2>{});
    };
    if (a.M <= 8) rows(KC<1>{});
    else rows(KC<2>{});
}

template <int XF, int WF> void run_tiles(const FwdArgs& a, const Plan& p, bool gated, bool ex, hipStream_t st) {
    auto go = [&](auto BMc, auto EXc) {
        constexpr int BM = decltype(BMc)::value;
        constexpr bool EX = decltype(EXc)::value;
        const dim3 g((unsigned)(p.tm * p.tn), (unsigned)p.splits);
        if (p.splits > 1) k_mm<XF, WF, BM, kOutPartial, EX><<<g, kMmThreads, 0, st>>>(a);
        else if (gated) k_mm<XF, WF, BM, kOutGated, EX><<<g, kMmThreads, 0, st>>>(a);
        else k_mm<XF, WF, BM, kOutLinear, EX><<<g, kMmThreads, 0, st>>>(a);
    };
    if (ex) {
        if (p.bm == 128) go(KC<128>{}, std::true_type{});
        else go(KC<64>{}, std::true_type{});
    } else {
        if (p.bm == 256) go(KC<256>{}, std::false_type{});
        else if (p.bm == 128) go(KC<128>{}, std::false_type{});
        else go(KC<64>{}, std::false_type{});
    }
}

}  // namespace

// enough for either kind of sum: the output types are not known here
int64_t mm_fwd_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool cast) {
    int64_t most = 0;
    for (int ex = cast ? 1 : 0; ex < 2; ++ex) {
        const Plan p = plan(M, N, K, gated, ex);
        const int64_t pb = cast && p.rows ? M * N * 4 : 0;
        most = std::max(most, up256(part_bytes(p, M, N, gated)) + pb);
    }
    return most;
}

void launch_mm_fwd(const MmFwd& f, hipStream_t st) {
    const bool gated = f.gated;
    const bool ex = f.M <= kExactMax || f.q || (f.y && f.ydt == kF32) || (f.z && f.zdt == kF32);
    const Plan p = plan(f.M, f.N, f.K, gated, ex);
    FwdArgs a{f.x, f.xs, f.w0, f.ws0, f.w1, f.ws1, f.M, f.N, f.K / 128, (uint32_t)p.tm, (uint32_t)p.tn, f.act,
              f.y, f.ydt, f.q, f.qfmt, f.sinv, f.z, f.zdt, 0, 0, gated, p.kper, nullptr};
    a.vec_y = f.N % 8 == 0 && (p.splits > 1 || al(f.y, 16));
    a.vec_z = f.N % 8 == 0 && al(f.z, 16);
    char* ws = (char*)f.ws;
    float* pbuf = nullptr;
    if (p.splits > 1) a.part = (float*)ws;
    if (f.q && p.rows) pbuf = (float*)ws;
    auto run = [&](auto X, auto W) {
        constexpr int XF = decltype(X)::value, WF = decltype(W)::value;
        if (p.rows) run_rows<XF, WF>(a, pbuf, gated, st);
        else run_tiles<XF, WF>(a, p, gated, ex, st);
    };
    if (f.xfmt == kE4M3) { if (f.wfmt == kE4M3) run(KC<0>{}, KC<0>{}); else run(KC<0>{}, KC<1>{}); }
    else { if (f.wfmt == kE4M3) run(KC<1>{}, KC<0>{}); else run(KC<1>{}, KC<1>{}); }
    if (p.splits > 1) {
        const JoinArgs j{a.part, p.splits, f.M, f.N, gated, f.act, f.y, f.ydt, f.z, f.zdt, f.q, f.qfmt, f.sinv};
        const int V = f.N % 4 == 0 ? 4 : 1;
        const unsigned g = (unsigned)std::min<int64_t>((f.M * (f.N / V) + 255) / 256, 4096);
        if (f.q) k_mm_join<4, true><<<g, 256, 0, st>>>(j);
        else if (V == 4) k_mm_join<4, false><<<g, 256, 0, st>>>(j);
        else k_mm_join<1, false><<<g, 256, 0, st>>>(j);
    }
    if (pbuf) launch_group128_cast(pbuf, kF32, f.M * (f.N / 128), f.qfmt, f.q, f.sinv, st);
}

}  // namespace fp8q
