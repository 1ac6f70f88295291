// fp8q_mm_fwd.hip -- the forward products on fp8 operands: one projection, or
// the gate and up projections with the activation and their product (and the
// group cast of it) in the same kernel.
//
//   y[m, n] = sum_kb xs[m, kb] ws[n/128, kb] sum_{k in kb} x[m, k] w[n, k]
//
// Many rows: bound by the matrix cores (k_mm).  Few rows: bound by the
// weights' bytes (k_mm_rows), whose sums are binary32 throughout.
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
        if constexpr (EX)
#pragma unroll
            for (int n = 0; n < 4; ++n) widen_codes<WF>(b[n], bw[n]);
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
            if constexpr (EX) {
                v4i xw[4];
                widen_codes<XF>(x[t], xw);
#pragma unroll
                for (int n = 0; n < 4; ++n) r[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < 4; ++n) r[n] = mfma_bf16(bw[n][k], xw[k], r[n]);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) r[n] = mfma_fp8<WF, XF>(b[n], x[t]);
            }
            if constexpr (decltype(NEXT)::value && BLATE)
                if (t == MT - 1) read_b(b, smem + nbuf * L::kStage);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float f = n < 2 ? f0 : f1;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][n][i] = __builtin_fmaf(r[n][i], f, acc[t][n][i]);
            }
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
        float p[MT][8];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int64_t row = m0 + wm * (BM / 2) + t * 16 + col;
            float g[8], u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] = acc[t][k >> 2][k & 3];
                u[k] = acc[t][2 + (k >> 2)][k & 3];
                p[t][k] = act_value(a.act, g[k]) * u[k];
            }
            if (row < a.M) {
                if (a.z) {
                    put8(a.z, a.zdt, row, 2 * (int64_t)a.N, nc, a.N, a.vec_z, g);
                    put8((char*)a.z + (int64_t)a.N * (a.zdt == kF32 ? 4 : 2), a.zdt, row, 2 * (int64_t)a.N, nc, a.N,
                         a.vec_z, u);
                }
                if (a.y) put8(a.y, a.ydt, row, a.N, nc, a.N, a.vec_y, p[t]);
            }
        }
        if (a.q) {
            __syncthreads();                               // the last stage's reads are done; LDS is free
            cast_tile<BM, MT>(a, p, (uint32_t*)smem, m0, n0, wm, wn, lane);
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
// then the epilogue.  With cast, p goes to pbuf in binary32 and the group cast
// follows as its own launch.
struct JoinArgs {
    const float* part;
    int splits;
    int64_t M;
    int N, gated, act;
    void* y;
    int ydt;
    float* pbuf;
    void* z;
    int zdt;
};

__device__ __forceinline__ void put1(void* y, int dt, int64_t e, float v) {
    if (dt == kF32) store1<kF32>(y, e, v);
    else if (dt == kBF16) store1<kBF16>(y, e, v);
    else store1<kF16>(y, e, v);
}

__global__ void __launch_bounds__(256) k_mm_join(JoinArgs a) {
    const int64_t total = a.M * a.N, W = a.gated ? 2 * (int64_t)a.N : a.N, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t m = i / a.N, n = i - m * a.N;
        const float* p = a.part + m * W + n;
        float g = 0.0f, u = 0.0f;
        for (int s = 0; s < a.splits; ++s) {
            g += p[(int64_t)s * a.M * W];
            if (a.gated) u += p[(int64_t)s * a.M * W + a.N];
        }
        float v = g;
        if (a.gated) {
            if (a.z) {
                put1(a.z, a.zdt, m * W + n, g);
                put1(a.z, a.zdt, m * W + a.N + n, u);
            }
            v = act_value(a.act, g) * u;
        }
        if (a.pbuf) a.pbuf[i] = v;
        else put1(a.y, a.ydt, i, v);
    }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// A workgroup of 8 waves owns 16 NT rows of the weights (of each of the two
// for a gated pair) and all of the rows of X (16 MT of them); its waves take
// every 8th block of K each, straight from memory to registers: nothing is
// read twice by a workgroup, and the eight waves' loads cover 1 KB runs of
// each weight row.  The waves' sums meet in LDS in a fixed order.
template <int XF, int WF, int MT, int NT, bool GATED, int NW>
__global__ void __launch_bounds__(64 * NW) k_mm_rows(FwdArgs a, float* pbuf) {
    constexpr int H = GATED ? 2 : 1, BT = NT * H;           // MFMA tiles of weights a wave holds
    __shared__ __attribute__((aligned(16))) float red[NW][BT][MT][64][4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, lr = lane >> 4;
    const int n0 = (int)blockIdx.x * 16 * NT;
    const int64_t pitch = (int64_t)a.KB * 128;

    const uint8_t* wp[BT];
#pragma unroll
    for (int j = 0; j < BT; ++j) {
        const int n = min(n0 + (j % NT) * 16 + col, a.N - 1);
        wp[j] = (j < NT ? a.w0 : a.w1) + n * pitch + lr * 16;
    }
    const uint8_t* xp[MT];
    const float* sp[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = min((int64_t)(t * 16 + col), a.M - 1);
        xp[t] = a.x + m * pitch + lr * 16;
        sp[t] = a.xs + m * a.KB;
    }
    const float* s0 = a.ws0 + (int64_t)(n0 >> 7) * a.KB;    // 16 NT divides 128: one block row a workgroup
    const float* s1 = GATED ? a.ws1 + (int64_t)(n0 >> 7) * a.KB : s0;

    v4f acc[BT][MT];
#pragma unroll
    for (int j = 0; j < BT; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[j][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    struct Block {
        v8i w[BT], x[MT];
        float sx[MT];
    };
    auto load = [&](Block& b, int kb) {
#pragma unroll
        for (int j = 0; j < BT; ++j) b.w[j] = frag_nt((const char*)wp[j] + kb * 128, (const char*)wp[j] + kb * 128 + 64);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            b.x[t] = frag((const char*)xp[t] + kb * 128, (const char*)xp[t] + kb * 128 + 64);
            b.sx[t] = sp[t][kb];
        }
    };
    auto mul = [&](const Block& b, int kb) {
        const float f0 = s0[kb], f1 = s1[kb];
        v4i ww[BT][4];
#pragma unroll
        for (int j = 0; j < BT; ++j) widen_codes<WF>(b.w[j], ww[j]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            v4i xw[4];
            widen_codes<XF>(b.x[t], xw);
            v4f r[BT];
#pragma unroll
            for (int j = 0; j < BT; ++j) r[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < BT; ++j) r[j] = mfma_bf16(ww[j][k], xw[k], r[j]);
#pragma unroll
            for (int j = 0; j < BT; ++j) {
                const float f = b.sx[t] * (j < NT ? f0 : f1);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][t][i] = __builtin_fmaf(r[j][i], f, acc[j][t][i]);
            }
        }
    };
    for (int kb = wave; kb < a.KB; kb += NW) {
        Block b;
        load(b, kb);
        mul(b, kb);
    }
#pragma unroll
    for (int j = 0; j < BT; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) *(v4f*)red[wave][j][t][lane] = acc[j][t];
    __syncthreads();
    // outputs: NT x MT tiles of 16 x 16; n fastest
    for (int i = threadIdx.x; i < NT * MT * 256; i += 64 * NW) {
        const int nl = i % (NT * 16), m = i / (NT * 16);
        const int j = nl >> 4, n = n0 + nl;
        if (m >= a.M || n >= a.N) continue;
        const int l = (m & 15) + ((nl & 15) >> 2) * 16, e = nl & 3, t = m >> 4;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            g += red[w][j][t][l][e];
            if constexpr (GATED) u += red[w][NT * (H - 1) + j][t][l][e];
        }
        float v = g;
        if constexpr (GATED) {
            if (a.z) {
                const int64_t at = m * 2 * (int64_t)a.N + n;
                put1(a.z, a.zdt, at, g);
                put1(a.z, a.zdt, at + a.N, u);
            }
            v = act_value(a.act, g) * u;
        }
        const int64_t at = m * (int64_t)a.N + n;
        if (pbuf) pbuf[at] = v;
        else put1(a.y, a.ydt, at, v);
    }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

constexpr int64_t kRowsMax = 64;       // rows that k_mm_rows takes
constexpr int NTV = 2, NWV = 16;

// How a product is tiled: rows a tile, and workgroups over K (splits)
struct Plan {
    bool rows;
    int bm, splits, kper;
    int64_t tm, tn;
};

// ex: binary32 sums (k_mm's EX), whose tiles are at most 128 rows tall: the
// widened fragments leave registers for no more
Plan plan(int64_t M, int64_t N, int64_t K, bool gated, bool ex) {
    Plan p{};
    const int64_t KB = K / 128;
    if (M <= kRowsMax) {
        p.rows = true;
        p.splits = 1;
        return p;
    }
    p.tn = (N + (gated ? 127 : 255)) / (gated ? 128 : 256);
    // the tallest tile that still gives most CUs one; below that, K is split
    p.bm = ex ? 128 : 256;
    while (p.bm > 64 && (M + p.bm - 1) / p.bm * p.tn < 200) p.bm /= 2;
    p.tm = (M + p.bm - 1) / p.bm;
    const int64_t tiles = p.tm * p.tn;
    int64_t s = 1;
    while (tiles * s * 2 <= 256 && KB / (s * 2) >= 8) s *= 2;
    p.kper = (int)((KB + s - 1) / s);
    if (p.kper < 1) p.kper = 1;
    p.splits = (int)std::max<int64_t>(1, (KB + p.kper - 1) / p.kper);
    return p;
}

int64_t part_bytes(const Plan& p, int64_t M, int64_t N, bool gated) {
    return p.splits > 1 ? p.splits * M * N * (gated ? 8 : 4) : 0;
}
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

template <int XF, int WF> void run_rows(const FwdArgs& a, float* pbuf, bool gated, hipStream_t st) {
    auto go = [&](auto MTc, auto NTc, auto NWc) {
        constexpr int MT = decltype(MTc)::value, NT = decltype(NTc)::value, NW = decltype(NWc)::value;
        const unsigned g = (unsigned)((a.N + 16 * NT - 1) / (16 * NT));
        if (gated) k_mm_rows<XF, WF, MT, NT, true, NW><<<g, 64 * NW, 0, st>>>(a, pbuf);
        else k_mm_rows<XF, WF, MT, 2 * NT, false, NW><<<(g + 1) / 2, 64 * NW, 0, st>>>(a, pbuf);
    };
    if (a.M <= 16) go(KC<1>{}, KC<NTV>{}, KC<NWV>{});
    else if (a.M <= 32) go(KC<2>{}, KC<1>{}, KC<8>{});
    else go(KC<4>{}, KC<1>{}, KC<8>{});
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
        const int64_t pb = cast && (p.rows || p.splits > 1) ? M * N * 4 : 0;
        most = std::max(most, up256(part_bytes(p, M, N, gated)) + pb);
    }
    return most;
}

void launch_mm_fwd(const MmFwd& f, hipStream_t st) {
    const bool gated = f.gated;
    const bool ex = f.q || (f.y && f.ydt == kF32) || (f.z && f.zdt == kF32);
    const Plan p = plan(f.M, f.N, f.K, gated, ex);
    FwdArgs a{f.x, f.xs, f.w0, f.ws0, f.w1, f.ws1, f.M, f.N, f.K / 128, (uint32_t)p.tm, (uint32_t)p.tn, f.act,
              f.y, f.ydt, f.q, f.qfmt, f.sinv, f.z, f.zdt, 0, 0, gated, p.kper, nullptr};
    a.vec_y = f.N % 8 == 0 && (p.splits > 1 || al(f.y, 16));
    a.vec_z = f.N % 8 == 0 && al(f.z, 16);
    char* ws = (char*)f.ws;
    float* pbuf = nullptr;
    if (p.splits > 1) a.part = (float*)ws;
    if (f.q && (p.rows || p.splits > 1)) pbuf = (float*)(ws + up256(part_bytes(p, f.M, f.N, gated)));
    auto run = [&](auto X, auto W) {
        constexpr int XF = decltype(X)::value, WF = decltype(W)::value;
        if (p.rows) run_rows<XF, WF>(a, pbuf, gated, st);
        else run_tiles<XF, WF>(a, p, gated, ex, st);
    };
    if (f.xfmt == kE4M3) { if (f.wfmt == kE4M3) run(KC<0>{}, KC<0>{}); else run(KC<0>{}, KC<1>{}); }
    else { if (f.wfmt == kE4M3) run(KC<1>{}, KC<0>{}); else run(KC<1>{}, KC<1>{}); }
    if (p.splits > 1) {
        const JoinArgs j{a.part, p.splits, f.M, f.N, gated, f.act, f.y, f.ydt, pbuf, f.z, f.zdt};
        const int64_t n = (f.M * f.N + 255) / 256;
        k_mm_join<<<(unsigned)std::min<int64_t>(n, 4096), 256, 0, st>>>(j);
    }
    if (pbuf) launch_group128_cast(pbuf, kF32, f.M * (f.N / 128), f.qfmt, f.q, f.sinv, st);
}

}  // namespace fp8q
