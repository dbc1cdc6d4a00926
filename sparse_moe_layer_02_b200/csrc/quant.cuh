// Weights in 4 bits with group scales: conversion both ways, and products with few
// tokens (one matrix, or the experts of a layer).
//
// A matrix [M, K] is held as q, uint8 [M, K/2] (column 2j in the low, 2j+1 in the high
// four bits of byte j) and scales s, bf16 [K/G, M], G = 32, 64 or 128:
//     w(m, k) = (q(m, k) - 8) * s(k / G, m).
// The scales lie group by group, so a tile's scales are rows of consecutive m that
// TMA can fetch; the codes lie as they would in a checkpoint.
#pragma once

#include "common.cuh"
#include "dispatch.cuh"
#include "gemm_sm100.cuh"
#include "grouped.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// Conversion.  s = bf16(max|w| / 7) over the group, q = round(w / s) + 8 (half to
// even; -8..7).  One block takes 32 rows x 256 columns; a warp takes 4 rows, a lane 8
// columns of each, so a group is 4, 8 or 16 neighbouring lanes and its maximum two to
// four shuffles.  The block's scales pass through shared memory to be stored 64 bytes
// at a time.  Bound by memory: 2.5 bytes + 2/G per weight either way.
// ---------------------------------------------------------------------------
constexpr int QZ_ROWS = 32, QZ_COLS = 256, QZ_THREADS = 256;

__global__ void __launch_bounds__(QZ_THREADS) quantize_kernel(const __nv_bfloat16 *__restrict__ W,
                                                              uint8_t *__restrict__ q,
                                                              __nv_bfloat16 *__restrict__ s, int M, int K,
                                                              int G) {
    __shared__ __nv_bfloat16 ss[QZ_COLS / 32][QZ_ROWS];
    const int lane = lane_id(), warp = warp_id();
    const int k = blockIdx.x * QZ_COLS + lane * 8, m0 = blockIdx.y * QZ_ROWS;
    const size_t e = blockIdx.z;
    const int per = G >> 3; // lanes of a group
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + warp * 4 + i;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (m < M && k < K)
            v[i] = __ldcs(reinterpret_cast<const uint4 *>(W + (e * M + m) * (size_t)K + k));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + warp * 4 + i;
        float w[8];
        unpack_bf16x2(v[i].x, w[0], w[1]);
        unpack_bf16x2(v[i].y, w[2], w[3]);
        unpack_bf16x2(v[i].z, w[4], w[5]);
        unpack_bf16x2(v[i].w, w[6], w[7]);
        // The maximum of the magnitudes' bit patterns: a NaN is above infinity, so
        // neither is lost.
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(w[j]) & 0x7FFFFFFFu);
        for (int d = 1; d < per; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        __nv_bfloat16 sb = __float2bfloat16_rn(__uint_as_float(top) / 7.0f);
        if (top >= 0x7F800000u) sb = __ushort_as_bfloat16(0x7FFF); // not finite: every value NaN
        const float sf = __bfloat162float(sb);
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // s = 0 (all zero, or too small for bf16) and s = NaN take the code of 0
            const float t = sf > 0.f ? fminf(fmaxf(rintf(w[j] / sf), -8.f), 7.f) : 0.f;
            c |= (uint32_t)((int)t + 8) << (4 * j);
        }
        if (m < M && k < K) *reinterpret_cast<uint32_t *>(q + (e * M + m) * (size_t)(K / 2) + k / 2) = c;
        if ((lane & (per - 1)) == 0) ss[lane / per][warp * 4 + i] = sb;
    }
    __syncthreads();
    const int groups = QZ_COLS / G;
    const int g = threadIdx.x / QZ_ROWS, r = threadIdx.x % QZ_ROWS; // 8 groups at most
    const int kg = blockIdx.x * groups + g;
    if (g < groups && kg < K / G && m0 + r < M) s[(e * (K / G) + kg) * (size_t)M + m0 + r] = ss[g][r];
}

__global__ void __launch_bounds__(QZ_THREADS) dequantize_kernel(const uint8_t *__restrict__ q,
                                                                const __nv_bfloat16 *__restrict__ s,
                                                                __nv_bfloat16 *__restrict__ W, int M, int K,
                                                                int G) {
    __shared__ __nv_bfloat16 ss[QZ_COLS / 32][QZ_ROWS];
    const int lane = lane_id(), warp = warp_id();
    const int k = blockIdx.x * QZ_COLS + lane * 8, m0 = blockIdx.y * QZ_ROWS;
    const size_t e = blockIdx.z;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + warp * 4 + i;
        c[i] = 0;
        if (m < M && k < K)
            c[i] = __ldcs(reinterpret_cast<const uint32_t *>(q + (e * M + m) * (size_t)(K / 2) + k / 2));
    }
    const int groups = QZ_COLS / G;
    const int g = threadIdx.x / QZ_ROWS, r = threadIdx.x % QZ_ROWS;
    const int kg = blockIdx.x * groups + g;
    if (g < groups && kg < K / G && m0 + r < M) ss[g][r] = s[(e * (K / G) + kg) * (size_t)M + m0 + r];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + warp * 4 + i;
        if (m >= M || k >= K) continue;
        const float sf = __bfloat162float(ss[lane * 8 / G][warp * 4 + i]);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) // products of 4 and 8 bits are exact in fp32
            o[j] = pack_bf16x2((float)((int)((c[i] >> (8 * j)) & 15u) - 8) * sf,
                               (float)((int)((c[i] >> (8 * j + 4)) & 15u) - 8) * sf);
        *reinterpret_cast<uint4 *>(W + (e * M + m) * (size_t)K + k) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---------------------------------------------------------------------------
// Products y(n, m) = sum_k x(n, k) w(m, k) for few tokens n: bound by reading the
// codes, so each is read once per 8 NT tokens and becomes a bf16 integer in registers,
// exact, right where the MMA wants it:
//
// - A tile of R weight rows is the MMA's M side, the tokens its N side (m16n8k16).
//   The sum over k does not care about order, only that both operands use the same.
//   A thread's word holds columns k0..k7; (word >> 4i) & 0x000F000F puts columns i and
//   i+4 into the halves of a register, so the MMA's pairs are (0,4), (1,5), (2,6),
//   (3,7), and the tokens' registers are paired alike by four byte permutes.
// - A code c becomes bf16 by setting the exponent of 128 above it (128 + c, exact in 8
//   bits) and subtracting 136.  The group's sum of integers times tokens is fp32 in
//   the MMA; its scale is applied once per group, in fp32.
//
// tcgen05 would want the bf16 weights in shared memory first (four times the codes'
// bytes written and read again) and has nothing to gain: the tensor work is small here.
//
// A block is one producer warp and eight consumer warps: RG groups of 32 rows x KS
// slices of 64 columns (RG * KS = 8).  The producer fills a ring: codes and scales by
// TMA, the tokens' rows by 16-byte asynchronous copies, which may come from anywhere
// (a routed token's row is fetched where it lies, without a gather pass) and are zero
// for absent tokens and columns past K.  At the end of a tile the KS partial sums are
// added in order through shared memory.  Two blocks share an SM.
// ---------------------------------------------------------------------------
enum QuantKind { QUANT_LINEAR = 0, QUANT_GATE_UP = 1, QUANT_DOWN = 2 };

constexpr int QM_THREADS = 288;
constexpr int QM_CONSUMERS = 256;
constexpr int QM_MAXE = 512;

template <int RG, int NT> struct QmCfg {
    static constexpr int KS = 8 / RG;
    static constexpr int R = 32 * RG;            // weight rows of a tile
    static constexpr int SK = 64 * KS;           // columns of a stage
    static constexpr int BOX = SK / 2 < 128 ? SK / 2 : 128; // bytes of a code box's row = swizzle span
    static constexpr int NBOX = SK / 2 / BOX;
    static constexpr int W_BYTES = R * SK / 2;   // 8 KiB
    static constexpr int S_BYTES = R * (SK / 32) * 2; // 1 KiB (G = 32; fewer for larger G)
    static constexpr int X_BYTES = NT * 8 * SK * 2;
    static constexpr int STAGE = W_BYTES + S_BYTES + X_BYTES;
    static constexpr int LD = R + 4;             // floats per token in the sums' buffer
    static constexpr int RED_BYTES = KS * 8 * NT * LD * 4;
    static constexpr int TAB_BYTES = 256 + (2 * QM_MAXE + 2) * 4;
    // two blocks per SM
    static constexpr int STAGES = (113 * 1024 - 1024 - RED_BYTES - TAB_BYTES) / STAGE;
    static constexpr int SMEM = 1024 + STAGES * STAGE + RED_BYTES + TAB_BYTES;
    static_assert(STAGES >= 2 && STAGES <= 15, "ring depth");
};

struct QuantArgs {
    const uint8_t *x;   // LINEAR: x; GATE_UP: x; DOWN: h of the routed rows
    const uint8_t *x_s; // shared tokens: GATE_UP x; DOWN h_sh
    int row_bytes, row_bytes_s;
    int N, E, k, G;
    int K, K_s;         // summed columns, routed / shared
    int ncols, ncols_s; // output columns (LINEAR M, GATE_UP d, DOWN D), routed / shared
    int nb, nb_s;       // row tiles
    int direct;         // one token: pair j is expert topk_idx[j]'s only row
    const int32_t *topk_idx;
    const float *topk_w;
    const int32_t *tile_off, *counts, *perm_tok; // dispatch tables (tiles of 8 NT rows)
    const float *w_perm;
    void *out;   // LINEAR y bf16; GATE_UP h bf16; DOWN slot fp32
    void *out_s; // GATE_UP h_sh bf16; DOWN osh fp32
    float gate_max, up_max;
    uint64_t wait_limit_ns;
};

struct QuantTile {
    bool shared;
    int e;    // expert of the weight map (0 for LINEAR and the shared expert)
    int row0; // first token row (LINEAR, shared: token; routed: permuted row)
    int cnt;  // tokens, at most 8 NT
    int nb;   // row tile
};

// Tile t; false where it has no work (an id of no expert in direct mode).
template <int KIND, int TT>
__device__ __forceinline__ bool quant_tile(int t, int routed, const QuantArgs &a, const int *s_tile,
                                           const int *s_cnt, QuantTile &c) {
    if (KIND == QUANT_LINEAR || t >= routed) {
        // token tiles of one row tile are neighbours: the codes are in L2 for the second
        const int l = KIND == QUANT_LINEAR ? t : t - routed;
        const int tt = (a.N + TT - 1) / TT;
        c.shared = KIND != QUANT_LINEAR;
        c.e = 0;
        c.nb = l / tt;
        c.row0 = (l - c.nb * tt) * TT;
        c.cnt = min(TT, a.N - c.row0);
        return true;
    }
    c.shared = false;
    if (a.direct) {
        const int p = t / a.nb;
        c.nb = t - p * a.nb;
        c.e = s_tile[p];
        c.row0 = p;
        c.cnt = 1;
        return c.e >= 0 && c.e < a.E;
    }
    c.e = find_expert(s_tile, a.E, a.nb, t);
    const int mt = s_tile[c.e + 1] - s_tile[c.e], l = t - s_tile[c.e] * a.nb;
    c.nb = l / mt;
    const int tt = l - c.nb * mt;
    c.row0 = (s_tile[c.e] + tt) * TT;
    c.cnt = min(TT, s_cnt[c.e] - tt * TT);
    return true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
// This thread's arrival on `bar` once its earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes i and i+4 of a word as the bf16 integers -8..7.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w, int i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u; // 128 + code
    const __nv_bfloat162 o =
        __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                __nv_bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308))); // - 136
    return *reinterpret_cast<const uint32_t *>(&o);
}

// Maps: mW codes [E, M, K/2] bytes, box BOX x R/2 x 1, swizzled; mS scales
// [E, K/G, M], box R/2 x SK/G x 1; the same of the shared expert (GATE_UP: its gate and
// up rows stacked).
template <int KIND, int RG, int NT>
__global__ void __launch_bounds__(QM_THREADS, 2)
    quant_product_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mS,
                         const __grid_constant__ CUtensorMap mW_s, const __grid_constant__ CUtensorMap mS_s,
                         const QuantArgs a) {
    using C = QmCfg<RG, NT>;
    constexpr int TT = 8 * NT, KS = C::KS, SK = C::SK, R = C::R, HALF = R / 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // ring: codes of all stages first (1024-byte aligned), then scales, then tokens
    uint8_t *ring_w = smem;
    uint8_t *ring_s = ring_w + C::STAGES * C::W_BYTES;
    uint8_t *ring_x = ring_s + C::STAGES * C::S_BYTES;
    float *red = reinterpret_cast<float *>(ring_x + C::STAGES * C::X_BYTES);
    uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(red) + C::RED_BYTES);
    uint64_t *empty = full + C::STAGES;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(empty + C::STAGES);
    int *s_tile = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(full) + 256);
    int *s_cnt = s_tile + QM_MAXE + 1;

    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 33); // the TMA issuer and 32 lanes' copies
            mbar_init(&empty[s], 8);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mW);
        tma_prefetch_desc(&mS);
        if (KIND != QUANT_LINEAR) {
            tma_prefetch_desc(&mW_s);
            tma_prefetch_desc(&mS_s);
        }
    }
    // Nothing above touches global memory; all that follows comes after the previous
    // kernel of the stream.
    grid_dep_wait();
    grid_dep_launch_dependents();
    int routed = 0;
    if (KIND != QUANT_LINEAR) {
        if (a.direct) {
            if (threadIdx.x < a.k) s_tile[threadIdx.x] = a.topk_idx[threadIdx.x];
        } else {
            for (int i = threadIdx.x; i <= a.E; i += QM_THREADS) {
                s_tile[i] = a.tile_off[i];
                if (i < a.E) s_cnt[i] = a.counts[i];
            }
        }
    }
    __syncthreads();
    if (KIND != QUANT_LINEAR) {
        routed = (a.direct ? a.k : s_tile[a.E]) * a.nb;
        if (KIND == QUANT_GATE_UP && a.direct && blockIdx.x == 0 && threadIdx.x < a.k &&
            (s_tile[threadIdx.x] < 0 || s_tile[threadIdx.x] > a.E))
            record_error(DEV_BAD_INDEX, 400);
    }
    const int tts = (a.N + TT - 1) / TT;
    const int total = KIND == QUANT_LINEAR ? a.nb * tts : routed + a.nb_s * tts;
    const int gps = SK / a.G; // groups of a stage
    const uint64_t limit = a.wait_limit_ns;

    if (warp == 8) {
        // ------------------------------ producer ------------------------------
        const int tok = lane >> 2, ch = lane & 3; // this lane's token and 8 columns of 32
        const uint32_t stage_bytes = C::W_BYTES + 2 * HALF * gps * 2;
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            QuantTile c;
            if (!quant_tile<KIND, TT>(t, routed, a, s_tile, s_cnt, c)) continue;
            const int K = c.shared ? a.K_s : a.K;
            const int nt = (c.cnt + 7) >> 3;
            const uint8_t *base = c.shared ? a.x_s : a.x;
            const size_t rb = c.shared ? a.row_bytes_s : a.row_bytes;
            const uint8_t *src[NT];
            bool on[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int i = j * 8 + tok;
                on[j] = i < c.cnt;
                int row = c.row0 + (on[j] ? i : 0);
                if (KIND == QUANT_GATE_UP && !c.shared) row = a.direct ? 0 : a.perm_tok[row];
                src[j] = base + (size_t)row * rb + ch * 16;
            }
            const CUtensorMap *w = c.shared ? &mW_s : &mW, *sc = c.shared ? &mS_s : &mS;
            // the tile's two halves: consecutive rows, or gate rows and the up rows of
            // the same columns
            const int r0 = KIND == QUANT_GATE_UP ? c.nb * HALF : c.nb * R;
            const int r1 = KIND == QUANT_GATE_UP ? r0 + (c.shared ? a.ncols_s : a.ncols) : r0 + HALF;
            const int stages = (K + SK - 1) / SK;
            for (int i = 0; i < stages; ++i, ++it) {
                const uint32_t s = it % C::STAGES, ph = (it / C::STAGES) & 1;
                if (lane == 0) ok = mbar_wait(&empty[s], ph ^ 1, limit, abort_flag, 401);
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], stage_bytes);
                    uint8_t *dw = ring_w + s * C::W_BYTES;
#pragma unroll
                    for (int b = 0; b < C::NBOX; ++b) {
                        const int kx = i * (SK / 2) + b * C::BOX;
                        tma_load_3d(w, &full[s], dw + b * R * C::BOX, kx, r0, c.e);
                        tma_load_3d(w, &full[s], dw + (b * R + HALF) * C::BOX, kx, r1, c.e);
                    }
                    uint8_t *ds = ring_s + s * C::S_BYTES;
                    tma_load_3d(sc, &full[s], ds, r0, i * gps, c.e);
                    tma_load_3d(sc, &full[s], ds + C::S_BYTES / 2, r1, i * gps, c.e);
                }
                const uint32_t dx = smem_u32(ring_x + s * C::X_BYTES) + lane * 16;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (j >= nt) break;
#pragma unroll
                    for (int b = 0; b < SK / 32; ++b) {
                        const int kb = i * SK + b * 32; // K is a multiple of 32
                        const bool v = on[j] && kb < K;
                        cp_async16(dx + (j * (SK / 32) + b) * 512, v ? src[j] + (size_t)kb * 2 : base, v);
                    }
                }
                cp_async_arrive(&full[s]);
            }
        }
        if (!ok && lane == 0) {
            // Let copies already issued land before the block's memory goes away.
            const uint32_t first = it > C::STAGES ? it - C::STAGES : 0;
            for (uint32_t j = first; j < it; ++j) {
                volatile int no_abort = 0;
                mbar_wait(&full[j % C::STAGES], (j / C::STAGES) & 1, 10000000ull, &no_abort, 402);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------ consumers ------------------------------
        const int rg = warp / KS, ks = warp % KS;
        const int g = lane >> 2, t4 = lane & 3;
        // This lane's ldmatrix address: row mrow of an m16 tile, 16-byte chunk (32 columns)
        // of the slice, at the place the swizzle gives it (TMA xors the chunk with the
        // number of the 128-byte line: the row, or half the row for 64-byte rows).
        const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mch = lane >> 4;
        constexpr int CPR = C::BOX / 16;
        const int chunk = (ks * 2) % CPR + mch, box = ks * 2 / CPR;
        const int line = CPR == 8 ? lane & 7 : (lane & 7) >> 1;
        const uint32_t wbase =
            smem_u32(ring_w) + box * R * C::BOX + (uint32_t)(chunk ^ line) * 16;
        uint32_t woff[2], soff[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = rg * 32 + i * 16; // first row of the m16 tile in the tile
            woff[i] = (uint32_t)(row + mrow) * C::BOX; // halves lie one after the other
            soff[i] = (uint32_t)(row / HALF) * (C::S_BYTES / 2) + (uint32_t)(row % HALF) * 2;
        }
        const int ctid = threadIdx.x;
        uint32_t it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            QuantTile c;
            if (!quant_tile<KIND, TT>(t, routed, a, s_tile, s_cnt, c)) continue;
            const int K = c.shared ? a.K_s : a.K;
            const int nt = (c.cnt + 7) >> 3;
            const int stages = (K + SK - 1) / SK;
            float acc[2][NT][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.f;
            bool ok = true;
            for (int st = 0; st < stages; ++st, ++it) {
                const uint32_t s = it % C::STAGES, ph = (it / C::STAGES) & 1;
                ok = mbar_wait(&full[s], ph, limit, abort_flag, 411);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue; // abort: every wait fails at once, the walk stays matched
                uint32_t cw[2][4];
                ldmatrix_x4(wbase + s * C::W_BYTES + woff[0], cw[0]);
                ldmatrix_x4(wbase + s * C::W_BYTES + woff[1], cw[1]);
                const uint8_t *xs = ring_x + s * C::X_BYTES + (ks * 2) * 512 + lane * 16;
                const uint8_t *scs = ring_s + s * C::S_BYTES;
                float part[2][NT][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) { // 32 columns each
                    if (h == 0 || a.G == 32) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int r = 0; r < 4; ++r) part[i][j][r] = 0.f;
                    }
                    uint4 xv[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        if (j < nt)
                            xv[j] = *reinterpret_cast<const uint4 *>(xs + (j * (SK / 32) + h) * 512);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint32_t aw[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            aw[i][0] = codes_bf16x2(cw[i][2 * h], 2 * p);
                            aw[i][1] = codes_bf16x2(cw[i][2 * h + 1], 2 * p);
                            aw[i][2] = codes_bf16x2(cw[i][2 * h], 2 * p + 1);
                            aw[i][3] = codes_bf16x2(cw[i][2 * h + 1], 2 * p + 1);
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            if (j < nt) {
                                const uint32_t lo = p ? xv[j].y : xv[j].x, hi = p ? xv[j].w : xv[j].z;
                                const uint32_t b0 = __byte_perm(lo, hi, 0x5410);
                                const uint32_t b1 = __byte_perm(lo, hi, 0x7632);
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    mma_bf16(part[i][j], aw[i][0], aw[i][1], aw[i][2], aw[i][3], b0, b1);
                            }
                        }
                    }
                    if (h == 1 || a.G == 32) {
                        const int gi = (ks * 64 + h * 32) / a.G; // group in the stage
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const __nv_bfloat16 *sp =
                                reinterpret_cast<const __nv_bfloat16 *>(scs + soff[i]) + gi * HALF;
                            const float s0 = __bfloat162float(sp[g]), s1 = __bfloat162float(sp[g + 8]);
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                if (j < nt) {
                                    acc[i][j][0] = fmaf(s0, part[i][j][0], acc[i][j][0]);
                                    acc[i][j][1] = fmaf(s0, part[i][j][1], acc[i][j][1]);
                                    acc[i][j][2] = fmaf(s1, part[i][j][2], acc[i][j][2]);
                                    acc[i][j][3] = fmaf(s1, part[i][j][3], acc[i][j][3]);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
            }
            named_bar_sync(1, QM_CONSUMERS); // the last tile's sums have been read
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < nt) {
                        float *d = red + (ks * TT + j * 8 + 2 * t4) * C::LD + rg * 32 + i * 16 + g;
                        d[0] = acc[i][j][0];
                        d[C::LD] = acc[i][j][1];
                        d[8] = acc[i][j][2];
                        d[C::LD + 8] = acc[i][j][3];
                    }
            named_bar_sync(1, QM_CONSUMERS);
            if (!ok) continue;
            auto sum = [&](int tk, int row) {
                float v = red[tk * C::LD + row];
#pragma unroll
                for (int q = 1; q < KS; ++q) v += red[(q * TT + tk) * C::LD + row];
                return v;
            };
            const int nc = c.shared ? a.ncols_s : a.ncols;
            if (KIND == QUANT_GATE_UP) {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(c.shared ? a.out_s : a.out);
                for (int i = ctid; i < c.cnt * HALF; i += QM_CONSUMERS) {
                    const int tk = i / HALF, f = i % HALF, col = c.nb * HALF + f;
                    if (col < nc)
                        out[(size_t)(c.row0 + tk) * nc + col] = __float2bfloat16_rn(
                            swiglu_f(sum(tk, f), sum(tk, HALF + f), a.gate_max, a.up_max));
                }
            } else {
                for (int i = ctid; i < c.cnt * R; i += QM_CONSUMERS) {
                    const int tk = i / R, f = i % R, col = c.nb * R + f;
                    if (col >= nc) continue;
                    const size_t at = (size_t)(c.row0 + tk) * nc + col;
                    const float v = sum(tk, f);
                    if (KIND == QUANT_LINEAR)
                        static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
                    else if (c.shared)
                        static_cast<float *>(a.out_s)[at] = v;
                    else
                        static_cast<float *>(a.out)[at] =
                            v * (a.direct ? a.topk_w[c.row0] : a.w_perm[c.row0 + tk]);
                }
            }
        }
    }
}

// y(n) = the k weighted expert rows in slot order + the shared expert's row, fp32,
// rounded once.  One thread per 8 columns.
__global__ void __launch_bounds__(128) quant_combine_kernel(const QuantArgs a, const float *slot,
                                                            const float *osh, const int32_t *pos_of,
                                                            __nv_bfloat16 *y, int D) {
    grid_dep_wait();
    const int n = blockIdx.x, c = (blockIdx.y * 128 + threadIdx.x) * 8;
    if (c >= D) return;
    float v[8] = {};
    for (int j = 0; j < a.k; ++j) {
        int p;
        if (a.direct) {
            const int e = a.topk_idx[j];
            p = e >= 0 && e < a.E ? j : -1;
        } else {
            p = pos_of[(size_t)n * a.k + j];
        }
        if (p < 0) continue;
        const float4 *s = reinterpret_cast<const float4 *>(slot + (size_t)p * D + c);
        const float4 lo = __ldcg(s), hi = __ldcg(s + 1);
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
    }
    const float4 *o = reinterpret_cast<const float4 *>(osh + (size_t)n * D + c);
    const float4 lo = __ldcg(o), hi = __ldcg(o + 1);
    *reinterpret_cast<uint4 *>(y + (size_t)n * D + c) =
        make_uint4(pack_bf16x2(v[0] + lo.x, v[1] + lo.y), pack_bf16x2(v[2] + lo.z, v[3] + lo.w),
                   pack_bf16x2(v[4] + hi.x, v[5] + hi.y), pack_bf16x2(v[6] + hi.z, v[7] + hi.w));
}

}  // namespace moe
