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
// Conversion.  s = bf16(max|w| / 7) over the group, code = round(w / s) + 8 (half to
// even).  A warp takes rows of 256 columns, a lane 8 columns of each, so a group is 4, 8
// or 16 neighbouring lanes and its maximum two to four shuffles.  A block's scales pass
// through shared memory to be stored a row of them at a time.  Bound by memory: 2.5
// bytes + 2/G per weight either way; a warp keeps 4 rows (64 bytes a lane) in flight to
// quantize and 8 rows (32 bytes a lane) to dequantize.
//
// Both quotients are products with a reciprocal, and exact all the same.  max|w| / 7 is
// never nearer than 1/14 of a step to a tie of its rounding to bf16 (an 8-bit integer is
// no odd multiple of 7/2), the product within 2^-22 of it.  w / s is rounded to a multiple
// of 2^-12 on the way (the multiply-add with 1.5 * 2^11), then to an integer, half to
// even: w and s have 8-bit significands, so a quotient between 1/4 and 8 either is a
// multiple of 1/2 or lies at least 2^-11 away from every odd multiple of 1/2, while the
// product is within 2^-19 of the quotient.  |w / s| < 7.5 for scales that are normal
// numbers; below 2^-120, where s or 1/s is not, the code comes from the division and is
// clamped.  (With divisions and a mask and shift for each code the issue slots bound the
// kernel: 640 us for 32 x 4096 x 6144, 3.2 TB/s.)
// ---------------------------------------------------------------------------
constexpr int QZ_ROWS = 32, DQ_ROWS = 64, QZ_COLS = 256, QZ_THREADS = 256;

template <int G>
__global__ void __launch_bounds__(QZ_THREADS) quantize_kernel(const __nv_bfloat16 *__restrict__ W,
                                                              uint8_t *__restrict__ q,
                                                              __nv_bfloat16 *__restrict__ s, int M, int K) {
    constexpr int RW = QZ_ROWS / 8; // rows of a warp
    __shared__ __nv_bfloat16 ss[QZ_COLS / 32][QZ_ROWS];
    const int lane = lane_id(), warp = warp_id();
    const int k = blockIdx.x * QZ_COLS + lane * 8, m0 = blockIdx.y * QZ_ROWS;
    const size_t e = blockIdx.z;
    constexpr int PER = G / 8; // lanes of a group
    const int rows = k < K ? min(RW, M - m0 - warp * RW) : 0; // of this lane
    const size_t at = (e * M + m0 + warp * RW) * (size_t)K + k;
    uint4 v[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < rows) v[i] = __ldcs(reinterpret_cast<const uint4 *>(W + at + (size_t)i * K));
    }
    uint8_t *qp = q + at / 2;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        // The largest magnitude, two columns at a time (a NaN wins over all).
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&v[i]);
        __nv_bfloat162 t2 = __hmax2_nan(__hmax2_nan(__habs2(b[0]), __habs2(b[1])),
                                        __hmax2_nan(__habs2(b[2]), __habs2(b[3])));
#pragma unroll
        for (int d = 1; d < PER; d <<= 1) t2 = __hmax2_nan(t2, __shfl_xor_sync(0xffffffffu, t2, d));
        const float top = __bfloat162float(__hmax_nan(__low2bfloat16(t2), __high2bfloat16(t2)));
        __nv_bfloat16 sb = __float2bfloat16_rn(top * (1.0f / 7.0f));
        if (!(top < INFINITY)) sb = __ushort_as_bfloat16(0x7FFF); // every value NaN
        const float sf = __bfloat162float(sb);
        float w[8];
        unpack_bf16x2(v[i].x, w[0], w[1]);
        unpack_bf16x2(v[i].y, w[2], w[3]);
        unpack_bf16x2(v[i].z, w[4], w[5]);
        unpack_bf16x2(v[i].w, w[6], w[7]);
        uint32_t c = 0;
        if (sf >= 0x1p-120f) {
            float r;
            asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(sf));
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const float u = fmaf(w[j], r, 0x1.8p11f);                     // 1.5 * 2^11 + a multiple of 2^-12
                const uint32_t n = __float_as_uint(u + (12582920.0f - 0x1.8p11f)); // 0x4B400000 + code
                c = c * 16u + (n - 0x4B400000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // s = 0 (all zero, or too small for bf16) and s = NaN take the code of 0
                const float t = sf > 0.f ? fminf(fmaxf(rintf(w[j] / sf), -8.f), 7.f) : 0.f;
                c |= (uint32_t)((int)t + 8) << (4 * j);
            }
        }
        if (i < rows) *reinterpret_cast<uint32_t *>(qp + (size_t)i * (K / 2)) = c;
        if (lane % PER == 0) ss[lane / PER][warp * RW + i] = sb;
    }
    __syncthreads();
    constexpr int groups = QZ_COLS / G;
    const int g = threadIdx.x / QZ_ROWS, r = threadIdx.x % QZ_ROWS; // 8 groups at most
    const int kg = blockIdx.x * groups + g;
    if (g < groups && kg < K / G && m0 + r < M) s[(e * (K / G) + kg) * (size_t)M + m0 + r] = ss[g][r];
}

// A word's eight codes as the bf16 integers -8..7 in order: 128 + code, less 136.
__device__ __forceinline__ uint4 codes_bf16x8(uint32_t w) {
    const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
    const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
    const uint32_t k = 0x43434343u; // exponent of 128 as the upper bytes
    uint32_t v[4] = {__byte_perm(lo, k, 0x4140), __byte_perm(lo, k, 0x4342), __byte_perm(hi, k, 0x4140),
                     __byte_perm(hi, k, 0x4342)};
    const __nv_bfloat162 off(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308)); // 136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 o = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v[i]), off);
        v[i] = *reinterpret_cast<const uint32_t *>(&o);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int G>
__global__ void __launch_bounds__(QZ_THREADS) dequantize_kernel(const uint8_t *__restrict__ q,
                                                                const __nv_bfloat16 *__restrict__ s,
                                                                __nv_bfloat16 *__restrict__ W, int M, int K) {
    constexpr int RW = DQ_ROWS / 8;
    __shared__ __nv_bfloat16 ss[QZ_COLS / 32][DQ_ROWS];
    const int lane = lane_id(), warp = warp_id();
    const int k = blockIdx.x * QZ_COLS + lane * 8, m0 = blockIdx.y * DQ_ROWS;
    const size_t e = blockIdx.z;
    const int rows = k < K ? min(RW, M - m0 - warp * RW) : 0; // of this lane
    const size_t at = (e * M + m0 + warp * RW) * (size_t)K + k;
    uint32_t c[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        c[i] = 0;
        if (i < rows) c[i] = __ldcs(reinterpret_cast<const uint32_t *>(q + (at / 2 + (size_t)i * (K / 2))));
    }
    constexpr int groups = QZ_COLS / G;
    for (int j = threadIdx.x; j < groups * DQ_ROWS; j += QZ_THREADS) {
        const int g = j / DQ_ROWS, r = j % DQ_ROWS, kg = blockIdx.x * groups + g;
        if (kg < K / G && m0 + r < M) ss[g][r] = s[(e * (K / G) + kg) * (size_t)M + m0 + r];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        if (i >= rows) break;
        // integers -8..7 times the scale, in bf16: the one rounding
        const __nv_bfloat162 sb = __bfloat162bfloat162(ss[lane * 8 / G][warp * RW + i]);
        uint4 v = codes_bf16x8(c[i]);
        uint32_t o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&o[j]), sb);
            o[j] = *reinterpret_cast<const uint32_t *>(&r);
        }
        __stcs(reinterpret_cast<uint4 *>(W + at + (size_t)i * K), make_uint4(o[0], o[1], o[2], o[3]));
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
//   (3,7), and the tokens are brought into the same order.
// - A code is a bf16 as it stands: with exponent bits 0 the bits 0-7 of a bf16 are an
//   integer times 2^-133 (the lowest normal exponent continues the subnormals), so a
//   masked code at bits 0-3 is c 2^-133 and one at bits 4-7 is 16 c 2^-133, exactly.  One
//   bf16 multiply-add, by 2^127 (2^123) and less 2^-3, makes that (c - 8) / 64, exactly: four
//   logic operations and five multiply-adds for eight codes (centred_codes).
// - So the MMA sums centred weights times the tokens as they are: a column coded 8 adds
//   nothing, whatever its token, and no product of finite tokens leaves fp32's range.
//   (Summing c and taking 8 times the tokens' sum off per group saves the multiply-adds, but
//   its error goes with the tokens of columns coded 8 too, and it needs scaled tokens, which
//   leave fp32's range below 2^-72 and above 2^63.  us, that way / this: a layer of 32 tokens,
//   D 4096, 128 experts of 1408, 211 / 220; of 64, D 6144, 256 of 2048, groups of 64, 904 / 882;
//   16 tokens, 12288 x 6144, 27.4 / 23.6, as nobody sums the tokens.)
// - A group's sum is fp32 in the MMA; its scale is applied once per group in fp32, the
//   factor 64 once per tile.
//
// The tensor work is small here.  With more tokens tcgen05 takes over, its weights unpacked
// into TMEM (quant_wide_kernel).
//
// A block is one producer warp, one shaper warp and eight consumer warps: RG groups of 16 MT
// rows x KS slices of KW columns (RG * KS = 8).  The producer fills a ring: codes and
// scales by TMA, each token's columns by a bulk copy, which may come from anywhere (a
// routed token's row is fetched where it lies, without a gather pass).  A group's rows are 8 MT of the tile's
// first half and as many of its second, so a gate and its up value meet in one thread.  KS = 1 keeps
// a row's whole sum in one warp: no exchange, no barrier among the consumers; KS > 1, for
// few tiles, adds the slices' sums in order through shared memory.  With fewer tiles
// than SMs (or hardly more) the blocks of a cluster also share a tile's columns, and
// exchange their sums through distributed shared memory.
// ---------------------------------------------------------------------------
enum QuantKind { QUANT_LINEAR = 0, QUANT_GATE_UP = 1, QUANT_DOWN = 2 };

constexpr int QM_THREADS = 320;
constexpr int QM_CONSUMERS = 256;
constexpr int QM_MAXE = 512;

constexpr int qm_max(int a, int b) { return a > b ? a : b; }
template <int RG, int MT, int KW, int NT, int G> struct QmCfg {
    static constexpr int KS = 8 / RG;
    static constexpr int R = 16 * MT * RG, HALF = R / 2; // weight rows of a tile
    static constexpr int SK = KW * KS;              // columns of a stage
    static constexpr int UNIT = G < KW ? G : KW;    // columns of a slice under one scale
    static constexpr int BLOCKS = 2; // per SM
    static constexpr int BOX = SK / 2 < 128 ? SK / 2 : 128; // bytes of a code box's row = swizzle span
    static constexpr int NBOX = SK / 2 / BOX;
    static constexpr int W_BYTES = R * SK / 2;
    static constexpr int S_HALF = qm_max(128, HALF * (SK / G) * 2);
    static constexpr int XLD = SK * 2 + 64;         // a token's bytes: an odd multiple of 64
    static constexpr int X_BYTES = NT * 8 * XLD;
    static constexpr int PIECES = SK / 8;               // 16-byte pieces of a token's stage
    static constexpr int TURNS = NT * 8 * PIECES / 32;  // of a warp over all tokens
    static constexpr int STAGE = W_BYTES + 2 * S_HALF + X_BYTES;
    static constexpr int LD = R + 4; // floats per token in the sums' buffer
    static constexpr int RED_BYTES = KS > 1 ? KS * 8 * NT * LD * 4 : 0;
    static constexpr int JOIN_BYTES = KS > 1 ? 8 * NT * R * 4 : 0; // sums from the blocks of a cluster
    static constexpr int TAB_BYTES = 384 + (2 * QM_MAXE + 2) * 4;
    static constexpr int ROOM = (228 / BLOCKS - 1) * 1024;
    static constexpr int FIT = (ROOM - 1024 - RED_BYTES - JOIN_BYTES - TAB_BYTES) / STAGE;
    static constexpr int STAGES = FIT < 12 ? FIT : 12;
    static constexpr int SMEM = 1024 + STAGES * STAGE + RED_BYTES + JOIN_BYTES + TAB_BYTES;
    static_assert(STAGES >= 2 && (3 * STAGES + 2) * 8 + 8 <= 384, "ring depth");
};

struct QuantArgs {
    const uint8_t *x;   // LINEAR: x; GATE_UP: x; DOWN: h of the routed rows
    const uint8_t *x_s; // shared tokens: GATE_UP x; DOWN h_sh
    int row_bytes, row_bytes_s;
    int N, E, k, G;
    int K, K_s;         // summed columns, routed / shared
    int ncols, ncols_s; // output columns (LINEAR M, GATE_UP d, DOWN D), routed / shared
    int nb, nb_s;       // row tiles
    int split;          // blocks of a cluster that share a tile's columns (1, 2, 4 or 8)
    int direct;         // one token: pair j is expert topk_idx[j]'s only row
    const int32_t *topk_idx;
    const float *topk_w;
    const int32_t *tile_off, *counts, *perm_tok; // dispatch tables (tiles of 8 NT rows)
    const float *w_perm;
    void *out;   // LINEAR y bf16; GATE_UP h bf16; DOWN slot fp32
    void *out_s; // GATE_UP h_sh bf16; DOWN osh fp32
    float gate_max, up_max;
    int never_signal; // test hook: the shaper first waits for what never comes
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

__device__ __forceinline__ void fence_acq_rel_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

// Bulk copy of consecutive bytes into shared memory (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// c = a b, or c += a b.
__device__ __forceinline__ void mma_bf16(float (&c)[4], bool fresh, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if (fresh)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
constexpr uint32_t QM_LO = 0x000F000Fu, QM_HI = 0x00F000F0u;   // codes at bits 0-3, 4-7
constexpr uint32_t QM_C_LO = 0x7F007F00u, QM_C_HI = 0x7D007D00u; // 2^127, 2^123: codes / 64
constexpr uint32_t QM_OFF = 0xBE00BE00u;                       // -8 / 64
constexpr float QM_UNIT = 64.f;
// (code - 8) / 64 for the codes at bits 0-3 (lo) and 4-7 (hi) of each half of a word, or with
// p = 1 at bits 8-11 and 12-15.  These come down to bits 0-7 by bytes, which leaves nothing above
// them, so the low code is the byte less the high one, by a multiply-add in place of a mask:
// logic operations have half the rate (a layer of 32 tokens, D 4096, 128 experts of 1408: 220 us;
// with a shift and two masks 228).
__device__ __forceinline__ void centred_codes(uint32_t w, int p, uint32_t &lo, uint32_t &hi) {
    const uint32_t r = p ? __byte_perm(w, 0u, 0x4341) : w;
    const uint32_t h = r & QM_HI;
    hi = fma_bf16x2(h, QM_C_HI, QM_OFF);
    lo = p ? fma_bf16x2(r, QM_C_LO, fma_bf16x2(h, QM_C_LO ^ 0x80008000u, QM_OFF))
           : fma_bf16x2(r & QM_LO, QM_C_LO, QM_OFF);
}

// Maps: mW codes [E, M, K/2] bytes, box BOX x R x 1, swizzled; mS scales [E, K/G, M], box
// R x SK/G x 1 (GATE_UP: R/2 rows); the same of the shared expert (GATE_UP: its gate and
// up rows stacked).
template <int KIND, int RG, int MT, int KW, int NT, int G>
__global__ void __launch_bounds__(QM_THREADS, QmCfg<RG, MT, KW, NT, G>::BLOCKS)
    quant_product_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mS,
                         const __grid_constant__ CUtensorMap mW_s, const __grid_constant__ CUtensorMap mS_s,
                         const QuantArgs a) {
    using C = QmCfg<RG, MT, KW, NT, G>;
    constexpr int TT = 8 * NT, KS = C::KS, SK = C::SK, R = C::R, HALF = C::HALF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // ring: codes of all stages first (1024-byte aligned), then scales, then tokens
    uint8_t *ring_w = smem;
    uint8_t *ring_s = ring_w + C::STAGES * C::W_BYTES;
    uint8_t *ring_x = ring_s + C::STAGES * 2 * C::S_HALF;
    float *red = reinterpret_cast<float *>(ring_x + C::STAGES * C::X_BYTES);
    float *join = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(red) + C::RED_BYTES);
    uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(join) + C::JOIN_BYTES);
    uint64_t *empty = full + C::STAGES, *raw = empty + C::STAGES;
    uint64_t *jfull = raw + C::STAGES, *jempty = jfull + 1;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(jempty + 1);
    int *shaped = reinterpret_cast<int *>(jempty + 1) + 1; // stages that the shaper has arrived for
    int *s_tile = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(full) + 384);
    int *s_cnt = s_tile + QM_MAXE + 1;

    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 2); // the TMA issuer and the shaper
            mbar_init(&empty[s], 8);
            mbar_init(&raw[s], 1); // the copies of the tokens
        }
        mbar_init(jfull, 8 * a.split);
        mbar_init(jempty, 8 * a.split);
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
    // kernel of the stream.  Only DOWN, whose previous kernel is always the layer's GATE_UP,
    // waits further on: GATE_UP writes the tokens that DOWN reads and nothing else, and it
    // was complete up to its own previous kernel when it let DOWN start, so the tables
    // and the first stages of the weights are fetched while GATE_UP's last blocks run
    // (one token, D 4096, 128 experts of 1408: 30.6 to 29.0 us for the layer).
    if (KIND != QUANT_DOWN) {
        grid_dep_wait();
        grid_dep_launch_dependents();
    }
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
    // The blocks of a cluster take the same tiles, each a share of the columns' stages.
    const int split = KS > 1 ? a.split : 1;
    const int rank = KS > 1 && split > 1 ? (int)cluster_ctarank() : 0;
    const int tile0 = blockIdx.x / split, step = gridDim.x / split;
    if (split > 1)
        cluster_sync_all(); // every block's barriers are ready for the others' arrivals
    else
        __syncthreads();
    if (KIND != QUANT_LINEAR) {
        routed = (a.direct ? a.k : s_tile[a.E]) * a.nb;
        if (KIND == QUANT_GATE_UP && a.direct && blockIdx.x == 0 && threadIdx.x < a.k &&
            (s_tile[threadIdx.x] < 0 || s_tile[threadIdx.x] > a.E))
            record_error(DEV_BAD_INDEX, 400);
    }
    const int tts = (a.N + TT - 1) / TT;
    const int total = KIND == QUANT_LINEAR ? a.nb * tts : routed + a.nb_s * tts;
    constexpr int gps = SK / G; // groups of a stage
    const uint64_t limit = a.wait_limit_ns;
    if (KIND == QUANT_DOWN && warp != 8) {
        grid_dep_wait();
        grid_dep_launch_dependents();
    }

    uint32_t issued = 0, fetched = 0; // stages of tokens and of weights (the producer's)

    if (warp == 8) {
        // ------------------------------ producer ------------------------------
        const uint32_t stage_bytes = C::W_BYTES + 2 * HALF * gps * 2;
        uint32_t it = 0, s = 0, ph = 0; // stages issued, ring place and its parity
        bool ok = true;
        // Codes and scales of the tile's stage i to the ring's place s (one lane).
        auto fetch_weights = [&](const QuantTile &c, int i, uint32_t s) {
            const CUtensorMap *w = c.shared ? &mW_s : &mW, *sc = c.shared ? &mS_s : &mS;
            // GATE_UP's halves are gate rows and the up rows of the same columns, a box
            // each; otherwise the tile's rows are consecutive, one box
            const int r0 = KIND == QUANT_GATE_UP ? c.nb * HALF : c.nb * R;
            const int r1 = r0 + (c.shared ? a.ncols_s : a.ncols);
            mbar_arrive_expect_tx(&full[s], stage_bytes);
            uint8_t *dw = ring_w + s * C::W_BYTES;
#pragma unroll
            for (int b = 0; b < C::NBOX; ++b) {
                const int kx = i * (SK / 2) + b * C::BOX;
                tma_load_3d(w, &full[s], dw + b * R * C::BOX, kx, r0, c.e);
                if (KIND == QUANT_GATE_UP) tma_load_3d(w, &full[s], dw + (b * R + HALF) * C::BOX, kx, r1, c.e);
            }
            uint8_t *ds = ring_s + s * 2 * C::S_HALF;
            tma_load_3d(sc, &full[s], ds, r0, i * gps, c.e);
            if (KIND == QUANT_GATE_UP) tma_load_3d(sc, &full[s], ds + C::S_HALF, r1, i * gps, c.e);
        };
        uint32_t ahead = 0; // stages whose weights are on their way before the tokens are there
        if (KIND == QUANT_DOWN) {
            for (int t = tile0; t < total && ahead < C::STAGES; t += step) {
                QuantTile c;
                if (!quant_tile<KIND, TT>(t, routed, a, s_tile, s_cnt, c)) continue;
                const int stages = ((c.shared ? a.K_s : a.K) + SK - 1) / SK;
                for (int i = stages * rank / split; i < stages * (rank + 1) / split && ahead < C::STAGES; ++i, ++ahead)
                    if (lane == 0) fetch_weights(c, i, ahead);
            }
            __syncwarp();
            grid_dep_wait();
        }
        for (int t = tile0; t < total && ok; t += step) {
            QuantTile c;
            if (!quant_tile<KIND, TT>(t, routed, a, s_tile, s_cnt, c)) continue;
            const int K = c.shared ? a.K_s : a.K;
            const uint8_t *base = c.shared ? a.x_s : a.x;
            const size_t rb = c.shared ? a.row_bytes_s : a.row_bytes;
            // Lane i copies token i's columns of a stage.
            const uint8_t *src = nullptr;
            if (lane < c.cnt) {
                int row = c.row0 + lane;
                if (KIND == QUANT_GATE_UP && !c.shared) row = a.direct ? 0 : a.perm_tok[row];
                src = base + (size_t)row * rb;
            }
            const int stages = (K + SK - 1) / SK;
            for (int i = stages * rank / split; i < stages * (rank + 1) / split; ++i) {
                if (lane == 0) ok = mbar_wait(&empty[s], ph ^ 1, limit, abort_flag, 401);
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                if (lane == 0 && it >= ahead) fetch_weights(c, i, s);
                fence_proxy_async_smem(); // the shaper wrote there before
                const uint32_t bytes = (uint32_t)min(SK, K - i * SK) * 2;
                if (lane == 0) mbar_arrive_expect_tx(&raw[s], bytes * c.cnt);
                if (lane < c.cnt)
                    bulk_load(ring_x + s * C::X_BYTES + lane * C::XLD, src + (size_t)i * SK * 2, bytes, &raw[s]);
                ++it;
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        issued = it;
        fetched = it > ahead ? it : ahead;
    } else if (warp == 9) {
        // ------------------------------ shaper ------------------------------
        // Brings the tokens of a stage, in place, into the order of the MMA's operand (a lane's
        // 8 columns pair as (0,4), (1,5), (2,6), (3,7)), columns past K as zeros.
        uint32_t s = 0, ph = 0;
        int done = 0; // stages shaped
        bool ok = true;
        if (a.never_signal && tile0 < total)
            ok = __all_sync(0xffffffffu, mbar_wait(jfull, 0, limit, abort_flag, 404));
        for (int t = tile0; t < total && ok; t += step) {
            QuantTile c;
            if (!quant_tile<KIND, TT>(t, routed, a, s_tile, s_cnt, c)) continue;
            const int turns = (c.cnt * C::PIECES + 31) / 32;
            const int K = c.shared ? a.K_s : a.K, stages = (K + SK - 1) / SK;
            for (int i = stages * rank / split; i < stages * (rank + 1) / split; ++i) {
                ok = mbar_wait(&raw[s], ph, limit, abort_flag, 405);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break; // and no arrival: the others' waits end by the abort flag
                uint8_t *xs = ring_x + s * C::X_BYTES;
                // B turns of 32 pieces from turn j0 on (those past the tokens shape what
                // nobody reads).
                auto shape = [&](auto count, int j0) {
                    constexpr int B = decltype(count)::value;
                    uint4 v[B], *p[B];
#pragma unroll
                    for (int j = 0; j < B; ++j) {
                        const int at = (j0 + j) * 32 + lane, piece = at % C::PIECES;
                        p[j] = reinterpret_cast<uint4 *>(xs + at / C::PIECES * C::XLD + piece * 16);
                        v[j] = i * SK + piece * 8 < K ? *p[j] : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int j = 0; j < B; ++j)
                        *p[j] = make_uint4(__byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                                           __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
                };
                if (turns == 1) {
                    shape(IntC<1>{}, 0);
                } else {
                    constexpr int B = C::TURNS < 4 ? C::TURNS : 4;
#pragma unroll 1
                    for (int j0 = 0; j0 < turns; j0 += B) shape(IntC<B>{}, j0);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                ++done;
                if (++s == C::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) *shaped = done;
    } else {
        // ------------------------------ consumers ------------------------------
        const int rg = warp / KS, ks = warp % KS;
        const int g = lane >> 2, t4 = lane & 3;
        // This lane's ldmatrix address: a row of the group in one half, 16-byte chunk (32
        // columns) of the slice, at the place the swizzle gives it (TMA xors the chunk
        // with the number of the 128-byte line: the row, or half the row for 64-byte rows).
        constexpr int CPR = C::BOX / 16, PAIRS = KW / 64, UNIT = C::UNIT / 32;
        const int mch = lane >> 4, line = CPR == 8 ? lane & 7 : (lane & 7) >> 1;
        const uint32_t wbase = smem_u32(ring_w) +
                               (uint32_t)(((lane >> 3) & 1) * HALF + rg * 8 * MT + (lane & 7)) * C::BOX;
        uint32_t woff[PAIRS]; // 64 columns each
#pragma unroll
        for (int u = 0; u < PAIRS; ++u) {
            const int ch = ks * (KW / 32) + 2 * u;
            woff[u] = (uint32_t)(ch / CPR) * R * C::BOX + (uint32_t)((ch % CPR + mch) ^ line) * 16;
        }
        // this slice's first scale of the lane's row in the first half
        constexpr int SROW = KIND == QUANT_GATE_UP ? HALF : R;                // scales of a group
        constexpr int SHALF = KIND == QUANT_GATE_UP ? C::S_HALF / 2 : HALF;   // to the second half's
        const uint8_t *sbase = ring_s + ((ks * KW / G) * SROW + rg * 8 * MT + g) * 2;
        const uint8_t *xbase = ring_x + g * C::XLD + ks * KW * 2 + t4 * 16;
        const int ctid = threadIdx.x;
        // Output (token tk, row of the tile): v, or for GATE_UP gate v and up u.
        // The SwiGLU output is rounded to bf16, as in the fused forward: it is the down product's
        // MMA operand, whose type is the tokens'.  In two bf16 parts it would double that product's
        // MMAs and its tokens' bytes; as it is, the layer lies 2.3e-3 from fp64 (row norm), against
        // 1.7e-3 with an fp32 h.  The other sums stay in fp32 up to y.
        auto store = [&](const QuantTile &c, int tk, int row, float v, float u) {
            const int nc = c.shared ? a.ncols_s : a.ncols;
            const int col = c.nb * (KIND == QUANT_GATE_UP ? HALF : R) + row;
            if (col >= nc) return;
            const size_t at = (size_t)(c.row0 + tk) * nc + col;
            if (KIND == QUANT_LINEAR)
                static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
            else if (KIND == QUANT_GATE_UP)
                static_cast<__nv_bfloat16 *>(c.shared ? a.out_s : a.out)[at] =
                    __float2bfloat16_rn(swiglu_f(v, u, a.gate_max, a.up_max));
            else if (c.shared)
                static_cast<float *>(a.out_s)[at] = v;
            else
                static_cast<float *>(a.out)[at] = v * (a.direct ? a.topk_w[c.row0] : a.w_perm[c.row0 + tk]);
        };
        uint32_t s = 0, ph = 0, jph = 0;
        bool ok = true; // once false it stays so: no further arrival, but the barriers stay matched
        for (int t = tile0; t < total; t += step) {
            QuantTile c;
            if (!quant_tile<KIND, TT>(t, routed, a, s_tile, s_cnt, c)) continue;
            const int K = c.shared ? a.K_s : a.K;
            const int stages = (K + SK - 1) / SK;
            // The tile's sums for NTT blocks of 8 tokens (tokens past cnt hold
            // anything: a column of the product depends on its own token only).
            auto sums = [&](auto ntt) {
                constexpr int NTT = decltype(ntt)::value;
                float acc[MT][NTT][4];
                uint4 xv[NTT];
                bool on[NTT]; // this lane's token is there; absent ones are not fetched
#pragma unroll
                for (int j = 0; j < NTT; ++j) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.f;
                    xv[j] = make_uint4(0u, 0u, 0u, 0u);
                    on[j] = j * 8 + g < c.cnt;
                }
#pragma unroll 1
                for (int st = ok ? stages * rank / split : stages; st < stages * (rank + 1) / split; ++st) {
                    ok = mbar_wait(&full[s], ph, limit, abort_flag, 411);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t ws = wbase + s * C::W_BYTES;
                    const uint8_t *xs = xbase + s * C::X_BYTES, *scs = sbase + s * 2 * C::S_HALF;
                    float part[MT][NTT][4];
                    uint32_t cw[MT][4];
#pragma unroll
                    for (int b = 0; b < KW / 32; ++b) { // 32 columns each
                        if (b % 2 == 0) {
#pragma unroll
                            for (int i = 0; i < MT; ++i) ldmatrix_x4(ws + woff[b / 2] + i * 8 * C::BOX, cw[i]);
                        }
#pragma unroll
                        for (int j = 0; j < NTT; ++j)
                            if (on[j])
                                xv[j] = *reinterpret_cast<const uint4 *>(xs + j * 8 * C::XLD + b * 64);
#pragma unroll
                        for (int p = 0; p < 2; ++p)
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                uint32_t a0, a1, a2, a3;
                                centred_codes(cw[i][2 * (b % 2)], p, a0, a2);
                                centred_codes(cw[i][2 * (b % 2) + 1], p, a1, a3);
#pragma unroll
                                for (int j = 0; j < NTT; ++j)
                                    mma_bf16(part[i][j], b % UNIT == 0 && p == 0, a0, a1, a2, a3,
                                             p ? xv[j].z : xv[j].x, p ? xv[j].w : xv[j].y);
                            }
                        if ((b + 1) % UNIT == 0) { // the group, or its part here, ends
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                const __nv_bfloat16 *sp =
                                    reinterpret_cast<const __nv_bfloat16 *>(scs) + (b * 32 / G) * SROW + i * 8;
                                const float s0 = __bfloat162float(sp[0]);
                                const float s1 = __bfloat162float(sp[SHALF]);
#pragma unroll
                                for (int j = 0; j < NTT; ++j) {
                                    acc[i][j][0] = fmaf(s0, part[i][j][0], acc[i][j][0]);
                                    acc[i][j][1] = fmaf(s0, part[i][j][1], acc[i][j][1]);
                                    acc[i][j][2] = fmaf(s1, part[i][j][2], acc[i][j][2]);
                                    acc[i][j][3] = fmaf(s1, part[i][j][3], acc[i][j][3]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                    if (++s == C::STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NTT; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] *= QM_UNIT;
                if (KS == 1) {
                    if (!ok) return;
#pragma unroll
                    for (int j = 0; j < NTT; ++j)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int tk = j * 8 + 2 * t4 + r;
                            if (tk < c.cnt) {
#pragma unroll
                                for (int i = 0; i < MT; ++i) {
                                    const int row = (rg * MT + i) * 8 + g;
                                    if (KIND == QUANT_GATE_UP) {
                                        store(c, tk, row, acc[i][j][r], acc[i][j][2 + r]);
                                    } else {
                                        store(c, tk, row, acc[i][j][r], 0.f);
                                        store(c, tk, HALF + row, acc[i][j][2 + r], 0.f);
                                    }
                                }
                            }
                        }
                } else {
                    named_bar_sync(1, QM_CONSUMERS); // the last tile's sums have been read
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < NTT; ++j) {
                            float *d = red + (ks * TT + j * 8 + 2 * t4) * C::LD + (rg * MT + i) * 8 + g;
                            d[0] = acc[i][j][0];
                            d[C::LD] = acc[i][j][1];
                            d[HALF] = acc[i][j][2];
                            d[C::LD + HALF] = acc[i][j][3];
                        }
                }
            };
            if (c.cnt <= 8)
                sums(IntC<1>{});
            else
                sums(IntC<NT>{});
            if (KS == 1) continue;
            named_bar_sync(1, QM_CONSUMERS);
            if (!ok) continue;
            auto sum = [&](int tk, int row) {
                float v = red[tk * C::LD + row];
#pragma unroll
                for (int q = 1; q < KS; ++q) v += red[(q * TT + tk) * C::LD + row];
                return v;
            };
            constexpr int OUT = KIND == QUANT_GATE_UP ? HALF : R;
            if (split == 1) {
                for (int i = ctid; i < c.cnt * OUT; i += QM_CONSUMERS) {
                    const int tk = i / OUT, row = i % OUT;
                    store(c, tk, row, sum(tk, row), KIND == QUANT_GATE_UP ? sum(tk, HALF + row) : 0.f);
                }
                continue;
            }
            // Each block of the cluster finishes HALF / split rows of either half: the
            // others' sums come into its `join` [block][token][2][rows], and are added in
            // the blocks' order.
            const int own = HALF / split;
            ok = mbar_wait_cl(jempty, jph ^ 1, limit, abort_flag, 412); // all have read the last tile's
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            for (int i = ctid; i < c.cnt * R; i += QM_CONSUMERS) {
                const int tk = i / R, row = i % R, f = row % HALF;
                st_cluster_f32(mapa_shared(smem_u32(join + (rank * TT + tk) * 2 * own + (row / HALF) * own + f % own),
                                           f / own),
                               sum(tk, row));
            }
            fence_acq_rel_cluster();
            __syncwarp();
            if (lane < split) mbar_arrive_remote(mapa_shared(smem_u32(jfull), lane));
            ok = mbar_wait_cl(jfull, jph, limit, abort_flag, 413);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            auto joined = [&](int tk, int at) {
                float v = join[tk * 2 * own + at];
                for (int q = 1; q < split; ++q) v += join[(q * TT + tk) * 2 * own + at];
                return v;
            };
            const int out = KIND == QUANT_GATE_UP ? own : 2 * own;
            for (int i = ctid; i < c.cnt * out; i += QM_CONSUMERS) {
                const int tk = i / out, at = i % out, row = (at / own) * HALF + rank * own + at % own;
                store(c, tk, row, joined(tk, at), KIND == QUANT_GATE_UP ? joined(tk, own + at) : 0.f);
            }
            __syncwarp();
            if (lane < split) mbar_arrive_remote(mapa_shared(smem_u32(jempty), lane));
            jph ^= 1;
        }
    }
    // After a wait that ran out nobody waits for the last copies: let them land before the
    // block's memory goes away.  All roles have ended, so full lacks just the arrivals that the
    // shaper did not make.
    __syncthreads();
    if (*abort_flag && warp == 8 && lane == 0) {
        drain_copies(raw, C::STAGES, issued, limit, abort_flag, 402);
        for (uint32_t j = fetched > C::STAGES ? fetched - C::STAGES : 0; j < fetched; ++j)
            if ((int)j >= *shaped) mbar_arrive(&full[j % C::STAGES]);
        drain_copies(full, C::STAGES, fetched, limit, abort_flag, 403);
    }
    if (split > 1) {
        __syncwarp();
        cluster_sync_all(); // no block leaves while another may still write to it
    }
}

// ---------------------------------------------------------------------------
// The product of one matrix with more than 24 tokens (32 with groups of 64, 48 with groups of
// 32).  There the register kernel's MMA time grows with the tokens (mma.sync m16n8k16, 8 cycles
// each), so tcgen05 takes over: a tile is 128 weight rows x up to 96 tokens, one block per SM.
// Where that leaves SMs idle, the blocks of a cluster share a tile's columns: each sums its own,
// hands every block its tokens' sums through distributed shared memory, and those are added in
// the blocks' order.
//
//   warp 0       TMA producer of the codes: 128 columns (8 KiB) a stage
//   warp 2       TMA producer of the tokens: two swizzled boxes of 64 columns a stage
//   warps 1, 3   MMA issuers, the stages in turn (every group has an accumulator of its
//                own): M = 128 rows, N = the tokens in steps of 16, K = 16
//   warps 4-11   codes to bf16 integers -8..7 (exact), thread = row, written to TMEM,
//                where the MMA takes its A operand from: through shared memory they would
//                cost eight times the codes' bytes in writes and reads, and its bandwidth
//                was what bound the kernel then (1500 cycles a stage); two teams of four
//                warps take the stages in turn
//   warps 12-19  sums: each group has a TMEM accumulator of its own (4 to 12 take turns);
//                thread = row; sum += scale * group, in fp32 registers
//
// The weights are not rounded: integers times tokens are exact in the MMA's fp32 and the
// scale is applied once per group outside.  With A in TMEM a K = 16 MMA takes about 120
// cycles however few the tokens, so a stage's eight take some 950; measured are 0.63 us a
// stage (1200 cycles) with groups of 128, 0.9 with 64 and 1.5 with 32, whose sums bound it.
// Its codes would take 330 cycles from memory.  A wait costs the issuing thread some 200
// cycles more while MMAs are in flight, so there are two issuers, and the tokens' arrival
// counts on the unpacked tile's barrier.
// ---------------------------------------------------------------------------
constexpr int QW_THREADS = 640;
constexpr int QW_ROWS = 128, QW_TOK = 96, QW_COLS = 128;
constexpr int QW_CST = 8, QW_AST = 4; // stages of codes; of tokens
constexpr int QW_UST = 2;             // of unpacked weights: 64 TMEM columns each, from QW_UCOL on
constexpr int QW_UCOL = 512 - QW_UST * QW_COLS / 2;
constexpr int QW_MAXACC = 12; // TMEM accumulators in turn: QW_UCOL columns / tokens of a tile
constexpr int QW_C_BYTES = QW_ROWS * QW_COLS / 2;     // 8 KiB of codes
constexpr int QW_X_HALF = QW_TOK * 128;               // 64 columns of the tokens
constexpr int QW_X_BYTES = 2 * QW_X_HALF;             // 24 KiB
constexpr int QW_JOIN = QW_TOK + 8; // sums of a row from a cluster's blocks, each its share rounded up
constexpr int QW_SMEM = 1024 + QW_CST * QW_C_BYTES + QW_AST * QW_X_BYTES + QW_JOIN * QW_ROWS * 4 + 768;
static_assert(QW_SMEM <= 232448, "shared memory");
constexpr int QW_UNPACK = 4, QW_SUMS = 8;             // warps

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The same shape written: lane t's values to TMEM lane t, 32 consecutive columns.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (+)= A B with A in TMEM (lane = row, 16 bf16 in 8 columns), B by descriptor.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

struct QuantWideArgs {
    const __nv_bfloat16 *s;
    __nv_bfloat16 *y;
    int N, M, K;
    int tok;        // tokens of a tile (a multiple of 16)
    int accs, ld;   // batches of TMEM accumulators; columns of one
    int nb, tts;    // row tiles, token tiles
    int split, own; // blocks of a cluster that share a tile's columns; tokens each finishes
    int never_signal; // test hook: the MMA issuers first wait for what never comes
    uint64_t wait_limit_ns;
};

// Maps: mC codes [M, K/2] bytes, box 64 x 128, swizzled; mX tokens [N, K], box 64 x
// the tile's tokens, swizzled (large boxes: each TMA load costs its issuer 75-150 cycles).
// SPLIT: the blocks of a cluster share a tile's columns (a kernel of its own, as one for
// both ran 4 to 15 % slower unshared).
template <int G, bool SPLIT>
__global__ void __launch_bounds__(QW_THREADS, 1)
    quant_wide_kernel(const __grid_constant__ CUtensorMap mC, const __grid_constant__ CUtensorMap mX,
                      const QuantWideArgs a) {
    constexpr int GROUPS = QW_COLS / G;        // of a stage
    constexpr int BATCH = GROUPS > 1 ? 2 : 1;  // groups handed over at a time
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *cbuf = smem;
    uint8_t *xbuf = cbuf + QW_CST * QW_C_BYTES;
    float *join = reinterpret_cast<float *>(xbuf + QW_AST * QW_X_BYTES); // [block][token][row]
    uint64_t *cfull = reinterpret_cast<uint64_t *>(join + QW_JOIN * QW_ROWS);
    uint64_t *cempty = cfull + QW_CST;
    uint64_t *afull = cempty + QW_CST, *aempty = afull + QW_AST;
    uint64_t *uempty = aempty + QW_AST, *dfull = uempty + QW_UST, *dempty = dfull + QW_MAXACC, *drain = dempty + QW_MAXACC;
    uint64_t *jfull = drain + 2, *jempty = jfull + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(jempty + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint32_t *stopped = tmem_slot + 2; // each unpacking warp's first stage without its arrival
    const int warp = warp_id(), lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < QW_CST; ++i) {
            mbar_init(&cfull[i], 1);
            mbar_init(&cempty[i], QW_UNPACK);
        }
        for (int i = 0; i < QW_AST; ++i) {
            mbar_init(&afull[i], QW_UNPACK + 1); // unpacked weights, tokens
            mbar_init(&aempty[i], 1);
        }
        for (int i = 0; i < QW_UST; ++i) mbar_init(&uempty[i], 1);
        for (int i = 0; i < QW_MAXACC; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], QW_SUMS);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
        if (SPLIT) {
            mbar_init(jfull, QW_SUMS * a.split);
            mbar_init(jempty, QW_SUMS * a.split);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mC);
        tma_prefetch_desc(&mX);
    }
    // All that follows comes after the previous kernel of the stream.
    grid_dep_wait();
    grid_dep_launch_dependents();
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    if (SPLIT)
        cluster_sync_all(); // every block's barriers are ready for the others' arrivals
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = a.nb * a.tts; // token tiles of one row tile are neighbours
    const int split = SPLIT ? a.split : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
    const int tile0 = blockIdx.x / split, step = gridDim.x / split;
    // this block's stages and groups of a tile
    const int all = (a.K + QW_COLS - 1) / QW_COLS;
    const int st0 = all * rank / split, st1 = all * (rank + 1) / split;
    const int gr0 = st0 * GROUPS, groups = min(st1 * GROUPS, a.K / G) - gr0;
    const uint64_t limit = a.wait_limit_ns;

    uint32_t issued = 0; // stages of tokens (their producer's)

    if (warp == 0 || warp == 2) {
        if (lane == 0) {
            const bool codes = warp == 0;
            uint64_t *full = codes ? cfull : afull, *empty = codes ? cempty : aempty;
            const uint32_t ring = codes ? QW_CST : QW_AST;
            uint32_t it = 0, s = 0, ph = 0;
            bool ok = true;
            for (int t = tile0; t < total && ok; t += step) {
                const int m0 = t / a.tts * QW_ROWS, n0 = t % a.tts * a.tok;
                for (int i = st0; i < st1; ++i, ++it) {
                    if (!mbar_wait(&empty[s], ph ^ 1, limit, abort_flag, codes ? 501 : 503)) { ok = false; break; }
                    if (codes) {
                        mbar_arrive_expect_tx(&full[s], QW_C_BYTES);
                        tma_load_2d(&mC, &full[s], cbuf + s * QW_C_BYTES, i * (QW_COLS / 2), m0);
                    } else {
                        mbar_arrive_expect_tx(&full[s], a.tok * 256);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tma_load_2d(&mX, &full[s], xbuf + s * QW_X_BYTES + h * QW_X_HALF, i * QW_COLS + h * 64,
                                        n0);
                    }
                    if (++s == ring) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (codes)
                drain_copies(full, ring, it, limit, abort_flag, 502);
            else
                issued = it;
        }
        __syncwarp();
    } else if (warp == 1 || warp == 3) {
        if (lane == 0) {
            const uint32_t turn = warp >> 1;
            uint32_t it = 0, d = 0, ph = 0; // stages so far; accumulators of a batch and their round
            bool ok = true;
            if (a.never_signal && tile0 < total) ok = mbar_wait(&drain[turn], 0, limit, abort_flag, 511);
            auto next = [&]() {
                if (++d == (uint32_t)a.accs) {
                    d = 0;
                    ph ^= 1;
                }
            };
            for (int t = tile0; t < total && ok; t += step) {
                const int n = (min(a.tok, a.N - t % a.tts * a.tok) + 15) & ~15;
                const uint32_t idesc = umma_idesc_bf16(QW_ROWS, n);
                for (int i = 0; i < st1 - st0 && ok; ++i, ++it) {
                    const int ng = min(GROUPS, groups - i * GROUPS);
                    if ((it & 1) != turn) {
                        // The other's stage.  A wait must not fall two rounds behind its
                        // barrier: with two batches a stage, this one waits here too.
                        for (int u = 0; u < ng && ok; u += BATCH) {
                            if (GROUPS > BATCH) ok = mbar_wait(&dempty[d], ph ^ 1, limit, abort_flag, 513);
                            next();
                        }
                        continue;
                    }
                    const uint32_t b = it % QW_AST;
                    if (!mbar_wait(&afull[b], (it / QW_AST) & 1, limit, abort_flag, 512)) { ok = false; break; }
                    const uint64_t dx = umma_desc_sw128(smem_u32(xbuf + b * QW_X_BYTES));
                    const uint32_t ta = tmem_base + QW_UCOL + it % QW_UST * (QW_COLS / 2);
                    for (int u0 = 0; u0 < ng; u0 += BATCH) {
                        if (!mbar_wait(&dempty[d], ph ^ 1, limit, abort_flag, 514)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll
                        for (int v = 0; v < BATCH; ++v) {
                            const int u = u0 + v;
                            if (u >= ng) break;
#pragma unroll
                            for (int kk = 0; kk < G / 16; ++kk) {
                                const int k = u * (G / 16) + kk; // step of 16 columns in the stage
                                // (8 columns of A; steps of the descriptor's address field)
                                umma_bf16_ts(tmem_base + (d * BATCH + v) * a.ld, ta + k * 8,
                                             dx + ((k >> 2) * (QW_X_HALF / 16) + (k & 3) * 2), idesc, kk > 0 ? 1u : 0u);
                            }
                        }
                        umma_commit(&dfull[d]);
                        next();
                    }
                    if (!ok) break;
                    umma_commit(&uempty[it % QW_UST]);
                    umma_commit(&aempty[b]);
                }
            }
            // Drain: wait until every MMA issued by this thread has completed.
            umma_commit(&drain[turn]);
            settle(&drain[turn], 0, limit, abort_flag, 100000000ull, 515);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        // Row q * 32 + lane: its 64 bytes of codes are four pieces, swizzled by TMA.
        const int team = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
        const uint32_t ta = tmem_base + QW_UCOL + ((uint32_t)(q * 32) << 16);
        uint32_t it = 0;
        bool ok = true;
        for (int t = tile0; t < total && ok; t += step) {
            for (int i = st0; i < st1; ++i, ++it) {
                if ((int)(it & 1) != team) continue;
                const uint32_t s = it % QW_CST, b = it % QW_AST, u = it % QW_UST;
                ok = mbar_wait(&cfull[s], (it / QW_CST) & 1, limit, abort_flag, 521);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = *reinterpret_cast<const uint4 *>(cbuf + s * QW_C_BYTES + row * 64 +
                                                            ((j ^ ((row >> 1) & 3)) << 4));
                __syncwarp();
                if (lane == 0) mbar_arrive(&cempty[s]);
                // the MMAs that read this part of TMEM, and the tokens' stage, are done
                ok = mbar_wait(&uempty[u], ((it / QW_UST) & 1) ^ 1, limit, abort_flag, 522) &&
                     mbar_wait(&aempty[b], ((it / QW_AST) & 1) ^ 1, limit, abort_flag, 523);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) { // 64 columns each
                    uint32_t o[32];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 w = v[2 * h + j];
                        const uint4 e[4] = {codes_bf16x8(w.x), codes_bf16x8(w.y), codes_bf16x8(w.z), codes_bf16x8(w.w)};
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            o[j * 16 + r * 4] = e[r].x;
                            o[j * 16 + r * 4 + 1] = e[r].y;
                            o[j * 16 + r * 4 + 2] = e[r].z;
                            o[j * 16 + r * 4 + 3] = e[r].w;
                        }
                    }
                    tmem_st_32x32b_x32(ta + u * (QW_COLS / 2) + h * 32, o);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&afull[b]);
            }
        }
        if (lane == 0) stopped[warp - 4] = ok ? UINT32_MAX : it;
    } else {
        const int q = warp & 3; // TMEM lanes 32 q ..: rows q*32 + lane of the tile
        // this warp's tokens of the tile: the first or the second half, in steps of 16
        const int first = warp >= 16 ? (a.tok / 2 + 15) & ~15 : 0;
        const int most = warp >= 16 ? QW_TOK : (a.tok / 2 + 15) & ~15;
        uint32_t d = 0, ph = 0, jph = 0;
        for (int t = tile0; t < total; t += step) {
            const int m = t / a.tts * QW_ROWS + q * 32 + lane, n0 = t % a.tts * a.tok;
            const int cnt = min(min(a.tok, a.N - n0), most) - first; // tokens of this warp (any sign)
            const __nv_bfloat16 *sp = a.s + (size_t)gr0 * a.M + min(m, a.M - 1);
            float acc[48];
#pragma unroll
            for (int c = 0; c < 48; ++c) acc[c] = 0.f;
            bool ok = true;
            // Scales of four groups, and the next four on their way (some 1000 cycles from
            // memory; moving a register waits for its load, so they move once in four).
            __nv_bfloat16 sc[4], next[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) next[j] = sp[(size_t)min(j, groups - 1) * a.M];
            for (int g0 = 0; g0 < groups; g0 += BATCH) {
                if ((g0 & 3) == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sc[j] = next[j];
                        next[j] = sp[(size_t)min(g0 + 4 + j, groups - 1) * a.M];
                    }
                }
                ok = mbar_wait(&dfull[d], ph, limit, abort_flag, 531);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int gi = g0 + u;
                    if (u && gi >= groups) break;
                    const float s = __bfloat162float(gi & 2 ? (gi & 1 ? sc[3] : sc[2]) : (gi & 1 ? sc[1] : sc[0]));
                    const uint32_t base = tmem_base + (d * BATCH + u) * a.ld + first + ((uint32_t)(q * 32) << 16);
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        if (cnt > c * 16) {
                            uint32_t v[16];
                            tmem_ld_32x32b_x16(base + c * 16, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                acc[c * 16 + j] = fmaf(s, __uint_as_float(v[j]), acc[c * 16 + j]);
                        }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty[d]);
                if (++d == (uint32_t)a.accs) {
                    d = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
            if (SPLIT) {
                // all have read the last tile's
                ok = mbar_wait_cl(jempty, jph ^ 1, limit, abort_flag, 532);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t to = smem_u32(join) + (uint32_t)(rank * a.own * QW_ROWS + q * 32 + lane) * 4;
                int who = first / a.own, at = first - who * a.own; // block that finishes a token; its place there
#pragma unroll
                for (int c = 0; c < 48; ++c)
                    if (c < cnt) {
                        st_cluster_f32(mapa_shared(to + (uint32_t)at * (QW_ROWS * 4), who), acc[c]);
                        if (++at == a.own) {
                            at = 0;
                            ++who;
                        }
                    }
                fence_acq_rel_cluster();
                __syncwarp();
                if (lane < a.split) mbar_arrive_remote(mapa_shared(smem_u32(jfull), lane));
                ok = mbar_wait_cl(jfull, jph, limit, abort_flag, 533);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                // this block's tokens, a warp every second one of its 32 rows
                const int mine = min(a.own, min(a.tok, a.N - n0) - rank * a.own);
                for (int c = warp >= 16; c < mine; c += 2) {
                    const float *from = join + c * QW_ROWS + q * 32 + lane;
                    float v = from[0];
                    for (int r = 1; r < a.split; ++r) v += from[r * a.own * QW_ROWS];
                    if (m < a.M) a.y[(size_t)(n0 + rank * a.own + c) * a.M + m] = __float2bfloat16_rn(v);
                }
                __syncwarp();
                if (lane < a.split) mbar_arrive_remote(mapa_shared(smem_u32(jempty), lane));
                jph ^= 1;
                continue;
            }
            if (m < a.M) {
                __nv_bfloat16 *y = a.y + (size_t)(n0 + first) * a.M + m;
#pragma unroll
                for (int c = 0; c < 48; ++c)
                    if (c < cnt) y[(size_t)c * a.M] = __float2bfloat16_rn(acc[c]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
    // After a wait that ran out nobody waits for the tokens' last copies: let them land before
    // the block's memory goes away.  All roles have ended, so afull lacks just the arrivals
    // that the unpacking warps did not make.
    if (*abort_flag && warp == 2 && lane == 0) {
        for (uint32_t j = issued > QW_AST ? issued - QW_AST : 0; j < issued; ++j)
            for (int w = 0; w < QW_UNPACK; ++w)
                if (stopped[(j & 1) * QW_UNPACK + w] <= j) mbar_arrive(&afull[j % QW_AST]);
        drain_copies(afull, QW_AST, issued, limit, abort_flag, 502);
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync_all(); // no block leaves while another may still write to it
    }
}

// y(n) = the k weighted expert rows in slot order + the shared expert's row, fp32,
// rounded once.  One thread per 4 columns; eight rows are fetched before any is added (a
// row after the other, each behind its position's load, took 9 us for 16 tokens).
constexpr int QC_THREADS = 128;
__global__ void __launch_bounds__(QC_THREADS) quant_combine_kernel(const QuantArgs a, const float *slot,
                                                                   const float *osh, const int32_t *pos_of,
                                                                   __nv_bfloat16 *y, int D) {
    grid_dep_wait();
    const int n = blockIdx.x, c = (blockIdx.y * QC_THREADS + threadIdx.x) * 4;
    if (c >= D) return;
    const float4 o = __ldcg(reinterpret_cast<const float4 *>(osh + (size_t)n * D + c));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        int p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = -1;
            if (j0 + j < a.k) {
                if (a.direct) {
                    const int e = a.topk_idx[j0 + j];
                    if (e >= 0 && e < a.E) p[j] = j0 + j;
                } else {
                    p[j] = pos_of[(size_t)n * a.k + j0 + j];
                }
            }
        }
        float4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p[j] >= 0) w[j] = __ldcg(reinterpret_cast<const float4 *>(slot + (size_t)p[j] * D + c));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v.x += w[j].x;
            v.y += w[j].y;
            v.z += w[j].z;
            v.w += w[j].w;
        }
    }
    *reinterpret_cast<uint2 *>(y + (size_t)n * D + c) =
        make_uint2(pack_bf16x2(v.x + o.x, v.y + o.y), pack_bf16x2(v.z + o.z, v.w + o.w));
}

}  // namespace moe
