// Matrix products grouped by expert over ragged row segments, with both gradients.
// Row r in [off[e], off[e+1]) belongs to expert e; W is [E, M, K]:
//
//   forward  y_r  = W_e x_r                     rows x M,  sums over K
//   dgrad    dx_r = W_e^T dy_r                  rows x K,  sums over M
//   wgrad    dW_e = sum over e's rows dy_r x_r^T  M x K,   sums over the rows
//
// The segments are used where they lie: no permuted or padded copy.  A TMA box may
// start at any row, so a tile's 128 rows begin at the segment's own row.  Rows of a
// box past the segment's end belong to other experts: in forward and dgrad they
// only fill output rows that are not stored; in wgrad they would enter the sum,
// so the last k-block is cut to the 16 rows an MMA step takes and the rows past the
// end are zeroed in shared memory, in both operands (a NaN there must not meet a 0).
//
// bf16: tcgen05.mma, 128 x 256 output tiles, k-blocks of 64, fp32 accumulators in
// TMEM, one rounding to bf16.  Persistent, one CTA per SM, warp-specialised like the
// forward's GEMMs: warp 0 TMA, warp 1 MMA, the others epilogue; two accumulators.
// The operands keep their memory layout.  Where the summed index is contiguous the
// shared-memory tile is K-major (forward both, dgrad dy); where it is the row the
// tile is MN-major (dgrad W, wgrad both) and the MMA reads it transposed.
#pragma once

#include "common.cuh"
#include "gemm_sm100.cuh"

namespace moe {

enum GroupedMode { GRP_FORWARD = 0, GRP_DGRAD = 1, GRP_WGRAD = 2 };

constexpr int GRP_BM = 128;
constexpr int GRP_BN = 256;
constexpr int GRP_BK = 64;
constexpr int GRP_STAGES = 4;
constexpr int GRP_MAXE = 512;
constexpr int GRP_A_BYTES = GRP_BM * GRP_BK * 2; // 16 KiB
constexpr int GRP_B_BYTES = GRP_BN * GRP_BK * 2; // 32 KiB
constexpr int GRP_STAGE_BYTES = GRP_A_BYTES + GRP_B_BYTES;
constexpr int GRP_CHUNK = 64 * 64 * 2; // an MN-major box: 64 rows of 64 elements
constexpr int GRP_OUT_BUF = 32 * 64 * 2; // an epilogue warp's store box: 32 rows of 64 elements
// Shared memory (1024-byte aligned base): ring, one store box per epilogue warp, barriers,
// segment tables.  wgrad's tiles are short (an expert's rows), so its epilogue counts: it
// has eight warps instead of four; their boxes leave room for one table, all that it needs.
template <int MODE> struct GrpCfg {
    static constexpr int EPI = MODE == GRP_WGRAD ? 8 : 4; // epilogue warps
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr int COLS = GRP_BN * 4 / EPI;         // of a tile, per warp
    static constexpr int STG_OFF = GRP_STAGES * GRP_STAGE_BYTES;
    static constexpr int BAR_OFF = STG_OFF + EPI * GRP_OUT_BUF;
    static constexpr int TAB_OFF = BAR_OFF + 128;
    static constexpr int SMEM = TAB_OFF + (MODE == GRP_WGRAD ? 1 : 2) * (GRP_MAXE + 1) * 4;
    static_assert(SMEM <= 232448, "shared memory");
};
static_assert((2 * GRP_STAGES + 5) * 8 + 8 <= 128, "barrier block");

struct GroupedArgs {
    const int32_t *offsets; // [E+1]
    int rows, E;
    int M, K;     // W is [E, M, K]
    int red;      // forward K, dgrad M (wgrad: the segment's rows)
    int ncols;    // output columns: forward M, dgrad K, wgrad K
    int nb;       // output column blocks
    int mb;       // wgrad: output row blocks
    int wide;     // MN-major operands: one load for all of a tile's 64-column boxes
    void *out;
    int zero_rest; // forward, dgrad: write zeros to the rows of no expert
    int split;    // blocks of a cluster that share a tile's k-blocks
    int never_signal; // test hook: the MMA warp first waits for what never comes
    uint64_t wait_limit_ns;
};

// Shared-memory matrix descriptor of an MN-major tile written by TMA with 128-byte
// swizzle: rows of the summed index, 128 bytes (64 elements of M or N) each; eight
// rows are 1024 bytes (stride byte offset), the next 64 elements of M or N are one
// box further (leading byte offset).
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(uint32_t saddr, uint32_t box_bytes) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor bits: the operand is MN-major (transposed).
constexpr uint32_t UMMA_A_MN = 1u << 15;
constexpr uint32_t UMMA_B_MN = 1u << 16;

__device__ __forceinline__ void tma_load_3d(const CUtensorMap *map, uint64_t *bar, void *dst,
                                            int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(const CUtensorMap *map, uint64_t *bar, void *dst,
                                            int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1,
                                             int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// The segment table: s_off[0..E] the offsets, made safe (within [0, rows] and not
// decreasing; what was not is reported by one CTA), and s_tile[0..E] (unless null) the
// prefix of row tiles of `tile` rows.  One warp; lanes take consecutive experts.
__device__ __forceinline__ void grouped_table(const int32_t *offsets, int E, int rows, int tile,
                                              int *s_off, int *s_tile, bool report, int lane) {
    int top = 0; // running maximum of the offsets
    bool bad = false;
    for (int base = 0; base <= E; base += 32) {
        const int i = base + lane;
        const int raw = i <= E ? offsets[i] : rows;
        int v = min(max(raw, 0), rows);
        bad |= v != raw;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v = max(v, n);
        }
        v = max(v, top);
        bad |= i <= E && v != raw;
        if (i <= E) s_off[i] = v;
        top = __shfl_sync(0xffffffffu, v, 31);
    }
    if (report && __any_sync(0xffffffffu, bad) && lane == 0) record_error(DEV_BAD_INDEX, 300);
    __syncwarp();
    if (!s_tile) return;
    int carry = 0;
    for (int base = 0; base <= E; base += 32) {
        const int e = base + lane;
        const int v = e < E ? (s_off[e + 1] - s_off[e] + tile - 1) / tile : 0;
        int incl = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += n;
        }
        if (e <= E) s_tile[e] = carry + incl - v;
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// Zeros to the rows outside [lo, hi): threads tid, tid + step, ... of 16-byte pieces.
__device__ __forceinline__ void grouped_zero_rest(void *out, int rows, size_t row_bytes, int lo, int hi,
                                                  size_t tid, size_t step) {
    const size_t per = row_bytes >> 4;
    const size_t head = (size_t)lo * per, n = head + (size_t)(rows - hi) * per;
    uint4 *p = static_cast<uint4 *>(out);
    for (size_t i = tid; i < n; i += step)
        p[i < head ? i : (size_t)hi * per + (i - head)] = make_uint4(0u, 0u, 0u, 0u);
}

struct GroupedTile {
    int e;
    int r0, r1; // forward, dgrad: output rows [r0, r1); wgrad: summed rows [r0, r1)
    int m0;     // wgrad: first output row
    int n0;     // first output column
    int kb;     // k-blocks
};

template <int MODE>
__device__ __forceinline__ GroupedTile grouped_tile(int t, const GroupedArgs &a, const int *s_off,
                                                    const int *s_tile) {
    GroupedTile c;
    if (MODE == GRP_WGRAD) {
        const int per = a.nb * a.mb;
        c.e = t / per;
        const int l = t - c.e * per;
        const int n = l / a.mb;
        c.n0 = n * GRP_BN;
        c.m0 = (l - n * a.mb) * GRP_BM;
        c.r0 = s_off[c.e];
        c.r1 = s_off[c.e + 1];
        c.kb = (c.r1 - c.r0 + GRP_BK - 1) / GRP_BK;
    } else {
        // Expert by expert, column block by column block: the row tiles that read the
        // same weight tile are neighbours and run at the same time.
        c.e = find_expert(s_tile, a.E, a.nb, t);
        const int mt = s_tile[c.e + 1] - s_tile[c.e];
        const int l = t - s_tile[c.e] * a.nb;
        const int n = l / mt;
        c.n0 = n * GRP_BN;
        c.m0 = 0;
        c.r0 = s_off[c.e] + (l - n * mt) * GRP_BM;
        c.r1 = min(c.r0 + GRP_BM, s_off[c.e + 1]);
        c.kb = (a.red + GRP_BK - 1) / GRP_BK;
    }
    return c;
}

// Maps (wide, for columns that are a multiple of 64: an MN-major operand with its columns
// in blocks of 64 as a dimension of their own, so that one load brings all of a tile's
// boxes; a load costs its issuer 75-150 cycles, and six of them were more than a k-block's
// MMAs).  forward: mA x [rows, K] box 64 x 128 rows, mB W [E, M, K] box 64 x 256 x 1,
// mOut y [rows, M] box 64 x 32.  dgrad: mA dy [rows, M] box 64 x 128, mB W box
// 64 x 64 x 1, mOut dx [rows, K].  wgrad: mA dy box 64 x 64, mB x [rows, K] box
// 64 x 64, mOut dW [E, M, K] box 64 x 32 x 1.
//
// SPLIT, for few tiles with a long sum: the blocks of a cluster (2, 4 or 8) take a tile's
// k-blocks in equal shares, one tile a cluster.  The accumulators are cut into 16 parts of
// 32 rows x 64 columns; part p is finished by block p % split, which gets the others' sums
// through distributed shared memory (over the ring, which is empty by then) and adds them
// in the blocks' order.
template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(GrpCfg<MODE>::THREADS, 1)
    grouped_product_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                           const __grid_constant__ CUtensorMap mOut, const GroupedArgs a) {
    using C = GrpCfg<MODE>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + GRP_STAGES;
    uint64_t *tfull = empty + GRP_STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_off = reinterpret_cast<int *>(smem + C::TAB_OFF);
    int *s_tile = MODE == GRP_WGRAD ? nullptr : s_off + GRP_MAXE + 1;

    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int s = 0; s < GRP_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], C::EPI);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mA);
        tma_prefetch_desc(&mB);
        tma_prefetch_desc(&mOut);
    }
    // Nothing above touches global memory; all that follows comes after the previous
    // kernel of the stream.
    grid_dep_wait();
    grid_dep_launch_dependents();
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == 2)
        grouped_table(a.offsets, a.E, a.rows, GRP_BM, s_off, s_tile, blockIdx.x == 0, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = MODE == GRP_WGRAD ? a.E * a.nb * a.mb : s_tile[a.E] * a.nb;
    const uint64_t limit = a.wait_limit_ns;
    const int split = SPLIT ? a.split : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
    const int tile0 = blockIdx.x / split, step = gridDim.x / split;

    // An epilogue warp stores 32 rows (32 q ...) x 64 columns (64 ch ...) of a tile, a lane's
    // row in v.  wgrad's rows past M are clipped by the store's map; in the other modes a
    // part of 32 rows inside the segment is stored by TMA, a ragged one by each row's thread.
    auto emit = [&](const GroupedTile &c, int q, int ch, const uint32_t (&v)[2][32]) {
        uint8_t *stg = smem + C::STG_OFF + (warp - 2) * GRP_OUT_BUF + lane * 128; // this lane's row
        const int first = q * 32, col = c.n0 + ch * 64;
        const int rows = (MODE == GRP_WGRAD ? a.M - c.m0 : c.r1 - c.r0) - first;
        uint4 u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t *f = &v[j / 4][(j % 4) * 8];
            u[j] = make_uint4(pack_bf16x2(__uint_as_float(f[0]), __uint_as_float(f[1])),
                              pack_bf16x2(__uint_as_float(f[2]), __uint_as_float(f[3])),
                              pack_bf16x2(__uint_as_float(f[4]), __uint_as_float(f[5])),
                              pack_bf16x2(__uint_as_float(f[6]), __uint_as_float(f[7])));
        }
        if (MODE == GRP_WGRAD || rows >= 32) {
            if (lane == 0) bulk_wait_group_read<0>(); // the last box has left the buffer
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) // at the places of the 128-byte swizzle
                *reinterpret_cast<uint4 *>(stg + ((j ^ (lane & 7)) << 4)) = u[j];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (MODE == GRP_WGRAD)
                    tma_store_3d(&mOut, stg, col, c.m0 + first, c.e);
                else
                    tma_store_2d(&mOut, stg, col, c.r0 + first);
                bulk_commit_group();
            }
        } else if (lane < rows) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                   (size_t)(c.r0 + first + lane) * a.ncols + col);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + 8 * j < a.ncols) dst[j] = u[j];
        }
    };

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = tile0; t < total && ok; t += step) {
                const GroupedTile c = grouped_tile<MODE>(t, a, s_off, s_tile);
                // Column blocks of one row tile start at different k-blocks, so they do
                // not all ask for the same rows at once.  (wgrad keeps the order: its
                // last k-block is the one that is cut.)
                const int rot = MODE == GRP_WGRAD || SPLIT ? 0 : (c.n0 / GRP_BN) % c.kb;
                for (int i = c.kb * rank / split; i < c.kb * (rank + 1) / split; ++i, ++it) {
                    const int kb = i + rot < c.kb ? i + rot : i + rot - c.kb;
                    const uint32_t s = it % GRP_STAGES, ph = (it / GRP_STAGES) & 1;
                    if (!mbar_wait(&empty[s], ph ^ 1, limit, abort_flag, 301)) { ok = false; break; }
                    uint8_t *sa = ring + s * GRP_STAGE_BYTES, *sb = sa + GRP_A_BYTES;
                    mbar_arrive_expect_tx(&full[s], GRP_STAGE_BYTES);
                    const int kx = kb * GRP_BK;
                    if (MODE == GRP_FORWARD) {
                        tma_load_2d(&mA, &full[s], sa, kx, c.r0);
                        tma_load_3d(&mB, &full[s], sb, kx, c.n0, c.e);
                    } else if (MODE == GRP_DGRAD) {
                        tma_load_2d(&mA, &full[s], sa, kx, c.r0);
                        if (a.wide) {
                            tma_load_4d(&mB, &full[s], sb, 0, kx, c.n0 / 64, c.e);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tma_load_3d(&mB, &full[s], sb + j * GRP_CHUNK, c.n0 + 64 * j, kx, c.e);
                        }
                    } else if (a.wide) {
                        tma_load_3d(&mA, &full[s], sa, 0, c.r0 + kx, c.m0 / 64);
                        tma_load_3d(&mB, &full[s], sb, 0, c.r0 + kx, c.n0 / 64);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d(&mA, &full[s], sa + j * GRP_CHUNK, c.m0 + 64 * j, c.r0 + kx);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tma_load_2d(&mB, &full[s], sb + j * GRP_CHUNK, c.n0 + 64 * j, c.r0 + kx);
                    }
                }
            }
            drain_copies(full, GRP_STAGES, it, limit, abort_flag, 302);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------ MMA issuer --------------------------------
        // The whole warp walks the loop (it zeroes the rows past a segment's end);
        // lane 0 waits and issues.
        uint32_t it = 0, tc = 0;
        bool ok = true;
        if (a.never_signal && tile0 < total) {
            if (lane == 0) ok = mbar_wait(drain, 0, limit, abort_flag, 310);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        for (int t = tile0; t < total && ok; t += step) {
            const GroupedTile c = grouped_tile<MODE>(t, a, s_off, s_tile);
            const int i0 = c.kb * rank / split, i1 = c.kb * (rank + 1) / split;
            if (i0 == i1) continue; // wgrad of an expert without rows (or with few): zeros
            const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
            ++tc;
            // only the columns that exist, in steps of 16
            const int n = min(GRP_BN, (a.ncols - c.n0 + 15) & ~15);
            const uint32_t idesc = umma_idesc_bf16(GRP_BM, n) | (MODE == GRP_WGRAD ? UMMA_A_MN : 0u) |
                                   (MODE != GRP_FORWARD ? UMMA_B_MN : 0u);
            if (lane == 0) ok = mbar_wait(&tempty[acc], aph ^ 1, limit, abort_flag, 311);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * GRP_BN;
            for (int i = i0; i < i1; ++i, ++it) {
                const uint32_t s = it % GRP_STAGES, ph = (it / GRP_STAGES) & 1;
                if (lane == 0) ok = mbar_wait(&full[s], ph, limit, abort_flag, 312);
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                int steps = GRP_BK / 16;
                if (MODE == GRP_WGRAD && i == c.kb - 1) {
                    const int valid = c.r1 - c.r0 - i * GRP_BK; // rows of this k-block, 1..64
                    steps = (valid + 15) >> 4;
                    const int pad = steps * 16 - valid;
                    if (pad) {
                        uint4 *p = reinterpret_cast<uint4 *>(ring + s * GRP_STAGE_BYTES);
                        for (int j = lane; j < 6 * 8 * pad; j += 32) {
                            const int box = j / (8 * pad), o = j - box * 8 * pad;
                            p[box * (GRP_CHUNK / 16) + valid * 8 + o] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring + s * GRP_STAGE_BYTES);
                    const uint32_t sb = sa + GRP_A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < GRP_BK / 16; ++kk) {
                        if (MODE == GRP_WGRAD && kk >= steps) break;
                        const uint64_t da = MODE == GRP_WGRAD
                                                ? umma_desc_sw128_mn(sa + kk * 2048, GRP_CHUNK)
                                                : umma_desc_sw128(sa + kk * 32);
                        const uint64_t db = MODE != GRP_FORWARD
                                                ? umma_desc_sw128_mn(sb + kk * 2048, GRP_CHUNK)
                                                : umma_desc_sw128(sb + kk * 32);
                        umma_bf16_ss(d_tmem, da, db, idesc, (i > i0 || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(&empty[s]);
                }
            }
            if (!ok) break;
            if (lane == 0) umma_commit(&tfull[acc]);
        }
        if (lane == 0) {
            // Drain: wait until every MMA issued by this thread has completed.
            umma_commit(drain);
            settle(drain, 0, limit, abort_flag, 100000000ull, 313);
        }
        __syncwarp();
    } else if (SPLIT) {
        if (tile0 < total && lane == 0) {
            const GroupedTile c = grouped_tile<MODE>(tile0, a, s_off, s_tile);
            if (c.kb * rank / split < c.kb * (rank + 1) / split) mbar_wait(&tfull[0], 0, limit, abort_flag, 321);
        }
        __syncwarp();
    } else {
        // ------------------------------ epilogue ---------------------------------
        const int q = warp & 3; // TMEM lane quadrant: output rows q*32 + lane of the tile
        const int part = (warp - 2) >> 2; // of the tile's columns
        uint32_t tc = 0;
        for (int t = tile0; t < total; t += step) {
            const GroupedTile c = grouped_tile<MODE>(t, a, s_off, s_tile);
            const bool none = c.kb == 0; // nothing accumulated: zeros
            const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
            bool have = none;
            if (!none) {
                ++tc;
                if (lane == 0) have = mbar_wait(&tfull[acc], aph, limit, abort_flag, 321);
                have = __shfl_sync(0xffffffffu, have ? 1 : 0, 0) != 0;
            }
            __syncwarp();
            if (!have) continue;
            tc_fence_after();
            const uint32_t tbase = tmem_base + acc * GRP_BN + ((uint32_t)(q * 32) << 16);
            const int first = q * 32; // this warp's rows of the tile
            const int rows = (MODE == GRP_WGRAD ? a.M - c.m0 : c.r1 - c.r0) - first;
            if (none) {
                // zeros: one row after the other, whole lines at a time
                const int cols = min(GRP_BN, a.ncols - c.n0) / 8;
                for (int r = part; r < min(32, rows); r += C::EPI / 4)
                    if (lane < cols)
                        reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                  ((size_t)c.e * a.M + c.m0 + first + r) * a.ncols + c.n0)[lane] =
                            make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            // 64 columns at a time: while one box is read from shared memory, the next
            // columns come from TMEM (boxes of 32 columns, two in turn: 1300 cycles each,
            // more than the MMAs of a short tile).
#pragma unroll 1
            for (int ch = part * C::COLS / 64; ch < (part + 1) * C::COLS / 64; ++ch) {
                const int col = c.n0 + ch * 64;
                if (col >= a.ncols || rows <= 0) break;
                uint32_t v[2][32];
                tmem_ld_32x32b_x32(tbase + ch * 64, v[0]);
                tmem_ld_32x32b_x32(tbase + ch * 64 + 32, v[1]);
                tmem_ld_wait();
                emit(c, q, ch, v);
            }
            // Release the accumulator.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[acc]);
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync_all(); // every block's ring has been read
        if (warp >= 2 && tile0 < total) {
            const GroupedTile c = grouped_tile<MODE>(tile0, a, s_off, s_tile);
            const int q = warp & 3, rows = (MODE == GRP_WGRAD ? a.M - c.m0 : c.r1 - c.r0) - q * 32;
            const int part = (warp - 2) >> 2;
            tc_fence_after();
            if (c.kb * rank / split < c.kb * (rank + 1) / split && rows > 0) {
#pragma unroll 1
                for (int ch = part * C::COLS / 64; ch < (part + 1) * C::COLS / 64; ++ch) {
                    if (c.n0 + ch * 64 >= a.ncols) break;
                    uint32_t v[2][32];
                    const uint32_t from = tmem_base + ((uint32_t)(q * 32) << 16) + ch * 64;
                    tmem_ld_32x32b_x32(from, v[0]);
                    tmem_ld_32x32b_x32(from + 32, v[1]);
                    tmem_ld_wait();
                    // [own part][block][column][row]
                    const int p = q * 4 + ch;
                    const uint32_t to = mapa_shared(
                        smem_u32(ring) + (uint32_t)(((p / split) * split + rank) * 64 * 32 + lane) * 4, p % split);
#pragma unroll
                    for (int j = 0; j < 64; ++j) st_cluster_f32(to + j * 128, __uint_as_float(v[j / 32][j % 32]));
                }
            }
        }
        __syncwarp();
        cluster_sync_all(); // all sums are there
        if (warp >= 2 && tile0 < total) {
            const GroupedTile c = grouped_tile<MODE>(tile0, a, s_off, s_tile);
            for (int own = warp - 2; own < 16 / split; own += C::EPI) {
                const int p = own * split + rank, q = p / 4, ch = p % 4;
                const int rows = (MODE == GRP_WGRAD ? a.M - c.m0 : c.r1 - c.r0) - q * 32;
                if (c.n0 + ch * 64 >= a.ncols || rows <= 0) continue;
                uint32_t v[2][32];
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j / 32][j % 32] = 0;
                for (int r = 0; r < split; ++r) {
                    if (c.kb * r / split == c.kb * (r + 1) / split) continue; // nothing summed there
                    const float *from = reinterpret_cast<const float *>(ring) + (own * split + r) * 64 * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        v[j / 32][j % 32] = __float_as_uint(__uint_as_float(v[j / 32][j % 32]) + from[j * 32]);
                }
                emit(c, q, ch, v);
            }
        }
    }
    if (warp >= 2) {
        if (lane == 0) bulk_wait_group<0>(); // stores done
        if (MODE != GRP_WGRAD && a.zero_rest)
            grouped_zero_rest(a.out, a.rows, (size_t)a.ncols * 2, s_off[0], s_off[a.E],
                              (size_t)blockIdx.x * 128 + (threadIdx.x - 64), (size_t)gridDim.x * 128);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// fp32: the same three products on the CUDA cores, T x T output tiles, KB summed indices
// at a time in shared memory, fp32 sums in registers, one running sum each, in index
// order; the next KB (T = 64: the next two, 111 to 86 us for the input gradient of 2048
// rows, 16 x 768 x 768; T = 32 lost 30 % by it) are on their way from memory meanwhile.  The
// summed index never crosses a segment, so nothing is masked but loads.  Large batches
// take T = 64 with 8 x 8 sums a thread (four 16-byte shared loads for 64 multiply-adds;
// with 4 x 4 the shared memory's bandwidth is the bound), small ones T = 32 with 4 x 4:
// more tiles for the same SMs.
// ---------------------------------------------------------------------------
// Element (k, i) of an operand in shared memory; loads are 16 bytes along the contiguous
// index: the summed one (KCONT) or the other.
template <bool KCONT, int T, int KB, int NT> struct F32Operand {
    static constexpr int PER = KB * T / 4 / NT; // pieces of a thread
    float4 v[PER];
    static constexpr int LD = T == 32 ? T : T + 4;
    // Where 4 indices i.. of row k lie.  KCONT stores a piece as four scalars of four rows: with
    // T = 32 the xor spreads a warp's over all banks.
    static __device__ __forceinline__ int place(int k, int i) { return KCONT && T == 32 ? i ^ (k & 28) : i; }
    // rows: of the contiguous direction's other index; ld: elements from one to the next
    __device__ __forceinline__ void load(const float *p, size_t ld, int nk, int ni, int tid) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at = tid + j * NT;
            const int k = KCONT ? at % (KB / 4) * 4 : at / (T / 4), i = KCONT ? at / (KB / 4) : at % (T / 4) * 4;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < nk && i < ni) // counts along the contiguous index are multiples of 4
                v[j] = *reinterpret_cast<const float4 *>(p + (KCONT ? (size_t)i * ld + k : (size_t)k * ld + i));
        }
    }
    __device__ __forceinline__ void store(float (*s)[LD], int tid) const {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at = tid + j * NT;
            if (KCONT) {
                const int k = at % (KB / 4) * 4, i = at / (KB / 4);
                const int c = place(k, i);
                s[k][c] = v[j].x;
                s[k + 1][c] = v[j].y;
                s[k + 2][c] = v[j].z;
                s[k + 3][c] = v[j].w;
            } else {
                *reinterpret_cast<float4 *>(&s[at / (T / 4)][at % (T / 4) * 4]) = v[j];
            }
        }
    }
};

template <int V> struct IntC { static constexpr int value = V; };
template <int T> struct GrpF32 {
    static constexpr int SUMS = T == 64 ? 8 : 4; // of a thread, in each direction
    static constexpr int KB = T == 64 ? 16 : 32;
    static constexpr int AHEAD = T == 64 ? 2 : 1; // blocks of KB on their way
    static constexpr int THREADS = (T / SUMS) * (T / SUMS);
};

template <int MODE, int T>
__global__ void __launch_bounds__(GrpF32<T>::THREADS) grouped_f32_kernel(const float *A, const float *B,
                                                                         const GroupedArgs a) {
    constexpr int S = GrpF32<T>::SUMS, NT = GrpF32<T>::THREADS, KB = GrpF32<T>::KB, H = S / 4;
    constexpr int AHEAD = GrpF32<T>::AHEAD;
    using FA = F32Operand<MODE != GRP_WGRAD, T, KB, NT>;
    using FB = F32Operand<MODE == GRP_FORWARD, T, KB, NT>;
    __shared__ __align__(16) float sA[KB][FA::LD], sB[KB][FB::LD];
    __shared__ int s_off[GRP_MAXE + 1], s_tile[GRP_MAXE + 1];
    const int tid = threadIdx.x;
    grid_dep_wait(); // all that follows comes after the previous kernel of the stream
    grid_dep_launch_dependents();
    if (tid < 32) grouped_table(a.offsets, a.E, a.rows, T, s_off, s_tile, blockIdx.x == 0, tid);
    __syncthreads();
    const int total = MODE == GRP_WGRAD ? a.E * a.nb * a.mb : s_tile[a.E] * a.nb;
    const int tx = tid % (T / S), ty = tid / (T / S); // places 4 tx.. (and T/2 + 4 tx..), 4 ty..
    float *out = static_cast<float *>(a.out);
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        int e, i0, i1, n0, r0, red;
        if (MODE == GRP_WGRAD) {
            const int per = a.nb * a.mb;
            e = t / per;
            const int l = t - e * per;
            n0 = (l / a.mb) * T;
            i0 = (l % a.mb) * T;
            i1 = min(i0 + T, a.M);
            r0 = s_off[e];
            red = s_off[e + 1] - r0;
        } else {
            e = find_expert(s_tile, a.E, a.nb, t);
            const int mt = s_tile[e + 1] - s_tile[e], l = t - s_tile[e] * a.nb;
            n0 = (l / mt) * T;
            i0 = s_off[e] + (l % mt) * T;
            i1 = min(i0 + T, s_off[e + 1]);
            r0 = 0;
            red = a.red;
        }
        const float *We = B + (size_t)e * a.M * a.K; // forward, dgrad
        FA fa[AHEAD]; // forward x[i][k], dgrad dy[i][k], wgrad dy[r0+k][i]
        FB fb[AHEAD]; // forward W[n][k], dgrad W[k][n], wgrad x[r0+k][n]
        auto fetch = [&](auto slot, int k0) {
            auto &va = fa[decltype(slot)::value];
            auto &vb = fb[decltype(slot)::value];
            if (MODE == GRP_WGRAD) {
                va.load(A + (size_t)(r0 + k0) * a.M + i0, a.M, red - k0, i1 - i0, tid);
                vb.load(B + (size_t)(r0 + k0) * a.K + n0, a.K, red - k0, a.ncols - n0, tid);
            } else {
                va.load(A + (size_t)i0 * a.red + k0, a.red, red - k0, i1 - i0, tid);
                if (MODE == GRP_FORWARD)
                    vb.load(We + (size_t)n0 * a.K + k0, a.K, red - k0, a.ncols - n0, tid);
                else
                    vb.load(We + (size_t)k0 * a.K + n0, a.K, red - k0, a.ncols - n0, tid);
            }
        };
        float acc[S][S] = {};
        auto block = [&](auto slot, int k0) {
            fa[decltype(slot)::value].store(sA, tid);
            fb[decltype(slot)::value].store(sB, tid);
            __syncthreads();
            if (k0 + AHEAD * KB < red) fetch(slot, k0 + AHEAD * KB);
#pragma unroll 8
            for (int k = 0; k < KB; ++k) {
                float xa[S], wb[S];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sA[k][FA::place(k, h * (T / 2) + ty * 4)]);
                    const float4 w = *reinterpret_cast<const float4 *>(&sB[k][FB::place(k, h * (T / 2) + tx * 4)]);
                    xa[4 * h] = x.x, xa[4 * h + 1] = x.y, xa[4 * h + 2] = x.z, xa[4 * h + 3] = x.w;
                    wb[4 * h] = w.x, wb[4 * h + 1] = w.y, wb[4 * h + 2] = w.z, wb[4 * h + 3] = w.w;
                }
#pragma unroll
                for (int i = 0; i < S; ++i)
#pragma unroll
                    for (int n = 0; n < S; ++n) acc[i][n] = fmaf(xa[i], wb[n], acc[i][n]);
            }
            __syncthreads();
        };
        if (red > 0) fetch(IntC<0>{}, 0);
        if (AHEAD > 1 && red > KB) fetch(IntC<AHEAD - 1>{}, KB);
        for (int k0 = 0; k0 < red; k0 += AHEAD * KB) {
            block(IntC<0>{}, k0);
            if (AHEAD > 1 && k0 + KB < red) block(IntC<AHEAD - 1>{}, k0 + KB);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int n = n0 + h * (T / 2) + tx * 4;
            if (n >= a.ncols) break;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int row = i0 + (i / 4) * (T / 2) + ty * 4 + i % 4;
                if (row < i1) {
                    const size_t at = MODE == GRP_WGRAD ? (size_t)e * a.M + row : (size_t)row;
                    *reinterpret_cast<float4 *>(out + at * a.ncols + n) =
                        make_float4(acc[i][4 * h], acc[i][4 * h + 1], acc[i][4 * h + 2], acc[i][4 * h + 3]);
                }
            }
        }
    }
    if (MODE != GRP_WGRAD && a.zero_rest)
        grouped_zero_rest(a.out, a.rows, (size_t)a.ncols * 4, s_off[0], s_off[a.E],
                          (size_t)blockIdx.x * NT + tid, (size_t)gridDim.x * NT);
}

}  // namespace moe
