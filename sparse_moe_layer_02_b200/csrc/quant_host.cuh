// Host side of the 4-bit weights (moe_quantize, moe_dequantize, moe_linear_quant,
// moe_forward_quant).  Part of moe.cu's translation unit.
#pragma once

#include "quant.cuh"

namespace moe {
namespace {

bool quant_group_ok(int G) { return G == 32 || G == 64 || G == 128; }

// E matrices [M, K] of codes.
bool quant_shape_ok(int E, int M, int K, int G) {
    return quant_group_ok(G) && E > 0 && E <= 65535 && M > 0 && M <= (1 << 20) && M % 8 == 0 && K > 0 &&
           K <= (1 << 24) && K % G == 0;
}

// Maps of the codes and scales of E matrices [M, K] for the tiles of a configuration.
template <int RG, int MT, int KW>
bool make_quant_maps(CUtensorMap *mW, CUtensorMap *mS, const void *q, const void *s, int E, int M, int K,
                     int G, bool halves) {
    using C = QmCfg<RG, MT, KW, 1, 32>; // the boxes do not depend on NT and G
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t half = (cuuint64_t)K / 2, groups = (cuuint64_t)K / G;
    cuuint32_t estr[3] = {1, 1, 1};
    cuuint64_t wd[3] = {half, (cuuint64_t)M, (cuuint64_t)E};
    cuuint64_t ws[2] = {half, half * M};
    const cuuint32_t rows = halves ? C::HALF : C::R;
    cuuint32_t wb[3] = {C::BOX, rows, 1};
    cuuint64_t sd[3] = {(cuuint64_t)M, groups, (cuuint64_t)E};
    cuuint64_t ss[2] = {(cuuint64_t)M * 2, (cuuint64_t)M * 2 * groups};
    cuuint32_t sb[3] = {rows, (cuuint32_t)(C::SK / G), 1};
    return fn(mW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(q), wd, ws, wb, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              C::BOX == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           fn(mS, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(s), sd, ss, sb, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks that share a tile: as many as still run all at once (clusters do not fill every
// place, so two thirds of them are counted on), each with two stages of columns at least.
// A block alone on an SM has too few warps to hide its latencies: one token, groups of 128,
// 2816 x 4096 (22 tiles) takes 11.0 us unshared, 8.6 shared by 2 and 7.4 by 8; 6144 x 6144 (48)
// 15.5, 11.4 by 2 and 10.9 by 4; 12288 x 5120 (96) 14.1 and 14.3 by 2 (8 tokens 17.0 and 15.7).
// Sharing when the tiles already take several rounds costs: the exchange (2 us) then stalls
// the next tile's reading.
int quant_split(size_t tiles, size_t slots, int stages) {
    int best = 1;
    for (int c = 2; c <= 8 && tiles * c * 3 <= slots * 2 && stages >= 2 * c; c *= 2) best = c;
    return best;
}

template <int KIND, int RG, int MT, int KW, int NT, int G>
int launch_quant_g(const CUtensorMap &mW, const CUtensorMap &mS, const CUtensorMap &mW_s,
                 const CUtensorMap &mS_s, const QuantArgs &a, size_t tiles, DeviceInfo *info,
                 cudaStream_t st) {
    using C = QmCfg<RG, MT, KW, NT, G>;
    static bool attr_set[kMaxDevices] = {}; // function attributes are set per device
    const int dev = current_device_index();
    if (dev < 0) return MOE_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(quant_product_kernel<KIND, RG, MT, KW, NT, G>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
                return MOE_ERR_CUDA;
            attr_set[dev] = true;
        }
    }
    const size_t slots = (size_t)info->sms * C::BLOCKS;
    QuantArgs b = a;
    b.split = C::KS > 1 ? quant_split(tiles, slots, (std::max(a.K, a.K_s) + C::SK - 1) / C::SK) : 1;
    return launch_clusters(quant_product_kernel<KIND, RG, MT, KW, NT, G>, b.split,
                           (int)(std::min<size_t>(tiles, slots / b.split) * b.split), QM_THREADS, C::SMEM, st, mW, mS,
                           mW_s, mS_s, b);
}

template <int KIND, int RG, int MT, int KW, int NT>
int launch_quant(const CUtensorMap &mW, const CUtensorMap &mS, const CUtensorMap &mW_s,
                 const CUtensorMap &mS_s, const QuantArgs &a, size_t tiles, DeviceInfo *info,
                 cudaStream_t st) {
    switch (a.G) {
    case 32: return launch_quant_g<KIND, RG, MT, KW, NT, 32>(mW, mS, mW_s, mS_s, a, tiles, info, st);
    case 64: return launch_quant_g<KIND, RG, MT, KW, NT, 64>(mW, mS, mW_s, mS_s, a, tiles, info, st);
    default: return launch_quant_g<KIND, RG, MT, KW, NT, 128>(mW, mS, mW_s, mS_s, a, tiles, info, st);
    }
}

template <int RG, int MT, int KW, int NT>
int linear_quant_t(const void *q, const void *s, QuantArgs a, DeviceInfo *info, cudaStream_t st) {
    constexpr int R = 16 * MT * RG;
    CUtensorMap mW, mS;
    if (!make_quant_maps<RG, MT, KW>(&mW, &mS, q, s, 1, a.ncols, a.K, a.G, false)) return MOE_ERR_CUDA;
    a.nb = (a.ncols + R - 1) / R;
    const size_t tiles = (size_t)a.nb * ((a.N + 8 * NT - 1) / (8 * NT));
    return launch_quant<QUANT_LINEAR, RG, MT, KW, NT>(mW, mS, mW, mS, a, tiles, info, st);
}

// Blocks that share a tile of the wide product: its time is that of the tiles one after the
// other, each its share of the stages (0.6 us each with groups of 128) and what filling the
// pipeline and joining the sums take, about six stages' time with a cluster and one without
// (24 tokens through this kernel: 3 rounds of shares by 4 took 35 us where one round unshared
// took 29.5 for 12288 x 5120; 2816 x 4096, 22 row tiles on 148 SMs, took 11.4 shared by 6 and
// 23.7 unshared).
struct WideSplit {
    int split, grid;
};
WideSplit quant_wide_split(const int (&clusters)[9], size_t tiles, int stages) {
    WideSplit best = {1, (int)std::min<size_t>(tiles, clusters[1])};
    size_t least = SIZE_MAX;
    for (int c = 1; c <= 8; ++c) {
        if (clusters[c] <= 0 || stages < 2 * c) continue;
        const size_t n = std::min<size_t>(tiles, clusters[c]);
        const size_t time = ((tiles + n - 1) / n) * ((stages + c - 1) / c + (c > 1 ? 6 : 1));
        if (time < least) {
            least = time;
            best = {c, (int)n * c};
        }
    }
    return best;
}

template <int G>
int launch_quant_wide(const CUtensorMap &mC, const CUtensorMap &mX, QuantWideArgs a, DeviceInfo *info,
                      cudaStream_t st) {
    static int clusters[kMaxDevices][9] = {}; // of 1 to 8 blocks that run at once; found once per device
    const int dev = current_device_index();
    if (dev < 0) return MOE_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!clusters[dev][1]) {
            for (auto kernel : {quant_wide_kernel<G, false>, quant_wide_kernel<G, true>})
                if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, QW_SMEM) !=
                    cudaSuccess)
                    return MOE_ERR_CUDA;
            for (int c = 2; c <= 8; ++c)
                clusters[dev][c] = clusters_at_once(quant_wide_kernel<G, true>, c, QW_THREADS, QW_SMEM, info->sms);
            clusters[dev][1] = info->sms;
        }
    }
    const WideSplit w = quant_wide_split(clusters[dev], (size_t)a.nb * a.tts, (a.K + QW_COLS - 1) / QW_COLS);
    a.split = w.split;
    a.own = (a.tok + w.split - 1) / w.split;
    return launch_clusters(w.split > 1 ? quant_wide_kernel<G, true> : quant_wide_kernel<G, false>, w.split, w.grid,
                           QW_THREADS, QW_SMEM, st, mC, mX, a);
}

// y = x w^T for any number of tokens, on tcgen05.
int linear_quant_wide(const void *x, const void *q, const void *s, int N, int M, int K, int G, void *y,
                      DeviceInfo *info, cudaStream_t st) {
    QuantWideArgs a = {};
    a.s = static_cast<const __nv_bfloat16 *>(s);
    a.y = static_cast<__nv_bfloat16 *>(y);
    a.N = N;
    a.M = M;
    a.K = K;
    a.tts = (N + QW_TOK - 1) / QW_TOK;
    a.tok = ((N + a.tts - 1) / a.tts + 15) / 16 * 16; // even tiles
    a.tts = (N + a.tok - 1) / a.tok;
    a.nb = (M + QW_ROWS - 1) / QW_ROWS;
    a.ld = (a.tok + 31) / 32 * 32;
    a.accs = std::min(QW_UCOL / a.ld, QW_MAXACC) / (G < QW_COLS ? 2 : 1);
    a.wait_limit_ns = g_wait_limit_ns;
    a.never_signal = g_never_signal;
    CUtensorMap mC, mX;
    auto fn = encode_fn();
    if (!fn) return MOE_ERR_CUDA;
    cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)M};
    cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    cuuint32_t box[2] = {QW_COLS / 2, QW_ROWS};
    cuuint32_t estr[2] = {1, 1};
    if (fn(&mC, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        !make_map(&mX, x, K, N, K, a.tok))
        return MOE_ERR_CUDA;
    switch (G) {
    case 32: return launch_quant_wide<32>(mC, mX, a, info, st);
    case 64: return launch_quant_wide<64>(mC, mX, a, info, st);
    default: return launch_quant_wide<128>(mC, mX, a, info, st);
    }
}

// ---- the layer ----
struct QuantWs {
    size_t chunk_hist, counts, tile_off, meta, pos_of, perm_tok, w_perm, h, h_s, slot, osh, total;
    int nchunks;
    size_t rows_max;
    int tile_rows;
    bool direct;
};

// Tokens of a tile.  Tiles of 8 leave room for more stages of codes, tiles of 16 read an
// expert's codes once where its tokens are more than 8 (us for the layer, 8 / 16): D 4096,
// 128 experts of 1408, k 8: 12 tokens 149 / 157, 32 219 / 229, 64 265 / 272, 96 319 / 301,
// 128 387 / 334; D 4096, 40 of 1024, k 4: 32 tokens 89 / 95, 48 (4.8 an expert) 97 / 98, 64
// 103 / 101 to 107, 96 142 / 123.  The shared expert's codes are read again by every tile of
// tokens: D 6144, 256 of 2048, k 8, groups of 64, 128 tokens (four an expert) 1146 / 1088.
// (Small layers, with fewer tiles than places, would gain from 8 for longer: D 1024, 8 of 512,
// k 2: 64 tokens 20 / 22, 100 26 / 24.)  Tiles of 32 leave one block an SM and were slower
// everywhere: the first at 512 tokens 1182, against 893.
int quant_tile_tokens(int N, int k, int E) {
    return N <= 8 || (N <= 64 && (size_t)N * k <= (size_t)4 * E) ? 8 : 16;
}

bool plan_quant(int N, int D, int E, int d, int d_sh, int k, QuantWs &W) {
    const size_t nk = (size_t)N * k;
    if (nk > (size_t)INT32_MAX / 4) return false;
    W.direct = N == 1;
    W.tile_rows = quant_tile_tokens(N, k, E);
    W.rows_max = W.direct ? nk : nk + (size_t)(W.tile_rows - 1) * std::min<size_t>(E, std::max<size_t>(nk, 1));
    if (W.rows_max > (size_t)INT32_MAX / 4) return false;
    W.nchunks = (int)((nk + DISPATCH_CHUNK - 1) / DISPATCH_CHUNK);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = round_up(off + bytes, 256);
        return at;
    };
    W.chunk_hist = take((size_t)std::max(W.nchunks, 1) * E * 4);
    W.counts = take((size_t)E * 4);
    W.tile_off = take((size_t)(E + 1) * 4);
    W.meta = take(16 * 4);
    W.pos_of = take(nk * 4);
    W.perm_tok = take(W.rows_max * 4);
    W.w_perm = take(W.rows_max * 4);
    W.h = take(W.rows_max * d * 2);
    W.h_s = take((size_t)N * d_sh * 2);
    W.slot = take(W.rows_max * D * 4);
    W.osh = take((size_t)N * D * 4);
    W.total = off;
    return true;
}

bool quant_layer_shape_ok(int N, int D, int E, int d, int d_sh, int k, int G) {
    return N >= 0 && N <= (1 << 24) && k > 0 && k <= 32 && E <= DISPATCH_MAXE && d <= (1 << 19) &&
           d_sh <= (1 << 19) && quant_shape_ok(E, 2 * d, D, G) && quant_shape_ok(E, D, d, G) &&
           quant_shape_ok(1, 2 * d_sh, D, G) && quant_shape_ok(1, D, d_sh, G);
}

// A layer that moe_forward_quant takes, with its plan; tile numbers are 32-bit.
bool quant_layer_ok(int N, int D, int E, int d, int d_sh, int k, int G, QuantWs &W) {
    return quant_layer_shape_ok(N, D, E, d, d_sh, k, G) && plan_quant(N, D, E, d, d_sh, k, W) &&
           (W.rows_max / 8 + 1) * ((size_t)std::max(D, std::max(d, d_sh)) / 32 + 1) +
                   ((size_t)N / 8 + 1) * ((size_t)std::max(D, d_sh) / 16 + 1) <= (size_t)INT32_MAX / 2;
}

struct QuantLayer {
    const void *gu, *gu_s, *dn, *dn_s, *sgu, *sgu_s, *sdn, *sdn_s;
    int D, d, d_sh;
};

template <int RG, int MT, int KW, int NT>
int quant_layer_t(const QuantLayer &w, QuantArgs a, const void *x, uint8_t *ws, const QuantWs &W,
                  DeviceInfo *info, Profiler &prof, cudaStream_t st) {
    constexpr int R = 16 * MT * RG;
    const int tt_s = (a.N + 8 * NT - 1) / (8 * NT);
    const size_t tt_r = W.direct ? (size_t)a.k : W.rows_max / (8 * NT) + 1;
    CUtensorMap mW, mS, mWs, mSs;
    // gate and up rows, SwiGLU
    if (!make_quant_maps<RG, MT, KW>(&mW, &mS, w.gu, w.gu_s, a.E, 2 * w.d, w.D, a.G, true) ||
        !make_quant_maps<RG, MT, KW>(&mWs, &mSs, w.sgu, w.sgu_s, 1, 2 * w.d_sh, w.D, a.G, true))
        return MOE_ERR_CUDA;
    a.x = a.x_s = static_cast<const uint8_t *>(x);
    a.row_bytes = a.row_bytes_s = w.D * 2;
    a.K = a.K_s = w.D;
    a.ncols = w.d;
    a.ncols_s = w.d_sh;
    a.nb = (w.d + R / 2 - 1) / (R / 2);
    a.nb_s = (w.d_sh + R / 2 - 1) / (R / 2);
    a.out = ws + W.h;
    a.out_s = ws + W.h_s;
    int rc = launch_quant<QUANT_GATE_UP, RG, MT, KW, NT>(mW, mS, mWs, mSs, a, tt_r * a.nb + (size_t)tt_s * a.nb_s,
                                                 info, st);
    if (rc != MOE_OK) return rc;
    prof.mark();
    // down
    if (!make_quant_maps<RG, MT, KW>(&mW, &mS, w.dn, w.dn_s, a.E, w.D, w.d, a.G, false) ||
        !make_quant_maps<RG, MT, KW>(&mWs, &mSs, w.sdn, w.sdn_s, 1, w.D, w.d_sh, a.G, false))
        return MOE_ERR_CUDA;
    a.x = ws + W.h;
    a.x_s = ws + W.h_s;
    a.row_bytes = w.d * 2;
    a.row_bytes_s = w.d_sh * 2;
    a.K = w.d;
    a.K_s = w.d_sh;
    a.ncols = a.ncols_s = w.D;
    a.nb = a.nb_s = (w.D + R - 1) / R;
    a.out = ws + W.slot;
    a.out_s = ws + W.osh;
    rc = launch_quant<QUANT_DOWN, RG, MT, KW, NT>(mW, mS, mWs, mSs, a, tt_r * a.nb + (size_t)tt_s * a.nb_s, info, st);
    if (rc == MOE_OK) prof.mark();
    return rc;
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_quantize(const void *W, int E, int M, int K, int group, void *q, void *scales, void *stream) {
    if (!quant_shape_ok(E, M, K, group)) return MOE_ERR_SHAPE;
    for (const void *p : {W, (const void *)q, (const void *)scales})
        if (!p || !aligned16(p)) return MOE_ERR_ARG;
    DeviceInfo *dev = nullptr;
    int rc = current_device_info(&dev);
    if (rc != MOE_OK) return rc;
    if (dev->major != 10) return MOE_ERR_NO_DEVICE;
    const dim3 grid((K + QZ_COLS - 1) / QZ_COLS, (M + QZ_ROWS - 1) / QZ_ROWS, E);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto *w = static_cast<const __nv_bfloat16 *>(W);
    auto *c = static_cast<uint8_t *>(q);
    auto *s = static_cast<__nv_bfloat16 *>(scales);
    if (group == 32)
        quantize_kernel<32><<<grid, QZ_THREADS, 0, st>>>(w, c, s, M, K);
    else if (group == 64)
        quantize_kernel<64><<<grid, QZ_THREADS, 0, st>>>(w, c, s, M, K);
    else
        quantize_kernel<128><<<grid, QZ_THREADS, 0, st>>>(w, c, s, M, K);
    return launch_status();
}

int moe_dequantize(const void *q, const void *scales, int E, int M, int K, int group, void *W, void *stream) {
    if (!quant_shape_ok(E, M, K, group)) return MOE_ERR_SHAPE;
    for (const void *p : {q, scales, (const void *)W})
        if (!p || !aligned16(p)) return MOE_ERR_ARG;
    DeviceInfo *dev = nullptr;
    int rc = current_device_info(&dev);
    if (rc != MOE_OK) return rc;
    if (dev->major != 10) return MOE_ERR_NO_DEVICE;
    const dim3 grid((K + QZ_COLS - 1) / QZ_COLS, (M + DQ_ROWS - 1) / DQ_ROWS, E);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto *c = static_cast<const uint8_t *>(q);
    const auto *s = static_cast<const __nv_bfloat16 *>(scales);
    auto *w = static_cast<__nv_bfloat16 *>(W);
    if (group == 32)
        dequantize_kernel<32><<<grid, QZ_THREADS, 0, st>>>(c, s, w, M, K);
    else if (group == 64)
        dequantize_kernel<64><<<grid, QZ_THREADS, 0, st>>>(c, s, w, M, K);
    else
        dequantize_kernel<128><<<grid, QZ_THREADS, 0, st>>>(c, s, w, M, K);
    return launch_status();
}

int moe_linear_quant(const void *x, const void *q, const void *scales, int N, int M, int K, int group,
                     void *y, void *stream) {
    if (N < 0 || N > (1 << 24) || !quant_shape_ok(1, M, K, group)) return MOE_ERR_SHAPE;
    if (((size_t)M / 32 + 1) * ((size_t)N / 8 + 1) > (size_t)INT32_MAX / 2) return MOE_ERR_SHAPE;
    if (N == 0) return MOE_OK;
    for (const void *p : {x, q, scales, (const void *)y})
        if (!p || !aligned16(p)) return MOE_ERR_ARG;
    DeviceInfo *dev = nullptr;
    int rc = current_device_info(&dev);
    if (rc != MOE_OK) return rc;
    if (dev->major != 10) return MOE_ERR_NO_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    QuantArgs a = {};
    a.x = static_cast<const uint8_t *>(x);
    a.row_bytes = K * 2;
    a.N = N;
    a.G = group;
    a.K = K;
    a.ncols = M;
    a.out = y;
    a.wait_limit_ns = g_wait_limit_ns;
    a.never_signal = g_never_signal;
    // Tiles of 8 tokens, of 16, or the tcgen05 kernel, whose sums cost more the more groups a
    // stage has (us, in this order; G the group, - not measured):
    //   8 tokens   12288 x 5120, G 64 16.3 / 16.5 / 30.9   28672 x 4096, G 64 20.3 / 20.6 / 49.1
    //   16         12288 x 5120, G 128 22.3 / 20.9 / 29.1  28672 x 4096, G 128 35.0 / 25.8 / 44.6
    //   24         12288 x 5120, G 128 22.5 / 29.7 / 29.4  28672 x 4096, G 128 46.5 / 47.4 / 45.2
    //              12288 x 5120, G 64 23.4 / 31.1 / 34.9   2816 x 4096, G 64 10.7 / 11.8 / 12.1
    //              12288 x 5120, G 32 25.1 / 35.2 / 62.4   2816 x 4096, G 32 10.8 / 12.9 / 16.5
    //   32         12288 x 5120, G 128 38.2 / 29.8 / 29.6  2816 x 4096, G 128 13.3 / 11.7 / 11.5
    //              12288 x 5120, G 64 39.6 / 31.3 / 35.0   2816 x 4096, G 64 13.5 / 12.0 / 12.2
    //   48         12288 x 5120, G 64 43.3 / 31.4 / 35.9   2816 x 4096, G 64 14.0 / 14.2 / 12.8
    //              28672 x 4096, G 64 84.7 / 66.8 / 57.2
    //              12288 x 5120, G 32 47.0 / 35.3 / 60.4   2816 x 4096, G 32 14.3 / 14.9 / 17.2
    //   64         12288 x 5120, G 32 - / 59.5 / 68.8      2816 x 4096, G 32 - / 20.0 / 18.7
    if (N <= 8 || (N > 16 && N <= 24)) return linear_quant_t<4, 2, 128, 1>(q, scales, a, dev, st);
    if (N <= (group == 32 ? 48 : group == 64 ? 32 : 16)) return linear_quant_t<4, 2, 128, 2>(q, scales, a, dev, st);
    return linear_quant_wide(x, q, scales, N, M, K, group, y, dev, st);
}

size_t moe_forward_quant_workspace(int N, int D, int E, int d_moe, int d_sh, int k) {
    QuantWs W;
    return quant_layer_ok(N, D, E, d_moe, d_sh, k, 32, W) ? W.total : 0; // what any group allows, 32 does
}

int moe_forward_quant(const void *x, const void *gate_up, const void *gate_up_scales, const void *down,
                      const void *down_scales, const void *sh_gate_up, const void *sh_gate_up_scales,
                      const void *sh_down, const void *sh_down_scales, const int32_t *topk_idx,
                      const float *topk_w, int N, int D, int E, int d_moe, int d_sh, int k, int group,
                      float gate_max, float up_max, void *y, void *workspace, size_t ws_bytes,
                      void *stream) {
    if (gate_max != gate_max || up_max != up_max || up_max < 0.f) return MOE_ERR_ARG;
    QuantWs W;
    if (!quant_layer_ok(N, D, E, d_moe, d_sh, k, group, W)) return MOE_ERR_SHAPE;
    if (N == 0) return MOE_OK;
    for (const void *p : {x, gate_up, gate_up_scales, down, down_scales, sh_gate_up, sh_gate_up_scales,
                          sh_down, sh_down_scales, (const void *)topk_idx, (const void *)topk_w,
                          (const void *)y})
        if (!p || !aligned16(p)) return MOE_ERR_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < W.total)
        return MOE_ERR_WORKSPACE;
    DeviceInfo *dev = nullptr;
    int rc = current_device_info(&dev);
    if (rc != MOE_OK) return rc;
    if (dev->major != 10) return MOE_ERR_NO_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Profiler prof(st);

    QuantArgs a = {};
    a.N = N;
    a.E = E;
    a.k = k;
    a.G = group;
    a.direct = W.direct ? 1 : 0;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.gate_max = gate_max;
    a.up_max = up_max;
    a.wait_limit_ns = g_wait_limit_ns;
    a.never_signal = g_never_signal;
    DispatchParams dp = {};
    if (!W.direct) {
        dp.topk_idx = topk_idx;
        dp.topk_w = topk_w;
        dp.N = N;
        dp.k = k;
        dp.E = E;
        dp.nchunks = W.nchunks;
        dp.tile_rows = W.tile_rows;
        dp.chunk_hist = reinterpret_cast<int32_t *>(ws + W.chunk_hist);
        dp.counts = reinterpret_cast<int32_t *>(ws + W.counts);
        dp.tile_off = reinterpret_cast<int32_t *>(ws + W.tile_off);
        dp.meta = reinterpret_cast<int32_t *>(ws + W.meta);
        dp.pos_of = reinterpret_cast<int32_t *>(ws + W.pos_of);
        dp.perm_tok = reinterpret_cast<int32_t *>(ws + W.perm_tok);
        dp.w_perm = reinterpret_cast<float *>(ws + W.w_perm);
        if ((size_t)N * k <= DISPATCH_SMALL_IDS) {
            dispatch_small_kernel<<<1, DISPATCH_SMALL_THREADS, 0, st>>>(dp);
            if ((rc = launched(prof)) != MOE_OK) return rc;
        } else {
            dispatch_count_kernel<<<W.nchunks, DISPATCH_THREADS, 0, st>>>(dp);
            if ((rc = launch_status()) != MOE_OK) return rc;
            dispatch_scan_kernel<<<1, DISPATCH_MAXE, 0, st>>>(dp);
            if ((rc = launch_status()) != MOE_OK) return rc;
            dispatch_scatter_kernel<<<W.nchunks, DISPATCH_THREADS, 0, st>>>(dp);
            if ((rc = launched(prof)) != MOE_OK) return rc;
        }
        a.tile_off = dp.tile_off;
        a.counts = dp.counts;
        a.perm_tok = dp.perm_tok;
        a.w_perm = dp.w_perm;
    } else {
        prof.mark();
    }
    const QuantLayer w = {gate_up, gate_up_scales, down, down_scales, sh_gate_up, sh_gate_up_scales,
                          sh_down, sh_down_scales, D, d_moe, d_sh};
    // Tiles of 256 weight rows cost least per row (a row's sum stays in one warp, and the
    // tokens are laid out half as often), those of 128 are more even where there are few (us
    // for the layer, 256 / 128): D 4096, 128 experts of 1408: one token 35 / 30, 4 (about 360
    // tiles of 256 rows for 296 places) 82 / 74, 8 (715) 111 / 116, 32 219 / 239; D 6144, 256 of
    // 2048, groups of 64: 4 tokens (530) 150 / 151, 8 (1040) 244 / 246, 32 640 / 680.  The tiles
    // are estimated, as the routing is on the device.
    const size_t tt = std::max<size_t>(std::min<size_t>((size_t)N * k, E), (size_t)N * k / W.tile_rows) +
                      (N + W.tile_rows - 1) / W.tile_rows;
    const bool few = tt * ((d_moe + 127) / 128) < (size_t)dev->sms * 4;
    if (W.tile_rows == 8)
        rc = few ? quant_layer_t<4, 2, 128, 1>(w, a, x, ws, W, dev, prof, st)
                 : quant_layer_t<8, 2, 128, 1>(w, a, x, ws, W, dev, prof, st);
    else
        rc = few ? quant_layer_t<4, 2, 128, 2>(w, a, x, ws, W, dev, prof, st)
                 : quant_layer_t<8, 2, 128, 2>(w, a, x, ws, W, dev, prof, st);
    if (rc != MOE_OK) return rc;
    rc = launch_serial(quant_combine_kernel, dim3(N, (D + 4 * QC_THREADS - 1) / (4 * QC_THREADS), 1), QC_THREADS, 0, st, a,
                       (const float *)(ws + W.slot), (const float *)(ws + W.osh), (const int32_t *)dp.pos_of,
                       static_cast<__nv_bfloat16 *>(y), D);
    prof.mark();
    return rc;
}

}  // extern "C"
