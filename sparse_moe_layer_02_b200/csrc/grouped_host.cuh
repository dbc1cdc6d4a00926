// Host side of the grouped products (moe_grouped_linear and its two gradients):
// argument checks, tensor maps, launches.  Part of moe.cu's translation unit.
#pragma once

#include "grouped.cuh"

namespace moe {
namespace {

// 3-D bf16 map over [d2, d1, d0] (d0 contiguous), boxes of b0 x b1 x 1 elements with
// 128-byte swizzle; out-of-range elements read as zero and are not written.
bool make_map3(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b0,
               uint32_t b1) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {d0, d1, d2};
    cuuint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
    cuuint32_t box[3] = {b0, b1, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same with the columns in blocks of 64: [d2, cols / 64, d1, 64], boxes of blocks x
// rows x 64 elements.  cols is a multiple of 64.
bool make_map_blocks(CUtensorMap *m, const void *base, uint64_t cols, uint64_t d1, uint64_t d2,
                     uint32_t rows, uint32_t blocks, bool batched) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {64, d1, cols / 64, d2};
    cuuint64_t strides[3] = {cols * 2, 128, cols * d1 * 2};
    cuuint32_t box[4] = {64, rows, blocks, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, batched ? 4 : 3, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch with programmatic stream serialization: the kernel may become resident while
// its predecessor ends, and waits for it (griddepcontrol.wait) before it touches memory.
template <typename... KArgs, typename... Args>
int launch_serial(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t st, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (launch_ex(cfg, kernel, args...) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_status();
}

// Clusters of n blocks of a kernel that run at once, 0 where they cannot.
template <typename... KArgs>
int clusters_at_once(void (*kernel)(KArgs...), int n, int threads, int smem, int sms) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms / n * n, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int count = 0;
    if (cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) == cudaSuccess) return count;
    cudaGetLastError();
    return 0;
}

// Launch with clusters of `split` blocks, and with programmatic serialization as above.
template <typename... KArgs, typename... Args>
int launch_clusters(void (*kernel)(KArgs...), int split, int grid, int threads, int smem, cudaStream_t st,
                    Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (launch_ex(cfg, kernel, args...) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_status();
}

// kb: a tile's k-blocks (wgrad: on average).
template <int MODE>
int launch_grouped(const CUtensorMap &mA, const CUtensorMap &mB, const CUtensorMap &mOut,
                   GroupedArgs a, size_t tiles, int kb, DeviceInfo *info, cudaStream_t st) {
    using C = GrpCfg<MODE>;
    static int clusters[kMaxDevices][4] = {}; // of 1, 2, 4, 8 blocks at once; found once per device
    const int dev = current_device_index();
    if (dev < 0) return MOE_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!clusters[dev][0]) {
            for (auto kernel : {grouped_product_kernel<MODE, false>, grouped_product_kernel<MODE, true>})
                if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
                    cudaSuccess)
                    return MOE_ERR_CUDA;
            for (int i = 1; i < 4; ++i)
                clusters[dev][i] = clusters_at_once(grouped_product_kernel<MODE, true>, 1 << i, C::THREADS, C::SMEM,
                                                    info->sms);
            clusters[dev][0] = info->sms;
        }
    }
    // As many blocks share a tile as leave each tile a cluster of its own, at once, and each
    // block 8 k-blocks: joining costs 2 to 3 us (us, unshared / shared): forward, 1 row,
    // 1024 x 6144 37.5 / 13.9, 64 rows, 6144 x 6144 38.8 / 19.0; wgrad, 65536 rows, 512 x 512
    // 454 / 72.  With shares of 4: forward, 4096 rows, 4 x 512 x 512 9.1 / 12.0.
    a.split = 1;
    for (int i = 1; i < 4; ++i)
        if (tiles <= (size_t)clusters[dev][i] && kb >= 8 << i) a.split = 1 << i;
    if (a.split > 1)
        return launch_clusters(grouped_product_kernel<MODE, true>, a.split, (int)tiles * a.split, C::THREADS, C::SMEM,
                               st, mA, mB, mOut, a);
    return launch_serial(grouped_product_kernel<MODE, false>, dim3((unsigned)std::min<size_t>(tiles, info->sms), 1, 1),
                         C::THREADS, C::SMEM, st, mA, mB, mOut, a);
}

// One product.  A and B: forward x, W; dgrad dy, W; wgrad dy, x.
template <int MODE>
int grouped_impl(const void *A, const void *B, const int32_t *offsets, int rows, int E, int M, int K,
                 int dtype, void *out, int zero_rest, void *stream) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
    const int vec = dtype == MOE_BF16 ? 8 : 4; // 16-byte rows
    if (rows < 0 || E <= 0 || E > GRP_MAXE || M <= 0 || K <= 0 || M % vec || K % vec)
        return MOE_ERR_SHAPE;
    // tile numbers are 32-bit: bound their count at the smallest tile (32 x 32)
    const size_t most = INT32_MAX / 2;
    const size_t ncols = MODE == GRP_FORWARD ? M : K;
    if (M > (1 << 24) || K > (1 << 24) || rows > INT32_MAX - 256 ||
        ((size_t)rows / 32 + E) * (ncols / 32 + 1) > most ||
        (size_t)E * ((size_t)M / 32 + 1) * ((size_t)K / 32 + 1) > most)
        return MOE_ERR_SHAPE;
    if (rows == 0 && MODE != GRP_WGRAD) return MOE_OK;
    if (!out || !offsets || (rows > 0 && (!A || !B))) return MOE_ERR_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(offsets) & 3u))
        return MOE_ERR_ARG;
    DeviceInfo *dev = nullptr;
    int rc = current_device_info(&dev);
    if (rc != MOE_OK) return rc;
    if (dev->major != 10) return MOE_ERR_NO_DEVICE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) { // no row has a gradient
        const size_t es = dtype == MOE_BF16 ? 2 : 4;
        return cudaMemsetAsync(out, 0, (size_t)E * M * K * es, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    GroupedArgs a = {};
    a.offsets = offsets;
    a.rows = rows;
    a.E = E;
    a.M = M;
    a.K = K;
    a.red = MODE == GRP_FORWARD ? K : M;
    a.ncols = (int)ncols;
    a.out = out;
    a.zero_rest = zero_rest ? 1 : 0;
    a.wait_limit_ns = g_wait_limit_ns;
    a.never_signal = g_never_signal;

    if (dtype == MOE_F32) {
        // 64 x 64 tiles need less shared memory traffic, 32 x 32 tiles spread few rows over
        // the SMs and fill better where experts have few (us, 32 / 64): forward, 256 rows,
        // 16 x 256 x 256 8.9 / 18.1; 1024 rows, 8 x 512 x 512 (128 tiles of 64) 23 / 36; 2000
        // rows, 8 x 1024 x 512 (500) 77 / 61; 4000 rows, 8 x 1024 x 1024 290 / 231; 75 rows an
        // expert: 1500 rows, 20 x 512 x 900 71 / 104, its dgrad 72 / 92; 128 an expert: 2048
        // rows, 16 x 768 x 768 96 / 88.  wgrad, whose tiles do not depend on the rows:
        // 4 x 256 x 256 (64 tiles) 3.4 / 3.6, 16 x 256 x 256 (256) 5.7 / 4.2,
        // 16 x 512 x 512 25 / 16.
        bool small;
        if (MODE == GRP_WGRAD)
            small = (size_t)E * ((M + 63) / 64) * ((K + 63) / 64) * 2 < (size_t)dev->sms;
        else
            small = (size_t)rows * ncols / (64 * 64) * 2 < (size_t)dev->sms * 3 || rows < 96 * E;
        const int T = small ? 32 : 64;
        a.nb = (a.ncols + T - 1) / T;
        a.mb = (M + T - 1) / T;
        const size_t tiles = MODE == GRP_WGRAD ? (size_t)E * a.nb * a.mb
                                               : ((size_t)rows / T + std::min(rows, E)) * a.nb;
        const int grid = (int)std::min<size_t>(std::max<size_t>(tiles, 1), (size_t)dev->sms * 8);
        const float *fa = static_cast<const float *>(A), *fb = static_cast<const float *>(B);
        if (small) return launch_serial(grouped_f32_kernel<MODE, 32>, dim3(grid, 1, 1), GrpF32<32>::THREADS, 0, st, fa, fb, a);
        return launch_serial(grouped_f32_kernel<MODE, 64>, dim3(grid, 1, 1), GrpF32<64>::THREADS, 0, st, fa, fb, a);
    }

    a.nb = (a.ncols + GRP_BN - 1) / GRP_BN;
    a.mb = (M + GRP_BM - 1) / GRP_BM;
    CUtensorMap mA, mB, mOut;
    bool ok;
    if (MODE == GRP_FORWARD)
        ok = make_map(&mA, A, K, rows, K, GRP_BM) && make_map3(&mB, B, K, M, E, 64, GRP_BN) &&
             make_map(&mOut, out, M, rows, M, 32);
    else if (MODE == GRP_DGRAD) {
        a.wide = K % 64 == 0; // (dgrad 16384 rows, 32 x 4096 x 6144: 744 us, 749 without; wgrad 915, 923)
        ok = make_map(&mA, A, M, rows, M, GRP_BM) && make_map(&mOut, out, K, rows, K, 32) &&
             (a.wide ? make_map_blocks(&mB, B, K, M, E, 64, 4, true) : make_map3(&mB, B, K, M, E, 64, 64));
    } else {
        a.wide = K % 64 == 0 && M % 64 == 0;
        ok = make_map3(&mOut, out, K, M, E, 64, 32) &&
             (a.wide ? make_map_blocks(&mA, A, M, rows, 1, 64, 2, false) &&
                           make_map_blocks(&mB, B, K, rows, 1, 64, 4, false)
                     : make_map(&mA, A, M, rows, M, 64) && make_map(&mB, B, K, rows, K, 64));
    }
    if (!ok) return MOE_ERR_CUDA;
    const size_t tiles = MODE == GRP_WGRAD ? (size_t)E * a.nb * a.mb
                                           : ((size_t)rows / GRP_BM + std::min(rows, E)) * a.nb;
    const int kb = (int)((MODE == GRP_WGRAD ? (size_t)rows / E : (size_t)a.red) / GRP_BK);
    return launch_grouped<MODE>(mA, mB, mOut, a, tiles, kb, dev, st);
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_grouped_linear(const void *x, const void *W, const int32_t *offsets, int rows, int E, int M,
                       int K, int dtype, void *y, int zero_rest, void *stream) {
    return moe::grouped_impl<moe::GRP_FORWARD>(x, W, offsets, rows, E, M, K, dtype, y, zero_rest, stream);
}

int moe_grouped_linear_dgrad(const void *dy, const void *W, const int32_t *offsets, int rows, int E,
                             int M, int K, int dtype, void *dx, int zero_rest, void *stream) {
    return moe::grouped_impl<moe::GRP_DGRAD>(dy, W, offsets, rows, E, M, K, dtype, dx, zero_rest, stream);
}

int moe_grouped_linear_wgrad(const void *dy, const void *x, const int32_t *offsets, int rows, int E,
                             int M, int K, int dtype, void *dW, void *stream) {
    return moe::grouped_impl<moe::GRP_WGRAD>(dy, x, offsets, rows, E, M, K, dtype, dW, 0, stream);
}

}  // extern "C"
