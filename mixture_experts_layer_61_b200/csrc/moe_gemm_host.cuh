// moe_gemm_host.cuh -- host side shared by the tensor-core kernels' launchers:
// TMA tensor maps, persistent grid sizes and the grouped GEMM's launch.
#pragma once

#include <atomic>
#include <mutex>

#include "moe_gemm.cuh"
#include "moe_internal.h"

namespace moe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        cudaGetLastError();
    });
    return fn;
}

// [rows, kdim] row-major, box = box_rows x row_bytes (128 or 64) with the
// swizzle of that width, out-of-range elements read as zero.
inline bool make_map(CUtensorMap* m, CUtensorMapDataType dt, int elt_bytes, const void* base, long long rows, int kdim,
              int box_rows, int row_bytes = 128) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(kdim), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(kdim) * elt_bytes};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(row_bytes / elt_bytes), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// [n, rows, cols] row-major matrices, box = box_rows x 128 bytes of one of
// them with the 128-byte swizzle, out-of-range elements read as zero (of a
// store: not written).
inline bool make_map3(CUtensorMap* m, CUtensorMapDataType dt, int elt_bytes, const void* base, int n, long long rows,
                      int cols, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(n)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * elt_bytes,
                             static_cast<cuuint64_t>(cols) * elt_bytes * static_cast<cuuint64_t>(rows)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elt_bytes), static_cast<cuuint32_t>(box_rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [n, rows, cols] matrices of 16-bit elements, cols a multiple of 64, as
// (64 columns, rows, cols / 64, n): one box takes `chunks` 64-column blocks of
// box_rows rows, laid one after the other with the 128-byte swizzle.  (Rows
// whose length is no multiple of 64 have no such view inside the tensor.)
inline bool make_map_cols(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int n, long long rows, int cols,
                          int box_rows, int chunks) {
    EncodeTiledFn fn = encode_fn();
    if (!fn || cols % 64) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(cols) * 2;
    cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64),
                          static_cast<cuuint64_t>(n)};
    cuuint64_t strides[3] = {row, 128, row * static_cast<cuuint64_t>(rows)};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(chunks), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, dt, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of `kern` (a persistent kernel on clusters of kCta, one block per SM)
// that can be resident at once on the current device, with its shared-memory
// limit raised; cached per device in `cache` (0: not asked yet).
constexpr int kMaxCachedDevices = 64;
template <typename Kern>
int resident_blocks(Kern kern, int smem_bytes, int threads, int cta, const DeviceInfo& d, std::atomic<int>* cache,
                    int* blocks) {
    std::atomic<int>& c = cache[d.device];
    *blocks = c.load(std::memory_order_acquire);
    if (*blocks > 0) return 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) != cudaSuccess) {
        cudaGetLastError();
        return -3;
    }
    int n = d.num_sms;
    if (cta > 1) {
        // pairs must sit in one GPC: size the persistent grid by the clusters that fit
        cudaLaunchConfig_t oc = {};
        oc.gridDim = dim3(d.num_sms);
        oc.blockDim = dim3(threads);
        oc.dynamicSmemBytes = smem_bytes;
        cudaLaunchAttribute ca;
        ca.id = cudaLaunchAttributeClusterDimension;
        ca.val.clusterDim.x = cta;
        ca.val.clusterDim.y = 1;
        ca.val.clusterDim.z = 1;
        oc.attrs = &ca;
        oc.numAttrs = 1;
        int nclusters = 0;
        if (cudaOccupancyMaxActiveClusters(&nclusters, kern, &oc) != cudaSuccess || nclusters <= 0) {
            cudaGetLastError();
            return -3;
        }
        if (nclusters * cta < n) n = nclusters * cta;
    }
    c.store(n, std::memory_order_release);
    *blocks = n;
    return 0;
}

// kWMn: the weights are [n_groups, kdim, n_out], the features contiguous
template <typename T, typename OutT, int kEpi, int kMaxN, int kCta = 1, bool kWMn = false>
int launch_variant(const GemmLaunch& L, const GemmCtl& ctl, int num_sms, cudaStream_t stream) {
    constexpr bool kTrain = kWMn || kEpi == kEpiSwiGLUTrain;
    using C = GemmCfg<T, kEpi, kMaxN, kCta, kTrain>;
    auto kern = moe_gemm_kernel<T, OutT, kEpi, kMaxN, kCta, kWMn>;
    if (kCta == 2 && (num_sms & 1)) return -1;
    static std::atomic<int> cache[kMaxCachedDevices];  // per instantiation
    int grid_blocks = 0;
    DeviceInfo d;
    int rc = current_device(&d);
    if (rc != 0) return rc;
    if ((rc = resident_blocks(kern, C::kSmemBytes, kGemmThreads, kCta, d, cache, &grid_blocks)) != 0) return rc;
    CUtensorMap tm_w, tm_x, tm_x64, tm_xbig;
    constexpr int rb = C::kRowBytes;
    const bool joined = kWMn && kCta == 2 && L.n_out % 64 == 0;
    if (joined ? !make_map_cols(&tm_w, Elt<T>::kTma, L.w, L.n_groups, L.kdim, L.n_out, C::kStageK, 2 * C::kNW)
        : kWMn ? !make_map3(&tm_w, Elt<T>::kTma, Elt<T>::kBytes, L.w, L.n_groups, L.kdim, L.n_out, C::kStageK)
             : !make_map(&tm_w, Elt<T>::kTma, Elt<T>::kBytes, L.w, L.w_rows, L.kdim, 128, rb))
        return -3;
    const bool x_joined = C::kChunks > 1 && L.kdim % C::kBK == 0;
    auto x_map = [&](CUtensorMap* m, int rows) {
        if (x_joined) return make_map_cols(m, Elt<T>::kTma, L.x, 1, L.x_rows, L.kdim, rows, C::kChunks);
        return make_map(m, Elt<T>::kTma, Elt<T>::kBytes, L.x, L.x_rows, L.kdim, rows, rb);
    };
    if (!x_map(&tm_x, C::kXBoxRows) || !x_map(&tm_x64, C::kXBoxMid) || !x_map(&tm_xbig, kMaxN / kCta)) return -3;
    GemmParams p;
    p.seg_offsets = L.seg_offsets;
    p.n_groups = L.n_groups;
    p.seg_rows = L.seg_rows;
    p.n_out = L.n_out;
    p.kdim = L.kdim;
    p.w_group_stride = L.w_group_stride;
    p.up_offset = L.up_offset;
    p.out = L.out;
    p.out_ld = L.out_ld;
    p.pre = L.pre;
    p.w_joined = joined ? 1 : 0;
    p.x_joined = x_joined ? 1 : 0;
    p.counters = ctl.counters;
    p.partials = ctl.partials;
    p.status = ctl.status;
    p.wait_limit_ns = wait_limit_ns();
    p.withhold_first_load = take_withhold_flag();
    // fewest k-iterations of a slice; training: 16, as adding up a slice's partial
    // sums takes longer than fewer (8 experts of 512 x 512, 192 tokens, gate/up
    // gradient: 13.5 us, in slices of 4 26.3 us; 64 of 1024 x 512, 64 tokens:
    // 14.4 us, 20.7 us; only a single token gains from slices of 4: 8 of 2048 x
    // 1024, gate/up with pre-activations: 15.8 us, 14.4 us)
    p.sk_min_units = (kTrain ? 16 : 4) / C::kChunks;
    p.max_split = L.max_split > 0 ? L.max_split : 4;
    p.split_tail = split_tail_mode();
    int grid = grid_blocks;
    if (L.sms > 0 && L.sms < grid) grid = L.sms >= 2 * kCta ? L.sms - L.sms % kCta : kCta;
    cudaError_t e = launch_kernel_cluster(kern, dim3(grid), dim3(kGemmThreads), C::kSmemBytes, stream, kCta,
                                          tm_w, tm_x, tm_x64, tm_xbig, p);
    count_launch();
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? 0 : -3;
}

}  // namespace moe
