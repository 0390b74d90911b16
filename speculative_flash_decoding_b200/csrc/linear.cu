// Host side of alspec_linear: argument checks, tensor maps, the split and
// the launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "alspec.h"
#include "host.h"
#include "linear_kernels.cuh"
#include "linear_plan.h"

namespace alspec {
namespace {

// Views of a bf16 matrix [rows][k] with rows `stride` elements apart, boxes
// of `box` rows with 128-byte swizzle: `whole` as 64-column blocks, `group`
// of them in a box, and `end` as plain columns.
alspec_status encode_matrix(CUtensorMap* whole, CUtensorMap* end, const void* base, int k, int rows,
                            int64_t stride, int box, int group) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const alspec_status st = tiled_map_encoder(&encode);
    if (st != ALSPEC_OK) return st;
    const cuuint32_t estr[3] = {1, 1, 1};
    for (int w = 0; w < 2; ++w) {
        CUtensorMap* map = w ? whole : end;
        if (w && k < kLinK) continue;
        const cuuint64_t dims[3] = {(cuuint64_t)(w ? kLinK : k), (cuuint64_t)rows,
                                    (cuuint64_t)(k / kLinK)};
        const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, kLinK * 2};
        const cuuint32_t boxes[3] = {kLinK, (cuuint32_t)box, (cuuint32_t)group};
        const CUresult r =
            encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w ? 3 : 2, const_cast<void*>(base), dims,
                   strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return ALSPEC_ERR_INVALID_ARG;
    }
    if (k < kLinK) *whole = *end;  // no whole block: never used
    return ALSPEC_OK;
}

// Clusters of the kernel that the current device holds at once (asked once).
LinClusters g_clusters[kMaxDevices] = {};
bool g_clusters_known[kMaxDevices] = {};
std::mutex g_clusters_mutex;

bool resident_clusters(LinClusters* out) {
    int dev = 0;
    if (!ok(cudaGetDevice(&dev)) || dev < 0 || dev >= kMaxDevices) return false;
    if (smem_attr_once(reinterpret_cast<const void*>(linear_kernel<false>), kLinSmem) != ALSPEC_OK)
        return false;
    std::lock_guard<std::mutex> lock(g_clusters_mutex);
    LinClusters& fit = g_clusters[dev];
    for (int c = 1; c <= kLinMaxSplit && !g_clusters_known[dev]; ++c) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)c);
        cfg.blockDim = dim3(kLinThreads);
        cfg.dynamicSmemBytes = kLinSmem;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = c;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        // A size that does not fit is no error: it is not chosen.
        if (cudaOccupancyMaxActiveClusters(&fit.n[c], linear_kernel<false>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            fit.n[c] = 0;
        }
    }
    g_clusters_known[dev] = true;
    *out = fit;
    return true;
}

}  // namespace
}  // namespace alspec

using namespace alspec;

extern "C" alspec_status alspec_linear(const void* x, int64_t x_stride, const void* w,
                                       const void* bias, const void* residual, void* y,
                                       int out_dtype, int activation, int rows, int n, int k,
                                       uint32_t* err, void* stream) {
    if (rows < 0 || n < 1 || k < 8 || k % 8 != 0) return ALSPEC_ERR_INVALID_ARG;
    if (out_dtype != ALSPEC_F32 && out_dtype != ALSPEC_BF16) return ALSPEC_ERR_INVALID_ARG;
    if (activation < ALSPEC_ACT_NONE || activation > ALSPEC_ACT_SILU)
        return ALSPEC_ERR_INVALID_ARG;
    const uintptr_t ymask = out_dtype == ALSPEC_F32 ? 3u : 1u;
    if (x_stride != 0 && (x_stride < k || x_stride % 8 != 0 || x_stride >= ((int64_t)1 << 39)))
        return ALSPEC_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(bias) & 1u) || (reinterpret_cast<uintptr_t>(residual) & ymask) ||
        (reinterpret_cast<uintptr_t>(y) & ymask) || (reinterpret_cast<uintptr_t>(err) & 3u))
        return ALSPEC_ERR_INVALID_ARG;
    if (rows == 0) return ALSPEC_OK;
    if (!x || !w || !y || !aligned16(x) || !aligned16(w)) return ALSPEC_ERR_INVALID_ARG;

    LinearParams p{};
    // Batch rows per tile: equal shares of at most 256 (fp32 outputs: 128, for
    // room in TMEM, see below; 200 x 8192 x 8192 takes 44.4 us with them and 33.1
    // with bf16 outputs), in steps of 16 (the step of a 128-row tcgen05 shape).
    const int most = out_dtype == ALSPEC_F32 ? kLinMaxN / 2 : kLinMaxN;
    p.row_tiles = (int)(((int64_t)rows + most - 1) / most);
    p.nt = (int)((((int64_t)rows + p.row_tiles - 1) / p.row_tiles + 15) / 16 * 16);
    p.row_tiles = (rows - 1) / p.nt + 1;
    LinClusters fit{};
    if (!resident_clusters(&fit)) return ALSPEC_ERR_CUDA;
    const bool pair = lin_pairs(fit, p.nt, n);
    if (pair) {
        p.nt = (p.nt + 31) / 32 * 32;
        p.row_tiles = (rows - 1) / p.nt + 1;
    }
    const int ctas = pair ? 2 : 1;
    const int64_t tiles = ((int64_t)n + ctas * kLinM - 1) / (ctas * kLinM) * p.row_tiles;
    p.kblocks = (k - 1) / kLinK + 1;
    p.whole = k / kLinK;
    p.split = lin_split(fit, tiles, p.kblocks, ctas);
    if (tiles * p.split * ctas > 0x7fffffff || n > 0x7fffffff - kLinM) return ALSPEC_ERR_UNSUPPORTED;
    // Blocks of a stage: four (512 consecutive bytes of a row of W) where the
    // ring holds two such stages, else two.  DRAM wants neighbouring columns
    // asked for together: one block a stage, a ring of 200 KB, took 35.1 us
    // for 16 x 8192 x 8192, two 26.4, four 26.9; for 33 x 4096 x 6144 two 16.0,
    // four 15.0.
    const int rows_tile = std::min(p.nt, rows);
    p.push = p.nt <= kLinPush;
    p.slice = (rows_tile + p.split - 1) / p.split;
    const int exchange = p.push ? p.split * p.slice * kLinM * 4 : 0;
    const int ring = kLinSmem - 1024 - exchange;
    const int block = (kLinM + p.nt / ctas) * 128;
    p.group = block * 8 <= ring ? 4 : 2;
    const int stage = block * p.group;
    const int fills = ((p.kblocks + p.split - 1) / p.split + p.group - 1) / p.group;
    p.stages = std::min({kLinMaxStages, ring / stage, std::max(2, fills)});
    // An MMA's sum may lose 2^-23 of its running value at every step: for fp32
    // outputs the blocks go round several accumulators, as many as TMEM holds,
    // up to eight (16 x 8192 x 8192: 4.4e-6 of the result off with one, 1.0e-6
    // with four; bf16 outputs round at 4e-3).
    p.sum_cols = 32;
    while (p.sum_cols < p.nt) p.sum_cols *= 2;
    p.sums = out_dtype == ALSPEC_F32 ? std::min(8, 512 / p.sum_cols) : 1;
    p.tmem_cols = p.sum_cols * p.sums;
    const int smem =
        std::max({p.stages * stage + exchange, p.push ? 0 : p.nt * kLinM * 4, kLinMinSmem}) + 1024;
    alspec_status st = encode_matrix(&p.tw, &p.tw_end, w, k, n, k, kLinM, p.group);
    if (st != ALSPEC_OK) return st;
    if ((st = encode_matrix(&p.tx, &p.tx_end, x, k, rows, x_stride ? x_stride : k,
                            p.nt / ctas, p.group)) != ALSPEC_OK)
        return st;
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.residual = residual;
    p.y = y;
    p.rows = rows;
    p.n = n;
    p.out_bf16 = out_dtype == ALSPEC_BF16;
    p.act = activation;
    const uintptr_t quad = out_dtype == ALSPEC_F32 ? 15u : 7u;
    p.vec = n % 4 == 0 && !(reinterpret_cast<uintptr_t>(y) & quad) &&
            !(reinterpret_cast<uintptr_t>(residual) & quad);
    p.err = err;
    p.timeout_ns = 2000000000ull;
    void (*const fn)(LinearParams) = pair ? linear_kernel<true> : linear_kernel<false>;
    if ((st = smem_attr_once(reinterpret_cast<const void*>(fn), kLinSmem)) != ALSPEC_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * p.split * ctas));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2] = {programmatic_launch()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split * ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return ok(cudaLaunchKernelEx(&cfg, fn, p)) ? ALSPEC_OK : ALSPEC_ERR_CUDA;
}
