// Host side of alspec_linear: argument checks, tensor maps, the split and
// the launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "alspec.h"
#include "host.h"
#include "linear_kernels.cuh"

namespace alspec {
namespace {

// A 2-D bf16 matrix [rows][k] with rows `stride` elements apart; boxes of 64
// columns x `box` rows with 128-byte swizzle.
alspec_status encode_matrix(CUtensorMap* map, const void* base, int k, int rows, int64_t stride,
                            int box) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const alspec_status st = tiled_map_encoder(&encode);
    if (st != ALSPEC_OK) return st;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {kLinK, (cuuint32_t)box};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r =
        encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
               boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ALSPEC_OK : ALSPEC_ERR_INVALID_ARG;
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
    // Batch rows per tile: equal shares of at most 256, in steps of 16 (the
    // step of a 128-row tcgen05 shape).
    p.row_tiles = (int)(((int64_t)rows + kLinMaxN - 1) / kLinMaxN);
    p.nt = (int)((((int64_t)rows + p.row_tiles - 1) / p.row_tiles + 15) / 16 * 16);
    p.row_tiles = (rows - 1) / p.nt + 1;
    const int64_t tiles = ((int64_t)n + kLinM - 1) / kLinM * p.row_tiles;
    p.kblocks = (k - 1) / kLinK + 1;
    // K is split over a cluster while that finds idle SMs, at least four
    // 64-column slices a CTA.
    const int sms = sm_count_for_plan();
    p.split = (int)std::max<int64_t>(
        1, std::min<int64_t>({8, sms / std::max<int64_t>(tiles, 1), p.kblocks / 4}));
    if (tiles * p.split > 0x7fffffff || n > 0x7fffffff - kLinM) return ALSPEC_ERR_UNSUPPORTED;
    const int stage = (kLinM + p.nt) * 128;
    p.stages = std::min({kLinMaxStages, kLinRing / stage,
                         std::max(2, (p.kblocks + p.split - 1) / p.split)});
    p.tmem_cols = 32;
    while (p.tmem_cols < p.nt) p.tmem_cols *= 2;
    const int smem = std::max({p.stages * stage, p.nt * kLinM * 4, kLinMinSmem}) + 1024;
    alspec_status st = encode_matrix(&p.tw, w, k, n, k, kLinM);
    if (st != ALSPEC_OK) return st;
    if ((st = encode_matrix(&p.tx, x, k, rows, x_stride ? x_stride : k, p.nt)) != ALSPEC_OK)
        return st;
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.residual = residual;
    p.y = y;
    p.rows = rows;
    p.n = n;
    p.out_bf16 = out_dtype == ALSPEC_BF16;
    p.act = activation;
    p.err = err;
    p.timeout_ns = 2000000000ull;
    const void* fn = reinterpret_cast<const void*>(linear_kernel);
    if ((st = smem_attr_once(fn, kLinRing + 1024)) != ALSPEC_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2] = {programmatic_launch()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return ok(cudaLaunchKernelEx(&cfg, linear_kernel, p)) ? ALSPEC_OK : ALSPEC_ERR_CUDA;
}
