// What the library's kernels share: limits, device error bits, the fixed
// words at the head of a workspace, and small device functions.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace alspec {

constexpr int kSmemLimit = 227 * 1024;

constexpr unsigned kErrSeqLen = 1u;   // ALSPEC_DEVERR_SEQ_LEN
constexpr unsigned kErrTimeout = 2u;  // ALSPEC_DEVERR_TIMEOUT
constexpr unsigned kErrBounds = 4u;   // ALSPEC_DEVERR_BOUNDS (debug build)
constexpr unsigned kErrPage = 8u;     // ALSPEC_DEVERR_PAGE

// Words at the head of a workspace: the decode queue and its exits, and the
// error word that alspec_get_device_error reads.
constexpr int kCtrQueue = 0;
constexpr int kCtrDone = 1;
constexpr int kCtrError = 2;
constexpr int kCtrFixed = 4;

// Weight of a partial with max m against the merged max M: exactly 1 when
// m == M, so merging one partial with empty ones reproduces it bit for bit.
__device__ __forceinline__ float merge_weight(float m, float M) {
    return m == M ? 1.f : exp2f(m - M);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace alspec
