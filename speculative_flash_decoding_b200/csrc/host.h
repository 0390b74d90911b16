// Host helpers that the library's translation units share; defined in
// alspec.cu.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "alspec.h"

namespace alspec {

constexpr int kMaxDevices = 64;

// True for cudaSuccess; any other value is kept for alspec_last_cuda_error.
bool ok(cudaError_t e);

// SMs of the current device (148 where there is none).
int sm_count_for_plan();

// cuTensorMapEncodeTiled, looked up in the driver at its first use.
alspec_status tiled_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

// Lets `kernel` use `bytes` of dynamic shared memory on the current device
// (set once per device, until alspec_shutdown).
alspec_status smem_attr_once(const void* kernel, int bytes);

// Launch attribute of a kernel that may be placed while the one ahead on the
// stream still runs; it waits (griddepcontrol.wait) before it touches
// anything that one reads or writes.
inline cudaLaunchAttribute programmatic_launch() {
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace alspec
