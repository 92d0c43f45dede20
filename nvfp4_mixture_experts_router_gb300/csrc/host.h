// Host helpers shared by the entry points of libmoe_nvfp4.so.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_nvfp4.h"

namespace moe {

// Prepares the current device on its first call (kernel attributes, tensor-
// map encoder) and returns its number of SMs; MOE_ERR_UNSUPPORTED on a device
// this binary carries no code for.
moe_status device_state(int* sms, int* device = nullptr);

// cuTensorMapEncodeTiled (after a successful device_state).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace moe
