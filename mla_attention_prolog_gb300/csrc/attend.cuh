// What the entry points of the attention and page operators share.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mla_prolog.h"
#include "prolog.cuh"

namespace mlap {

// api.cu: the error text of mla_prolog_last_cuda_error(), and the driver's
// cuTensorMapEncodeTiled (null where the driver has none).
int report_cuda(cudaError_t e, const char* where);
void* tensor_map_encoder();

inline bool ptr_ok(const void* p, uintptr_t align) {
    return p && reinterpret_cast<uintptr_t>(p) % align == 0;
}

// The current device and its SM count; MLA_ERR_DEVICE unless it is sm_103.
// Two attribute queries (no cudaGetDeviceProperties): cheap on every call.
inline int current_sm103(int* sms) {
    int dev = 0, major = 0, minor = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return report_cuda(e, "device query");
    return major == 10 && minor == 3 ? MLA_OK : MLA_ERR_DEVICE;
}

__device__ __forceinline__ void raise_status(int32_t* status, int bits) {
    if (status && bits) atomicOr(status, bits);
}

}  // namespace mlap
