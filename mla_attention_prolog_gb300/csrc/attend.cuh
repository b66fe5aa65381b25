// What the entry points of the attention and page operators share.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mla_prolog.h"
#include "prolog.cuh"

namespace mlap {

constexpr int kStatusSeqRange = MLA_STATUS_SEQ_RANGE;
constexpr int kStatusPageRange = MLA_STATUS_PAGE_RANGE;
constexpr int kStatusPoolFull = MLA_STATUS_POOL_FULL;

// api.cu: the error text of mla_prolog_last_cuda_error(), and the driver's
// cuTensorMapEncodeTiled (null where the driver has none).
int report_cuda(cudaError_t e, const char* where);
void* tensor_map_encoder();

// A softmax scale whose product with log2 e and a score keeps its meaning in FP32.
inline bool scale_ok(float scale) { return scale > 0.f && scale <= 1e30f; }

inline bool ptr_ok(const void* p, uintptr_t align) {
    return p && reinterpret_cast<uintptr_t>(p) % align == 0;
}

// The current device's SM count; MLA_ERR_DEVICE unless it is sm_103.  Asked of
// the driver once per device.
inline int current_sm103(int* sms) {
    static std::atomic<int> known[64];
    int dev = 0, major = 0, minor = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return MLA_OK;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return report_cuda(e, "device query");
    if (major != 10 || minor != 3) return MLA_ERR_DEVICE;
    if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
    return MLA_OK;
}

// Lets `kernel` use `bytes` of dynamic shared memory on the current device;
// `ready` (one bit per device) remembers for which that was done.
template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>* ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (ready->load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready->fetch_or(bit, std::memory_order_release);
    return e;
}

inline bool encode_bf16_dims(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[3],
                             const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3]) {
    auto fn = reinterpret_cast<CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                            CUtensorMapFloatOOBfill)>(tensor_map_encoder());
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// BF16 operand [outer, mid, inner] (contiguous), loaded in boxes of box_outer
// x box_mid x 64 columns with 128-byte swizzle; what lies outside reads as 0.
inline bool encode_bf16_3d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t mid, uint64_t outer,
                           uint32_t box_mid, uint32_t box_outer) {
    return encode_bf16_dims(m, base, {inner, mid, outer}, {inner * 2, inner * mid * 2}, {64, box_mid, box_outer});
}

// The whole 64-column chunks of a BF16 operand [rows, inner] as [chunk][row]
// [64]: one copy brings `count` chunks of box_rows rows, chunk after chunk.
inline bool encode_bf16_chunks(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                               uint32_t count) {
    return encode_bf16_dims(m, base, {64, rows, inner / 64}, {inner * 2, 128}, {64, box_rows, count});
}

__device__ __forceinline__ void raise_status(int32_t* status, int bits) {
    if (status && bits) atomicOr(status, bits);
}

}  // namespace mlap
