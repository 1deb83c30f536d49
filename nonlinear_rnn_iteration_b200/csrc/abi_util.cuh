// abi_util.cuh -- argument checks and error returns shared by the entry points
// of gated_scan.cu and layer_norm.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "common.cuh"
#include "pararnn_b200.h"

namespace pararnn {
void set_last_error(const char* msg);   // pararnn_abi.cu
bool pointer_on_device(const void* p);  // pararnn_abi.cu

namespace abi {

inline pararnn_status fail(const char* who, const char* msg) {
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", who, msg);
    set_last_error(buf);
    return PARARNN_EINVAL;
}
inline pararnn_status cuda_fail(const char* who, const char* what) {
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", who, what);
    set_last_error(buf);
    return PARARNN_ECUDA;
}
inline bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// a pointer that is null though required, misaligned or not reachable by the GPU
inline bool bad_pointer(const void* p, size_t align, bool required) {
    if (!p) return required;
    return misaligned(p, align) || !pointer_on_device(p);
}
inline bool bad_dtype(pararnn_dtype t) { return t != PARARNN_F32 && t != PARARNN_BF16; }

// Clears the header of a workspace, so that the call's status can be read
// from it.  Where the workspace is optional a null one records nothing.
inline pararnn_status open_status(const char* who, void* workspace, size_t ws_bytes, size_t need, bool required,
                                  cudaStream_t st) {
    if (!workspace && !required) return PARARNN_OK;
    if (!workspace || ws_bytes < need || misaligned(workspace, 16) || !pointer_on_device(workspace))
        return fail(who, "workspace missing, too small, not 16-byte aligned or not device memory");
    if (cudaMemsetAsync(workspace, 0, kHeaderBytes, st) != cudaSuccess) return cuda_fail(who, "workspace reset failed");
    return PARARNN_OK;
}
inline pararnn_status launched(const char* who) {
    return cudaGetLastError() == cudaSuccess ? PARARNN_OK : cuda_fail(who, "kernel launch failed");
}

}  // namespace abi

// rounding of a result to the type of the array it goes to
template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace pararnn
