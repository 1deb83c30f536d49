// abi_util.cuh -- argument checks and error returns shared by the entry points
// of gated_scan.cu and layer_norm.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
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
    cudaGetLastError();  // reported here: the caller's next check of the runtime is not to find it again
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
// A kernel's attributes are set once per device; `done` holds a bit per device.
template <class Kern>
bool prepare_kernel(Kern kern, size_t smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

inline int sm_count() {
    static thread_local int dev_of = -1, sms = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev != dev_of) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        dev_of = dev;
    }
    return sms;
}

// A launch that may begin while the stream's previous kernel is still running, if
// that kernel allows it (follow_previous): the blocks wait for its end, and for its memory to be
// visible, before they touch global memory, so only the launch itself overlaps.
// `ranks` blocks form a cluster.
template <class... P, class... A>
pararnn_status launch(const char* who, void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int ranks,
                      const A&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? PARARNN_OK : cuda_fail(who, "kernel launch failed");
}

}  // namespace abi

// Allows the stream's next kernel to be launched, and waits for the previous one and its
// memory; before the first access to global memory.
__device__ __forceinline__ void follow_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// rounding of a result to the type of the array it goes to
template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace pararnn
