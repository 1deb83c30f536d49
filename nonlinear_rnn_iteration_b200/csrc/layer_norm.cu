// layer_norm.cu -- layer normalisation of (M, P, N) rows, forward and
// backward, with a scale and a shift for each of the P gates or heads.
//
//   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps), y = xh w + b
//   with d = dy w:  dx = rstd (d - mean(d) - xh mean(d xh)),
//   dw = sum over M of dy xh,  db = sum over M of dy
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "abi_util.cuh"
#include "common.cuh"
#include "pararnn_b200.h"

namespace pararnn {
namespace ln {

typedef __nv_bfloat16 bf16;
constexpr int kThreads = 128;
constexpr int kSplits = 64;  // row ranges whose column sums are formed apart

struct Params {
    const void* x;
    const float* w;
    const float* b;
    void* y;
    float* mean;
    float* rstd;
    unsigned* status;
    int64_t M, P, N;
    float eps;
};
struct BwdParams {
    const void* x;
    const float* w;
    const float* mean;
    const float* rstd;
    const void* dy;
    void* dx;
    float* part;  // [kSplits][2][P * N]
    unsigned* status;
    int64_t M, P, N;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// one warp per row
template <typename T>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Params pr) {
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= pr.M * pr.P) return;
    const T* x = static_cast<const T*>(pr.x) + row * pr.N;
    T* y = static_cast<T*>(pr.y) + row * pr.N;
    const int64_t at = (row % pr.P) * pr.N;
    float s = 0.0f;
    for (int64_t j = lane; j < pr.N; j += 32) s += PxTraits<T>::cvt(x[j]);
    const float mean = warp_sum(s) / (float)pr.N;
    s = 0.0f;
    for (int64_t j = lane; j < pr.N; j += 32) {
        const float c = PxTraits<T>::cvt(x[j]) - mean;
        s = __fmaf_rn(c, c, s);
    }
    const float rstd = 1.0f / sqrtf(warp_sum(s) / (float)pr.N + pr.eps);
    bool bad = false;
    for (int64_t j = lane; j < pr.N; j += 32) {
        const float xh = (PxTraits<T>::cvt(x[j]) - mean) * rstd;
        const float v = __fmaf_rn(xh, pr.w ? pr.w[at + j] : 1.0f, pr.b ? pr.b[at + j] : 0.0f);
        y[j] = to_out<T>(v);
        bad |= !isfinite(v);
    }
    if (lane == 0 && pr.mean) pr.mean[row] = mean;
    if (lane == 0 && pr.rstd) pr.rstd[row] = rstd;
    if (bad && pr.status) atomicOr(pr.status, kStatusNonFinite);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dx_kernel(const BwdParams pr) {
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= pr.M * pr.P) return;
    const T* x = static_cast<const T*>(pr.x) + row * pr.N;
    const T* dy = static_cast<const T*>(pr.dy) + row * pr.N;
    T* dx = static_cast<T*>(pr.dx) + row * pr.N;
    const int64_t at = (row % pr.P) * pr.N;
    const float mean = pr.mean[row], rstd = pr.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t j = lane; j < pr.N; j += 32) {
        const float xh = (PxTraits<T>::cvt(x[j]) - mean) * rstd;
        const float d = PxTraits<T>::cvt(dy[j]) * (pr.w ? pr.w[at + j] : 1.0f);
        s1 += d;
        s2 = __fmaf_rn(d, xh, s2);
    }
    const float m1 = warp_sum(s1) / (float)pr.N, m2 = warp_sum(s2) / (float)pr.N;
    bool bad = false;
    for (int64_t j = lane; j < pr.N; j += 32) {
        const float xh = (PxTraits<T>::cvt(x[j]) - mean) * rstd;
        const float d = PxTraits<T>::cvt(dy[j]) * (pr.w ? pr.w[at + j] : 1.0f);
        const float v = rstd * (d - m1 - xh * m2);
        dx[j] = to_out<T>(v);
        bad |= !isfinite(v);
    }
    if (bad) atomicOr(pr.status, kStatusNonFinite);
}

// column sums of dy xh and dy over a range of the M positions
template <typename T>
__global__ void __launch_bounds__(kThreads) columns_kernel(const BwdParams pr) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x, C = pr.P * pr.N;
    if (c >= C) return;
    const int64_t p = c / pr.N;
    const int64_t m0 = pr.M * blockIdx.y / kSplits, m1 = pr.M * (blockIdx.y + 1) / kSplits;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t m = m0; m < m1; ++m) {
        const float d = PxTraits<T>::cvt(static_cast<const T*>(pr.dy)[m * C + c]);
        const float x = PxTraits<T>::cvt(static_cast<const T*>(pr.x)[m * C + c]);
        sw = __fmaf_rn(d, (x - pr.mean[m * pr.P + p]) * pr.rstd[m * pr.P + p], sw);
        sb += d;
    }
    pr.part[(int64_t)blockIdx.y * 2 * C + c] = sw;
    pr.part[(int64_t)blockIdx.y * 2 * C + C + c] = sb;
}

__global__ void reduce_kernel(const float* part, float* dw, float* db, int64_t C) {
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= C) return;
    float sw = 0.0f, sb = 0.0f;
    for (int q = 0; q < kSplits; ++q) {
        sw += part[(int64_t)q * 2 * C + c];
        sb += part[(int64_t)q * 2 * C + C + c];
    }
    if (dw) dw[c] = sw;
    if (db) db[c] = sb;
}

bool bad_sizes(int64_t M, int64_t P, int64_t N) {
    const int64_t lim = int64_t(1) << 31;
    return M < 0 || P < 1 || N < 1 || M >= lim || P >= lim || N >= lim || M * P >= lim || P * N >= lim ||
           (double)M * P * N > 4.0e12;
}
}  // namespace ln
}  // namespace pararnn

using namespace pararnn;

extern "C" {

size_t pararnn_layer_norm_workspace_bytes(int64_t M, int64_t P, int64_t N) {
    if (ln::bad_sizes(M, P, N)) return 0;
    return kHeaderBytes + (size_t)(P * N) * 2 * ln::kSplits * sizeof(float);
}

pararnn_status pararnn_layer_norm_forward(int64_t M, int64_t P, int64_t N, pararnn_dtype dtype, const void* x,
                                          const float* weight, const float* bias, float eps, void* y, float* mean,
                                          float* rstd, void* workspace, size_t ws_bytes, void* stream) {
    static const char* who = "pararnn_layer_norm_forward";
    set_last_error("");
    if (ln::bad_sizes(M, P, N)) return abi::fail(who, "bad sizes");
    if (abi::bad_dtype(dtype)) return abi::fail(who, "unknown dtype");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return abi::fail(who, "eps must be finite and not negative");
    const size_t esz = dtype == PARARNN_F32 ? 4 : 2;
    if (abi::bad_pointer(x, esz, M > 0) || abi::bad_pointer(y, esz, M > 0) || abi::bad_pointer(weight, 4, false) ||
        abi::bad_pointer(bias, 4, false) || abi::bad_pointer(mean, 4, false) || abi::bad_pointer(rstd, 4, false))
        return abi::fail(who, "a pointer is null, misaligned or not device memory");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    pararnn_status s = abi::open_status(who, workspace, ws_bytes, kHeaderBytes, false, st);
    if (s != PARARNN_OK || M == 0) return s;
    ln::Params pr;
    memset(&pr, 0, sizeof pr);
    pr.x = x;
    pr.w = weight;
    pr.b = bias;
    pr.y = y;
    pr.mean = mean;
    pr.rstd = rstd;
    pr.status = static_cast<unsigned*>(workspace);
    pr.M = M;
    pr.P = P;
    pr.N = N;
    pr.eps = eps;
    const unsigned grid = (unsigned)((M * P + 3) / 4);
    if (dtype == PARARNN_F32)
        ln::forward_kernel<float><<<grid, ln::kThreads, 0, st>>>(pr);
    else
        ln::forward_kernel<ln::bf16><<<grid, ln::kThreads, 0, st>>>(pr);
    return abi::launched(who);
}

pararnn_status pararnn_layer_norm_backward(int64_t M, int64_t P, int64_t N, pararnn_dtype dtype, const void* x,
                                           const float* weight, const float* mean, const float* rstd,
                                           const void* dL_dy, void* dL_dx, float* dL_dweight, float* dL_dbias,
                                           void* workspace, size_t ws_bytes, void* stream) {
    static const char* who = "pararnn_layer_norm_backward";
    set_last_error("");
    if (ln::bad_sizes(M, P, N)) return abi::fail(who, "bad sizes");
    if (abi::bad_dtype(dtype)) return abi::fail(who, "unknown dtype");
    const size_t esz = dtype == PARARNN_F32 ? 4 : 2;
    if (abi::bad_pointer(x, esz, M > 0) || abi::bad_pointer(dL_dy, esz, M > 0) || abi::bad_pointer(dL_dx, esz, M > 0) ||
        abi::bad_pointer(mean, 4, M > 0) || abi::bad_pointer(rstd, 4, M > 0) || abi::bad_pointer(weight, 4, false) ||
        abi::bad_pointer(dL_dweight, 4, false) || abi::bad_pointer(dL_dbias, 4, false))
        return abi::fail(who, "a pointer is null, misaligned or not device memory");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    pararnn_status s =
        abi::open_status(who, workspace, ws_bytes, pararnn_layer_norm_workspace_bytes(M, P, N), true, st);
    if (s != PARARNN_OK) return s;
    if (M == 0) {
        cudaError_t e = cudaSuccess;
        if (dL_dweight) e = cudaMemsetAsync(dL_dweight, 0, (size_t)(P * N) * 4, st);
        if (e == cudaSuccess && dL_dbias) e = cudaMemsetAsync(dL_dbias, 0, (size_t)(P * N) * 4, st);
        return e == cudaSuccess ? PARARNN_OK : abi::cuda_fail(who, "clearing failed");
    }
    ln::BwdParams pr;
    memset(&pr, 0, sizeof pr);
    pr.x = x;
    pr.w = weight;
    pr.mean = mean;
    pr.rstd = rstd;
    pr.dy = dL_dy;
    pr.dx = dL_dx;
    pr.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeaderBytes);
    pr.status = static_cast<unsigned*>(workspace);
    pr.M = M;
    pr.P = P;
    pr.N = N;
    const int64_t C = P * N;
    const unsigned grid = (unsigned)((M * P + 3) / 4);
    const dim3 cols((unsigned)((C + ln::kThreads - 1) / ln::kThreads), ln::kSplits);
    if (dtype == PARARNN_F32) {
        ln::dx_kernel<float><<<grid, ln::kThreads, 0, st>>>(pr);
        if (dL_dweight || dL_dbias) ln::columns_kernel<float><<<cols, ln::kThreads, 0, st>>>(pr);
    } else {
        ln::dx_kernel<ln::bf16><<<grid, ln::kThreads, 0, st>>>(pr);
        if (dL_dweight || dL_dbias) ln::columns_kernel<ln::bf16><<<cols, ln::kThreads, 0, st>>>(pr);
    }
    s = abi::launched(who);
    if (s != PARARNN_OK || !(dL_dweight || dL_dbias)) return s;
    ln::reduce_kernel<<<(unsigned)((C + 127) / 128), 128, 0, st>>>(pr.part, dL_dweight, dL_dbias, C);
    return abi::launched(who);
}

}  // extern "C"
