// gated_scan.cu -- the gated linear recurrence: forward over sequences,
// adjoint, and the single-token step on a cache of states.
//
//   r = sig(p_r), i = sig(p_i), y = c softplus(lambda) r, a = e^-y,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t
//
// The gates do not depend on h, so the recurrence is affine and one pass is
// exact (pararnn-torch page, News section).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "abi_util.cuh"
#include "common.cuh"
#include "pararnn_b200.h"

namespace pararnn {
namespace gs {

typedef __nv_bfloat16 bf16;
constexpr int kThreads = 128;
// steps between two states that the forward keeps for the adjoint
template <typename T>
struct Ck {
    static constexpr int kSteps = sizeof(T) == 4 ? 8 : 16;
};

struct Params {
    const void* px;        // (B,T,3,D)
    const float* lam;      // (D)
    const uint8_t* reset;  // (B,T) or null
    const float* h0;       // (B,D) or null
    void* H;               // (B,T,D)
    float* last;           // (B,D) or null
    float* ck;             // (B, ceil(T / Ck), D) or null
    unsigned* status;      // workspace header word 0, or null
    int64_t B, T, D;
    float decay;
};

struct BwdParams {
    const void* px;
    const float* lam;
    const uint8_t* reset;
    const float* ck;
    const void* dH;
    const float* dlast;  // (B,D) or null
    void* dpx;
    float* part;  // (B,D)
    float* dh0;   // (B,D) or null
    unsigned* status;
    int64_t B, T, D;
    float decay;
};

__device__ __forceinline__ float softplus_f(float x) { return x > 20.0f ? x : log1pf(expf(x)); }

// a = e^-y and m = 1 - a for y >= 0.  Below 1/2 m is y times the Taylor series
// of (1 - e^-y) / y to y^8 (the first omitted term is y^9/10!, below 1e-9 of it) and
// a is 1 - m, rounded to nearest: an error of a that leans to one side would
// add up over a memory of 1/m steps.  Above 1/2 a is the exponential, which
// keeps the digits of a small a, and m is 1 - a, which cancels at most one and
// a half bits there.
__device__ __forceinline__ void decay_of(float y, float& a, float& m) {
    float s = __fmaf_rn(y, -1.0f / 362880.0f, 1.0f / 40320.0f);
    s = __fmaf_rn(y, -s, 1.0f / 5040.0f);
    s = __fmaf_rn(y, -s, 1.0f / 720.0f);
    s = __fmaf_rn(y, -s, 1.0f / 120.0f);
    s = __fmaf_rn(y, -s, 1.0f / 24.0f);
    s = __fmaf_rn(y, -s, 1.0f / 6.0f);
    s = __fmaf_rn(y, -s, 0.5f);
    s = __fmaf_rn(y, -s, 1.0f);
    const float e = exp2_approx(y * -kLog2e);
    m = y < 0.5f ? y * s : 1.0f - e;
    a = y < 0.5f ? 1.0f - m : e;
}

struct Row {
    float r, i, x, y, a, v;  // v = 1 - a^2
};
__device__ __forceinline__ Row gates(float pr, float pi, float x, float k) {
    Row o;
    o.r = sigmoid_f(pr);
    o.i = sigmoid_f(pi);
    o.x = x;
    o.y = k * o.r;
    float m;
    decay_of(o.y, o.a, m);
    o.v = m * (2.0f - m);
    return o;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Params pr) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= pr.B * pr.D) return;
    const int64_t b = c / pr.D, d = c - b * pr.D;
    const T* px = static_cast<const T*>(pr.px) + b * pr.T * 3 * pr.D + d;
    T* H = static_cast<T*>(pr.H) + b * pr.T * pr.D + d;
    const float k = pr.decay * softplus_f(pr.lam[d]);
    const int64_t nck = (pr.T + Ck<T>::kSteps - 1) / Ck<T>::kSteps;
    float h = pr.h0 ? pr.h0[c] : 0.0f;
    bool bad = false;
    for (int64_t t = 0; t < pr.T; ++t) {
        if (pr.ck && t % Ck<T>::kSteps == 0) pr.ck[(b * nck + t / Ck<T>::kSteps) * pr.D + d] = h;
        const T* p = px + t * 3 * pr.D;
        const Row g = gates(PxTraits<T>::cvt(p[0]), PxTraits<T>::cvt(p[pr.D]), PxTraits<T>::cvt(p[2 * pr.D]), k);
        const float u = sqrtf(g.v) * g.i * g.x;
        h = (pr.reset && pr.reset[b * pr.T + t]) ? u : __fmaf_rn(g.a, h, u);
        H[t * pr.D] = to_out<T>(h);
        bad |= !isfinite(h);
    }
    if (pr.last) pr.last[c] = h;
    if (bad && pr.status) atomicOr(pr.status, kStatusNonFinite);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BwdParams pr) {
    constexpr int R = Ck<T>::kSteps;
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= pr.B * pr.D) return;
    const int64_t b = c / pr.D, d = c - b * pr.D;
    const T* px = static_cast<const T*>(pr.px) + b * pr.T * 3 * pr.D + d;
    const T* dH = static_cast<const T*>(pr.dH) + b * pr.T * pr.D + d;
    T* dpx = static_cast<T*>(pr.dpx) + b * pr.T * 3 * pr.D + d;
    const float k = pr.decay * softplus_f(pr.lam[d]);
    const int64_t nck = (pr.T + R - 1) / R;
    float mu = pr.dlast ? pr.dlast[c] : 0.0f, sum = 0.0f;
    bool bad = false;
    for (int64_t q = nck - 1; q >= 0; --q) {
        float before[R];
        float h = pr.ck[(b * nck + q) * pr.D + d];
        for (int j = 0; j < R; ++j) {
            const int64_t t = q * R + j;
            if (t >= pr.T) break;
            const T* p = px + t * 3 * pr.D;
            const Row g = gates(PxTraits<T>::cvt(p[0]), PxTraits<T>::cvt(p[pr.D]), PxTraits<T>::cvt(p[2 * pr.D]), k);
            if (pr.reset && pr.reset[b * pr.T + t]) h = 0.0f;
            before[j] = h;
            h = __fmaf_rn(g.a, h, sqrtf(g.v) * g.i * g.x);
        }
        float part = 0.0f;
        for (int j = R - 1; j >= 0; --j) {
            const int64_t t = q * R + j;
            if (t >= pr.T) continue;
            const T* p = px + t * 3 * pr.D;
            T* o = dpx + t * 3 * pr.D;
            const Row g = gates(PxTraits<T>::cvt(p[0]), PxTraits<T>::cvt(p[pr.D]), PxTraits<T>::cvt(p[2 * pr.D]), k);
            const float l = PxTraits<T>::cvt(dH[t * pr.D]) + mu;
            const float rs = g.v > 0.0f ? rsqrtf(g.v) : 0.0f;
            const float dx = l * (g.v * rs) * g.i;
            const float ah = g.a * before[j];
            const float w = g.y * l * (g.a * g.a * rs * g.i * g.x - ah);
            const float dpr = w * (1.0f - g.r);
            o[0] = to_out<T>(dpr);
            o[pr.D] = to_out<T>(dx * g.x * (1.0f - g.i));
            o[2 * pr.D] = to_out<T>(dx);
            part += w;
            bad |= !isfinite(dpr) || !isfinite(dx);
            mu = (pr.reset && pr.reset[b * pr.T + t]) ? 0.0f : g.a * l;
        }
        sum += part;
    }
    if (pr.dh0) pr.dh0[c] = mu;
    pr.part[c] = sum;
    if (bad) atomicOr(pr.status, kStatusNonFinite);
}

// dL/dlambda = sig(lambda) / softplus(lambda) * sum over b of the partials, in order
__global__ void dlam_kernel(const float* part, const float* lam, float* dlam, int64_t B, int64_t D) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= D) return;
    float s = 0.0f;
    for (int64_t b = 0; b < B; ++b) s += part[b * D + d];
    const float l = lam[d];
    const float ratio = l < -15.0f ? 1.0f : 1.0f / ((1.0f + expf(-l)) * softplus_f(l));
    dlam[d] = ratio * s;
}

struct StepParams {
    const void* px;  // (N,3,D)
    const float* lam;
    const int32_t* slots;  // (N) or null
    float* state;          // (n_slots, D)
    void* y;               // (N, D)
    unsigned* status;
    int64_t N, D, n_slots;
    float decay;
};

// one thread per channel walks the rows in order
template <typename T>
__global__ void __launch_bounds__(kThreads) step_kernel(const StepParams pr) {
    const int64_t d = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (d >= pr.D) return;
    const float k = pr.decay * softplus_f(pr.lam[d]);
    unsigned bad = 0;
    for (int64_t n = 0; n < pr.N; ++n) {
        const int64_t slot = pr.slots ? pr.slots[n] : n;
        if (slot < 0 || slot >= pr.n_slots) {
            if (slot >= pr.n_slots) bad |= kStatusBadIndex;
            continue;
        }
        const T* p = static_cast<const T*>(pr.px) + n * 3 * pr.D + d;
        const Row g = gates(PxTraits<T>::cvt(p[0]), PxTraits<T>::cvt(p[pr.D]), PxTraits<T>::cvt(p[2 * pr.D]), k);
        const float h = __fmaf_rn(g.a, pr.state[slot * pr.D + d], sqrtf(g.v) * g.i * g.x);
        pr.state[slot * pr.D + d] = h;
        static_cast<T*>(pr.y)[n * pr.D + d] = to_out<T>(h);
        if (!isfinite(h)) bad |= kStatusNonFinite;
    }
    if (bad && pr.status) atomicOr(pr.status, bad);
}

bool bad_sizes(int64_t B, int64_t T, int64_t D) {
    return B < 0 || T < 0 || D < 0 || B >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) || B * T >= (int64_t(1) << 31) ||
           D >= (int64_t(1) << 31) || (double)B * T * D > 4.0e12 || (double)B * D > 1.0e11;
}
int64_t n_checkpoints(int64_t T, pararnn_dtype dt) {
    const int s = dt == PARARNN_F32 ? Ck<float>::kSteps : Ck<bf16>::kSteps;
    return (T + s - 1) / s;
}

}  // namespace gs
}  // namespace pararnn

using namespace pararnn;

extern "C" {

size_t pararnn_gated_scan_checkpoint_bytes(int64_t B, int64_t T, int64_t D, pararnn_dtype dtype) {
    if (gs::bad_sizes(B, T, D) || abi::bad_dtype(dtype)) return 0;
    return (size_t)(B * gs::n_checkpoints(T, dtype) * D) * sizeof(float);
}

size_t pararnn_gated_scan_workspace_bytes(int64_t B, int64_t T, int64_t D) {
    if (gs::bad_sizes(B, T, D)) return 0;
    return kHeaderBytes + (size_t)(B * D) * sizeof(float);
}

pararnn_status pararnn_gated_scan_forward(int64_t B, int64_t T, int64_t D, pararnn_dtype dtype, const void* preacts,
                                          const float* lambda, float decay, const float* h0, const uint8_t* reset,
                                          void* H_out, float* h_last, float* checkpoints, void* workspace,
                                          size_t ws_bytes, void* stream) {
    static const char* who = "pararnn_gated_scan_forward";
    set_last_error("");
    if (gs::bad_sizes(B, T, D)) return abi::fail(who, "bad sizes");
    if (abi::bad_dtype(dtype)) return abi::fail(who, "unknown dtype");
    if (!(decay > 0.0f) || !std::isfinite(decay)) return abi::fail(who, "decay must be positive and finite");
    const size_t esz = dtype == PARARNN_F32 ? 4 : 2;
    const bool empty = B == 0 || T == 0 || D == 0;
    if (abi::bad_pointer(preacts, esz, !empty) || abi::bad_pointer(lambda, 4, !empty) ||
        abi::bad_pointer(H_out, esz, !empty) || abi::bad_pointer(h0, 4, false) || abi::bad_pointer(reset, 1, false) ||
        abi::bad_pointer(h_last, 4, false) || abi::bad_pointer(checkpoints, 4, false))
        return abi::fail(who, "a pointer is null, misaligned or not device memory");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    pararnn_status s = abi::open_status(who, workspace, ws_bytes, kHeaderBytes, false, st);
    if (s != PARARNN_OK) return s;
    if (empty) {
        if (h_last && h_last != h0 && B * D > 0) {
            const size_t n = (size_t)(B * D) * 4;
            const cudaError_t e = h0 ? cudaMemcpyAsync(h_last, h0, n, cudaMemcpyDeviceToDevice, st)
                                     : cudaMemsetAsync(h_last, 0, n, st);
            if (e != cudaSuccess) return abi::cuda_fail(who, "copy failed");
        }
        return PARARNN_OK;
    }
    gs::Params pr;
    memset(&pr, 0, sizeof pr);
    pr.px = preacts;
    pr.lam = lambda;
    pr.reset = reset;
    pr.h0 = h0;
    pr.H = H_out;
    pr.last = h_last;
    pr.ck = checkpoints;
    pr.status = static_cast<unsigned*>(workspace);
    pr.B = B;
    pr.T = T;
    pr.D = D;
    pr.decay = decay;
    const unsigned grid = (unsigned)((B * D + gs::kThreads - 1) / gs::kThreads);
    if (dtype == PARARNN_F32)
        gs::forward_kernel<float><<<grid, gs::kThreads, 0, st>>>(pr);
    else
        gs::forward_kernel<gs::bf16><<<grid, gs::kThreads, 0, st>>>(pr);
    return abi::launched(who);
}

pararnn_status pararnn_gated_scan_backward(int64_t B, int64_t T, int64_t D, pararnn_dtype dtype, const void* preacts,
                                           const float* lambda, float decay, const uint8_t* reset,
                                           const float* checkpoints, const void* dL_dH, const float* dL_dh_last,
                                           void* dL_dpx, float* dL_dlambda, float* dL_dh0, void* workspace,
                                           size_t ws_bytes, void* stream) {
    static const char* who = "pararnn_gated_scan_backward";
    set_last_error("");
    if (gs::bad_sizes(B, T, D)) return abi::fail(who, "bad sizes");
    if (abi::bad_dtype(dtype)) return abi::fail(who, "unknown dtype");
    if (!(decay > 0.0f) || !std::isfinite(decay)) return abi::fail(who, "decay must be positive and finite");
    const size_t esz = dtype == PARARNN_F32 ? 4 : 2;
    const bool empty = B == 0 || T == 0 || D == 0;
    if (abi::bad_pointer(preacts, esz, !empty) || abi::bad_pointer(lambda, 4, !empty) ||
        abi::bad_pointer(checkpoints, 4, !empty) || abi::bad_pointer(dL_dH, esz, !empty) ||
        abi::bad_pointer(dL_dpx, esz, !empty) || abi::bad_pointer(reset, 1, false) ||
        abi::bad_pointer(dL_dh_last, 4, false) || abi::bad_pointer(dL_dlambda, 4, false) ||
        abi::bad_pointer(dL_dh0, 4, false))
        return abi::fail(who, "a pointer is null, misaligned or not device memory");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    pararnn_status s =
        abi::open_status(who, workspace, ws_bytes, pararnn_gated_scan_workspace_bytes(B, T, D), true, st);
    if (s != PARARNN_OK) return s;
    if (empty) {
        cudaError_t e = cudaSuccess;
        if (dL_dlambda && D > 0) e = cudaMemsetAsync(dL_dlambda, 0, (size_t)D * 4, st);
        if (e == cudaSuccess && dL_dh0 && dL_dh0 != dL_dh_last && B * D > 0)
            e = dL_dh_last ? cudaMemcpyAsync(dL_dh0, dL_dh_last, (size_t)(B * D) * 4, cudaMemcpyDeviceToDevice, st)
                           : cudaMemsetAsync(dL_dh0, 0, (size_t)(B * D) * 4, st);
        return e == cudaSuccess ? PARARNN_OK : abi::cuda_fail(who, "copy failed");
    }
    gs::BwdParams pr;
    memset(&pr, 0, sizeof pr);
    pr.px = preacts;
    pr.lam = lambda;
    pr.reset = reset;
    pr.ck = checkpoints;
    pr.dH = dL_dH;
    pr.dlast = dL_dh_last;
    pr.dpx = dL_dpx;
    pr.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeaderBytes);
    pr.dh0 = dL_dh0;
    pr.status = static_cast<unsigned*>(workspace);
    pr.B = B;
    pr.T = T;
    pr.D = D;
    pr.decay = decay;
    const unsigned grid = (unsigned)((B * D + gs::kThreads - 1) / gs::kThreads);
    if (dtype == PARARNN_F32)
        gs::backward_kernel<float><<<grid, gs::kThreads, 0, st>>>(pr);
    else
        gs::backward_kernel<gs::bf16><<<grid, gs::kThreads, 0, st>>>(pr);
    s = abi::launched(who);
    if (s != PARARNN_OK || !dL_dlambda) return s;
    gs::dlam_kernel<<<(unsigned)((D + 127) / 128), 128, 0, st>>>(pr.part, lambda, dL_dlambda, B, D);
    return abi::launched(who);
}

pararnn_status pararnn_gated_scan_step(int64_t N, int64_t D, pararnn_dtype dtype, const void* preacts,
                                       const float* lambda, float decay, int64_t n_slots, const int32_t* slots,
                                       float* state, void* y, void* workspace, size_t ws_bytes, void* stream) {
    static const char* who = "pararnn_gated_scan_step";
    set_last_error("");
    if (gs::bad_sizes(N, 1, D) || gs::bad_sizes(n_slots, 1, D)) return abi::fail(who, "bad sizes");
    if (abi::bad_dtype(dtype)) return abi::fail(who, "unknown dtype");
    if (!(decay > 0.0f) || !std::isfinite(decay)) return abi::fail(who, "decay must be positive and finite");
    if (!slots && n_slots < N) return abi::fail(who, "fewer slots than rows");
    const size_t esz = dtype == PARARNN_F32 ? 4 : 2;
    const bool empty = N == 0 || D == 0;
    if (abi::bad_pointer(preacts, esz, !empty) || abi::bad_pointer(lambda, 4, !empty) ||
        abi::bad_pointer(state, 4, !empty && n_slots > 0) || abi::bad_pointer(y, esz, !empty) ||
        abi::bad_pointer(slots, 4, false))
        return abi::fail(who, "a pointer is null, misaligned or not device memory");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    pararnn_status s = abi::open_status(who, workspace, ws_bytes, kHeaderBytes, false, st);
    if (s != PARARNN_OK || empty) return s;
    gs::StepParams pr;
    memset(&pr, 0, sizeof pr);
    pr.px = preacts;
    pr.lam = lambda;
    pr.slots = slots;
    pr.state = state;
    pr.y = y;
    pr.status = static_cast<unsigned*>(workspace);
    pr.N = N;
    pr.D = D;
    pr.n_slots = n_slots;
    pr.decay = decay;
    const unsigned grid = (unsigned)((D + gs::kThreads - 1) / gs::kThreads);
    if (dtype == PARARNN_F32)
        gs::step_kernel<float><<<grid, gs::kThreads, 0, st>>>(pr);
    else
        gs::step_kernel<gs::bf16><<<grid, gs::kThreads, 0, st>>>(pr);
    return abi::launched(who);
}

}  // extern "C"
