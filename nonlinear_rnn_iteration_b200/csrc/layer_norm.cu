// layer_norm.cu -- layer normalisation of (M, P, N) rows, forward and
// backward, with a scale and a shift for each of the P gates or heads.
//
//   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps), y = xh w + b
//   with d = dy w:  dx = rstd (d - mean(d) - xh mean(d xh)),
//   dw = sum over M of dy xh,  db = sum over M of dy
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "abi_util.cuh"
#include "bulk.cuh"
#include "common.cuh"
#include "pararnn_b200.h"

namespace pararnn {
namespace ln {

typedef __nv_bfloat16 bf16;

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
    int tpr;           // threads per row
    int pb, gpp, npc;  // row slots of one block: pb of the P parameter rows, gpp positions each; ranges of P
};
struct BwdParams {
    const void* x;
    const float* w;
    const float* mean;
    const float* rstd;
    const void* dy;
    void* dx;
    float* part;  // [range of positions][2][P * N], or null
    unsigned* status;
    int64_t M, P, N;
    int tpr, pb, gpp, npc;
};

// ---- rows in registers ----------------------------------------------------------
// A row of N values belongs to `tpr` threads (a power of two), each with K vectors of V
// values, read and written once.  A thread's rows all have the same p, so that it
// keeps its weights, and in the backward pass its column sums, in registers over all
// its rows.  U rows are read and reduced at a time: that keeps enough bytes in flight and
// shares a block barrier between them.  Two reductions of a row in the forward pass
// (the variance is taken about the mean), one of two sums in the backward pass.
// Batches in which every thread of the block has all its values take a copy of the code without
// conditions where that was measured to gain (replayed from a graph, with and without): in the forward with
// vector accesses and 256 threads of up to 32 values (100000x1x256 bfloat16 20.1 us, 23.5; 131072x1x1024
// float32 184, 190) and in the backward with up to 8 values (100000x1x256 37.4, 41.1).  Not with the larger blocks of
// longer rows (8x1x8192 bfloat16 11.3, 10.6; 16384x1x16384 float32 374, 354), with single values
// (20000x1x1001 float32 53.4, 50.9), nor with 64 values forward (32768x3x2048 bfloat16 163, 152) or 16
// backward (283, 248).  What the compiler reports as spilled does not follow these gains.
// Measured: 131072x1x1024 float32 186 us forward, 5.8 TB/s, and 245 us backward, 6.6 TB/s, bound by HBM;
// 32768x3x2048 bfloat16 149 us, 5.4 TB/s, bound by the latency of the row loads, for which
// registers are left, and 249 us, 4.9 TB/s, bound by issue and the rows' barrier; rows of 64, 32768x8x64
// bfloat16, 15 us and 28 us, bound by instructions.
template <typename T, int V, int K>
constexpr int words_of = K * (V * (int)sizeof(T) >= 4 ? V * (int)sizeof(T) / 4 : 1);
constexpr int batch_of(int words) { return words >= 16 ? 1 : words >= 8 ? 2 : 4; }
template <typename T, int V>
struct Vec {
    static constexpr int kWords = V * sizeof(T) / 4;
    uint32_t r[kWords > 0 ? kWords : 1];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
    Vec<T, V> v;
    if constexpr (V * sizeof(T) == 16) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v.r[0] = q.x, v.r[1] = q.y, v.r[2] = q.z, v.r[3] = q.w;
    } else if constexpr (V * sizeof(T) == 4) {
        v.r[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        v.r[0] = *reinterpret_cast<const uint16_t*>(p);
    }
    return v;
}
template <typename T, int V>
__device__ __forceinline__ float value(const Vec<T, V>& v, int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(v.r[i]);
    return __uint_as_float(i & 1 ? v.r[i / 2] & 0xffff0000u : v.r[i / 2] << 16);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4)
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        else
            p[0] = v[0];
    } else if constexpr (V == 1) {
        p[0] = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// Sums over a row's threads of n values.  Rows of more than a warp meet in shared
// memory, two buffers in turn; every thread of the block takes part.
template <int n>
__device__ __forceinline__ void row_sums(float (&a)[n], int tpr, float (*buf)[32][n], int& turn) {
    for (int o = min(tpr, 32) >> 1; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, per = tpr >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < n; ++i) buf[turn][warp][i] = a[i];
        __syncthreads();
        const float(*q)[n] = buf[turn] + warp / per * per;
#pragma unroll
        for (int i = 0; i < n; ++i) a[i] = 0.0f;
        for (int w = 0; w < per; ++w)
#pragma unroll
            for (int i = 0; i < n; ++i) a[i] += q[w][i];
        turn ^= 1;
    }
}

// the rows of this thread's group: positions m, m + dm, ... below M with parameter row p.  Positions
// fit 32 bits (dm is at most the threads of the device); rows and values are counted in 64.
struct Rows {
    int64_t p, row, drow;  // the first row, and the way to the next
    uint32_t m, dm, steps;  // steps: of the whole block, the most rows that one of its groups has
    uint32_t full;          // the first steps in which every thread of the block has `each` values
    bool on;
};
template <class P>
__device__ __forceinline__ Rows rows_of(const P& pr, int each) {
    const int g = threadIdx.x / pr.tpr;
    const int64_t range = blockIdx.x % pr.npc, slot = blockIdx.x / pr.npc, slots = gridDim.x / pr.npc;
    Rows r;
    r.p = range * pr.pb + g % pr.pb;
    r.m = (uint32_t)(slot * pr.gpp + g / pr.pb);
    r.dm = (uint32_t)(slots * pr.gpp);
    r.row = (int64_t)r.m * pr.P + r.p;
    r.drow = (int64_t)r.dm * pr.P;
    r.on = g < pr.pb * pr.gpp && r.p < pr.P;
    r.steps = (uint32_t)((pr.M - slot * pr.gpp + r.dm - 1) / r.dm);
    const int64_t last = pr.M - (slot * pr.gpp + pr.gpp - 1);
    const bool all = pr.pb * pr.gpp * pr.tpr == (int)blockDim.x && (range + 1) * pr.pb <= pr.P && pr.N == pr.tpr * each;
    r.full = all && last > 0 ? (uint32_t)((last + r.dm - 1) / r.dm) : 0u;
    return r;
}

// The E = K V values of a thread in pairs, so that two go through one packed instruction:
// pair e is values 2e, 2e + 1.  Only where V is 1 can a pair be half inside the row.
template <typename T, int V, int K>
__device__ __forceinline__ f2 pair(const Vec<T, V> (&v)[K], int e) {
    if constexpr (V == 1) return f2{value<T, V>(v[2 * e], 0), value<T, V>(v[2 * e + 1], 0)};
    return f2{value<T, V>(v[2 * e / V], 2 * e % V), value<T, V>(v[2 * e / V], 2 * e % V + 1)};
}
// columns of a thread: which of its values lie in the row
template <int V, int K, bool kFull = false>
struct Columns {
    int j0, dj, N;
    __device__ __forceinline__ int of(int e) const { return j0 + e / V * dj + e % V; }
    __device__ __forceinline__ bool in(int k) const { return kFull || j0 + k * dj < N; }
    // a pair with zeros in place of the values past the row, where V is 1
    __device__ __forceinline__ f2 mask(f2 x, int e) const {
        if constexpr (V > 1 || kFull) return x;
        return f2{in(2 * e) ? x.x : 0.0f, in(2 * e + 1) ? x.y : 0.0f};
    }
    // f(e) for the pairs that lie in the row, at least in part
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        if constexpr (V == 1) {
#pragma unroll
            for (int e = 0; e < K / 2; ++e) f(e);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in(k))
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) f(k * (V / 2) + i);
        }
    }
};
__device__ __forceinline__ float total(f2 x) { return x.x + x.y; }

// s / n from inv = 1 / n, rounded: the product is up to 1.5 steps off (of a constant row's mean, with n = 1000, for
// most values), and what it leaves of s, which one fused multiply-add gives exactly, corrects it (P. W. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000", IBM J. Res. Dev. 34 (1990)): where s is a
// multiple of n the mean is exact, so that a constant row, whatever its size, has no spread.  A division
// in its place is a call, around which most of these kernels spill.
__device__ __forceinline__ float mean_of(float s, float n, float inv) {
    const float q = s * inv;
    return __fmaf_rn(__fmaf_rn(-q, n, s), inv, q);
}

// The 16-byte accesses of a warp to a batch of rows, kN of them, brought ahead as pieces of 512
// bytes by a bulk copy of one lane each, into the warp's own part of the shared memory: bytes are
// in flight while the batch before is at work, without registers for them.
template <int kN>
struct Ring {
    static constexpr int kBytes = kN * 512;
    unsigned char* piece;
    uint64_t* bar;
    unsigned phase = 0;

    __device__ __forceinline__ Ring(unsigned char* all, uint64_t* bars)
        : piece(all + threadIdx.x / 32 * kBytes), bar(bars + threadIdx.x / 32) {
        if (threadIdx.x % 32 == 0) {
            mbar_init(bar, 1);
            mbar_fence_init();
        }
        __syncwarp();
    }
    // where(i, src) gives the bytes of piece i and its place; 0 for none
    template <class F>
    __device__ __forceinline__ void fill(F where) {
        const int lane = threadIdx.x % 32;
        const void* src = nullptr;
        const unsigned n = lane < kN ? where(lane, src) : 0u, all = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) mbar_arrive_expect_tx(bar, all);
        __syncwarp();
        if (n) bulk_load(piece + lane * 512, reinterpret_cast<uintptr_t>(src), n, bar);
    }
    __device__ __forceinline__ void wait(bool& late) {
        wait_bar<false>(bar, phase, late);
        phase ^= 1;
    }
    template <class V>
    __device__ __forceinline__ V read(int i) const {
        const uint4 q = *reinterpret_cast<const uint4*>(piece + i * 512 + threadIdx.x % 32 * 16);
        V v;
        v.r[0] = q.x, v.r[1] = q.y, v.r[2] = q.z, v.r[3] = q.w;
        return v;
    }
};
struct NoRing {
    __device__ __forceinline__ NoRing(unsigned char*, uint64_t*) {}
};
// Where rows are brought ahead: with 16-byte accesses, and where a row has a warp at least (more
// than 8 values a thread).  Measured on earlier code, with and without: in the backward pass (131072x1x1024
// float32 251 us, 279; 32768x3x2048 bfloat16 249, 253), but not with 1024 threads, whose 64 registers spill
// (16384x1x16384 float32 1435 us, 1250).  In the forward only with 512 threads, one block to an SM
// (16384x1x16384 float32 377, 454); more blocks hide the loads themselves, and the rings
// take their shared memory (32768x3x2048 bfloat16 164, 152).
template <typename T, int V, int K, int kThreads, bool kForward>
constexpr bool kRing = V * sizeof(T) == 16 && V * K > 8 && (kForward ? kThreads == 512 : kThreads <= 512);
// rows that a thread of the backward pass reads at a time
template <typename T, int V, int K, int kThreads>
constexpr int kBackRows = kThreads > 512 ? 1 : batch_of(words_of<T, V, K>);

template <typename T, int V, int K, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 1) forward_rows(const Params pr) {
    constexpr int U = batch_of(words_of<T, V, K>), E = K * V;
    // the weights in registers, or, for more values, in shared memory: [w, b][quads][threads of a row]
    constexpr bool kHold = E <= 16;
    constexpr bool kAhead = kRing<T, V, K, kThreads, true>;
    __shared__ float buf[2][32][U];
    __shared__ uint64_t bars[kAhead ? 32 : 1];
    extern __shared__ __align__(16) float4 held[];
    follow_previous();
    Rows rows = rows_of(pr, E);
    const uint32_t M = (uint32_t)pr.M;
    const Columns<V, K> c0{(int)(threadIdx.x % pr.tpr) * V, pr.tpr * V, (int)pr.N};
    const int N = c0.N;
    const float n = (float)N, inv = 1.0f / n;
    int turn = 0;
    f2 chk{0.0f, 0.0f}, w[kHold ? E / 2 : 1], b[kHold ? E / 2 : 1];
    auto weight = [&](const float* from, int e, float none) {
        f2 o{none, none};
        if (from) {
            if constexpr (V == 1) {
                if (c0.of(2 * e) < N) o.x = from[rows.p * N + c0.of(2 * e)];
                if (c0.of(2 * e + 1) < N) o.y = from[rows.p * N + c0.of(2 * e + 1)];
            } else if (c0.of(2 * e) < N) {
                const float* q = from + rows.p * N + c0.of(2 * e);
                o = f2{q[0], q[1]};
            }
        }
        return o;
    };
    const int quads = pr.tpr * (E / 4), at = c0.j0 / V;
    if constexpr (kHold) {
        if (rows.on)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) w[e] = weight(pr.w, e, 1.0f), b[e] = weight(pr.b, e, 0.0f);
    } else {
        // the block's rows share one parameter row; its first group lays it out
        if ((int)threadIdx.x < pr.tpr)
#pragma unroll
            for (int e = 0; e < E / 2; e += 2) {
                f2 q = weight(pr.w, e, 1.0f), r = weight(pr.w, e + 1, 1.0f);
                held[e / 2 * pr.tpr + at] = make_float4(q.x, q.y, r.x, r.y);
                q = weight(pr.b, e, 0.0f), r = weight(pr.b, e + 1, 0.0f);
                held[quads + e / 2 * pr.tpr + at] = make_float4(q.x, q.y, r.x, r.y);
            }
        __syncthreads();
    }
    int64_t at0 = rows.row * N + c0.j0;  // the thread's first value
    const int64_t dat = rows.drow * N;
    bool late = false;
    auto fill = [&](auto& ring) {
        ring.fill([&](int i, const void*& src) {
            const int u = i / K, j = (c0.j0 & ~(32 * V - 1)) + i % K * c0.dj;
            src = static_cast<const T*>(pr.x) + rows.row * N + u * dat + j;
            return rows.on && rows.m + u * rows.dm < M && j < N ? min(32 * V, N - j) * (unsigned)sizeof(T) : 0u;
        });
    };
    std::conditional_t<kAhead, Ring<U * K>, NoRing> ring(
        reinterpret_cast<unsigned char*>(held) + (kHold ? 0 : (size_t)quads * 2 * sizeof(float4)), bars);
    if constexpr (kAhead) fill(ring);
    auto batch = [&](uint32_t it, auto full) {
        constexpr bool kFull = decltype(full)::value;
        const Columns<V, K, kFull> c{c0.j0, c0.dj, N};
        Vec<T, V> v[U][K];
        float s[U], mean[U];
        if constexpr (kAhead) ring.wait(late);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = kFull || (rows.on && rows.m + u * rows.dm < M);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                v[u][k] = Vec<T, V>{};
                if (on && c.in(k)) {
                    if constexpr (kAhead)
                        v[u][k] = ring.template read<Vec<T, V>>(u * K + k);
                    else
                        v[u][k] = load<T, V>(static_cast<const T*>(pr.x) + at0 + u * dat + k * c.dj);
                }
            }
        }
        const uint32_t m = rows.m;
        const int64_t row = rows.row, begin = at0;
        rows.m += U * rows.dm;
        rows.row += U * rows.drow;
        at0 += U * dat;
        if constexpr (kAhead)
            if (it + U < rows.steps) {
                __syncwarp();
                fill(ring);
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2 t{0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < E / 2; ++e) t = add2(t, pair(v[u], e));
            s[u] = total(t);
        }
        row_sums(s, pr.tpr, buf, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[u] = mean_of(s[u], n, inv);
            f2 t{0.0f, 0.0f};
            c.each([&](int e) {
                const f2 d = c.mask(sub2(pair(v[u], e), splat2(mean[u])), e);
                t = fma2(d, d, t);
            });
            s[u] = total(t);
        }
        row_sums(s, pr.tpr, buf, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!kFull && (!rows.on || m + u * rows.dm >= M)) continue;
            const float rstd = rsqrtf(s[u] * inv + pr.eps);  // within 2 ulp
            T* y = static_cast<T*>(pr.y) + begin + u * dat;
            auto out = [&](int e, f2 we, f2 be) {
                const f2 xh = mul2(sub2(pair(v[u], e), splat2(mean[u])), splat2(rstd));
                const f2 o = fma2(xh, we, be);
                chk = fma2(c.mask(o, e), splat2(0.0f), chk);
                return o;
            };
            auto value_of = [&](int e) {
                if constexpr (kHold) {
                    return out(e, w[e], b[e]);
                } else {
                    const float4 q = held[e / 2 * pr.tpr + at], r = held[quads + e / 2 * pr.tpr + at];
                    return out(e, e & 1 ? f2{q.z, q.w} : f2{q.x, q.y}, e & 1 ? f2{r.z, r.w} : f2{r.x, r.y});
                }
            };
            if constexpr (V == 1) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const f2 o = value_of(e);
                    if (c.in(2 * e)) store<T, 1>(y + 2 * e * c.dj, &o.x);
                    if (c.in(2 * e + 1)) store<T, 1>(y + (2 * e + 1) * c.dj, &o.y);
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (c.in(k)) {
                        float o[V];
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const f2 q = value_of(k * (V / 2) + i);
                            o[2 * i] = q.x, o[2 * i + 1] = q.y;
                        }
                        store<T, V>(y + k * c.dj, o);
                    }
            }
            if (c.j0 == 0 && pr.mean) pr.mean[row + u * rows.drow] = mean[u];
            if (c.j0 == 0 && pr.rstd) pr.rstd[row + u * rows.drow] = rstd;
        }
    };
    for (uint32_t it = 0; it < rows.steps; it += U) {
        if constexpr (kThreads == 256 && V > 1 && E <= 32)
            it + U <= rows.full ? batch(it, std::true_type{}) : batch(it, std::false_type{});
        else
            batch(it, std::false_type{});
    }
    const unsigned bits = (total(chk) != total(chk) ? kStatusNonFinite : 0u) | (late ? kStatusTimeout : 0u);
    if (pr.status && bits) atomicOr(pr.status, bits);
}

template <typename T, int V, int K, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1) backward_rows(const BwdParams pr) {
    constexpr int U = kBackRows<T, V, K, kThreads>, E = K * V;
    constexpr bool kHold = kThreads <= 512, kAhead = kRing<T, V, K, kThreads, false>;
    __shared__ float buf[2][32][2 * U];
    __shared__ uint64_t bars[kAhead ? 32 : 1];
    extern __shared__ __align__(16) float4 sums[];  // [K * V / 2][threads]; before that, the warps' rings
    follow_previous();
    Rows rows = rows_of(pr, E);
    const uint32_t M = (uint32_t)pr.M;
    const Columns<V, K> c0{(int)(threadIdx.x % pr.tpr) * V, pr.tpr * V, (int)pr.N};
    const int N = c0.N;
    const float n = (float)N, inv = 1.0f / n;
    int turn = 0;
    // with 1024 threads, of 64 registers, the column sums stay in shared memory (16384x1x16384 float32
    // 1110 us; in spilled registers, on earlier code, 1287)
    f2 w[E / 2], dw[kHold ? E / 2 : 1], db[kHold ? E / 2 : 1], chk{0.0f, 0.0f};
    auto params = [&]() {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            w[e] = splat2(1.0f);
            if (pr.w && rows.on) {
                if (c0.of(2 * e) < N) w[e].x = pr.w[rows.p * N + c0.of(2 * e)];
                if (c0.of(2 * e + 1) < N) w[e].y = pr.w[rows.p * N + c0.of(2 * e + 1)];
            }
        }
    };
    if constexpr (kHold) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) dw[e] = db[e] = splat2(0.0f);
        params();
    } else if (pr.part) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) sums[e * kThreads + threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    int64_t at0 = rows.row * N + c0.j0;  // the thread's first value
    const int64_t dat = rows.drow * N;
    bool late = false;
    auto fill = [&](auto& ring) {
        ring.fill([&](int i, const void*& src) {
            const int u = i / K / 2, j = (c0.j0 & ~(32 * V - 1)) + i % K * c0.dj;
            src = static_cast<const T*>(i / K % 2 ? pr.dy : pr.x) + rows.row * N + u * dat + j;
            return rows.on && rows.m + u * rows.dm < M && j < N ? min(32 * V, N - j) * (unsigned)sizeof(T) : 0u;
        });
    };
    float mean[U], rstd[U];
    auto stats = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = rows.on && rows.m + u * rows.dm < M;
            mean[u] = on ? pr.mean[rows.row + u * rows.drow] : 0.0f;
            rstd[u] = on ? pr.rstd[rows.row + u * rows.drow] : 0.0f;
        }
    };
    std::conditional_t<kAhead, Ring<2 * U * K>, NoRing> ring(reinterpret_cast<unsigned char*>(sums), bars);
    if constexpr (kAhead) {
        fill(ring);
        stats();
    }
    auto batch = [&](uint32_t it, auto full) {
        constexpr bool kFull = decltype(full)::value;
        const Columns<V, K, kFull> c{c0.j0, c0.dj, N};
        Vec<T, V> v[U][K], g[U][K];
        float s[2 * U];
        if constexpr (kAhead)
            ring.wait(late);
        else
            stats();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = kFull || (rows.on && rows.m + u * rows.dm < M);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                v[u][k] = Vec<T, V>{};
                g[u][k] = Vec<T, V>{};
                if (on && c.in(k)) {
                    if constexpr (kAhead) {
                        v[u][k] = ring.template read<Vec<T, V>>(2 * u * K + k);
                        g[u][k] = ring.template read<Vec<T, V>>((2 * u + 1) * K + k);
                    } else {
                        v[u][k] = load<T, V>(static_cast<const T*>(pr.x) + at0 + u * dat + k * c.dj);
                        g[u][k] = load<T, V>(static_cast<const T*>(pr.dy) + at0 + u * dat + k * c.dj);
                    }
                }
            }
        }
        const uint32_t m = rows.m;
        const int64_t begin = at0;
        rows.m += U * rows.dm;
        rows.row += U * rows.drow;
        at0 += U * dat;
        if constexpr (kAhead)
            if (it + U < rows.steps) {
                __syncwarp();
                fill(ring);
            }
        if (!kHold) params();
        // rows past M hold zeros: they add nothing
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2 t1{0.0f, 0.0f}, t2 = t1;
            c.each([&](int e) {
                // past the row dy is zero, but the mean need not be finite
                const f2 xh = c.mask(mul2(sub2(pair(v[u], e), splat2(mean[u])), splat2(rstd[u])), e);
                const f2 dy = pair(g[u], e), d = mul2(dy, w[e]);
                t1 = add2(t1, d);
                t2 = fma2(d, xh, t2);
                if constexpr (kHold) {
                    db[e] = add2(db[e], dy);
                    dw[e] = fma2(dy, xh, dw[e]);
                } else if (pr.part) {
                    float4& q = sums[e * kThreads + threadIdx.x];
                    const f2 tw = fma2(dy, xh, f2{q.x, q.y}), tb = add2(f2{q.z, q.w}, dy);
                    q = make_float4(tw.x, tw.y, tb.x, tb.y);
                }
            });
            s[2 * u] = total(t1);
            s[2 * u + 1] = total(t2);
        }
        row_sums(s, pr.tpr, buf, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!kFull && (!rows.on || m + u * rows.dm >= M)) continue;
            const f2 m1 = splat2(mean_of(s[2 * u], n, inv)), m2 = splat2(-s[2 * u + 1] * inv);
            T* o = static_cast<T*>(pr.dx) + begin + u * dat;
            auto out = [&](int e) {
                const f2 xh = mul2(sub2(pair(v[u], e), splat2(mean[u])), splat2(rstd[u]));
                const f2 q = mul2(fma2(xh, m2, sub2(mul2(pair(g[u], e), w[e]), m1)), splat2(rstd[u]));
                chk = fma2(c.mask(q, e), splat2(0.0f), chk);
                return q;
            };
            if constexpr (V == 1) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const f2 q = out(e);
                    if (c.in(2 * e)) store<T, 1>(o + 2 * e * c.dj, &q.x);
                    if (c.in(2 * e + 1)) store<T, 1>(o + (2 * e + 1) * c.dj, &q.y);
                }
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (c.in(k)) {
                        float q[V];
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const f2 t = out(k * (V / 2) + i);
                            q[2 * i] = t.x, q[2 * i + 1] = t.y;
                        }
                        store<T, V>(o + k * c.dj, q);
                    }
            }
        }
        if constexpr (kAhead) stats();  // of the next batch
    };
    for (uint32_t it = 0; it < rows.steps; it += U) {
        if constexpr (E <= 8)
            it + U <= rows.full ? batch(it, std::true_type{}) : batch(it, std::false_type{});
        else
            batch(it, std::false_type{});
    }
    const unsigned bits = (total(chk) != total(chk) ? kStatusNonFinite : 0u) | (late ? kStatusTimeout : 0u);
    if (bits) atomicOr(pr.status, bits);
    if (!pr.part) return;
    if constexpr (kAhead) __syncthreads();  // the sums lie where the rings were
    // the block's column sums: the groups of one parameter row in order
    if constexpr (kHold)
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
            sums[e * blockDim.x + threadIdx.x] = make_float4(dw[e].x, dw[e].y, db[e].x, db[e].y);
    __syncthreads();
    const int g0 = threadIdx.x / pr.tpr;
    if (g0 < pr.pb && rows.p < pr.P) {
        float* to = pr.part + (int64_t)(blockIdx.x / pr.npc) * 2 * pr.P * N + rows.p * N;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int q = 0; q < pr.gpp; ++q) {
                const float4 u = sums[e * blockDim.x + threadIdx.x + q * pr.pb * pr.tpr];
                t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
            }
            const int j = c0.of(2 * e), j1 = c0.of(2 * e + 1);
            if (j < N) to[j] = t.x, to[pr.P * N + j] = t.z;
            if (j1 < N) to[j1] = t.y, to[pr.P * N + j1] = t.w;
        }
    }
}

// ---- rows of any length -----------------------------------------------------------
// For rows that do not fit a block's registers: a block per row, which reads it
// once for each sum; the column sums are formed by a kernel of their own.  4096x1x20000 bfloat16 207 us
// forward, 460 backward (the bytes of one reading and writing at the copy's rate: 50 and 75), float32 237 and 584
// (100 and 150): values are loaded one at a time, and each input three times.
constexpr int kLongThreads = 512;

__device__ __forceinline__ float2 block_sum(float a, float b) {
    __shared__ float2 buf[kLongThreads / 32];
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < kLongThreads / 32; ++i) a += buf[i].x, b += buf[i].y;
    return make_float2(a, b);
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) forward_long(const Params pr) {
    follow_previous();
    float chk = 0.0f;
    for (int64_t row = blockIdx.x; row < pr.M * pr.P; row += gridDim.x) {
        const T* x = static_cast<const T*>(pr.x) + row * pr.N;
        T* y = static_cast<T*>(pr.y) + row * pr.N;
        const int64_t at = (row % pr.P) * pr.N;
        float s = 0.0f;
        for (int64_t j = threadIdx.x; j < pr.N; j += kLongThreads) s += PxTraits<T>::cvt(x[j]);
        const float mean = block_sum(s, 0.0f).x / (float)pr.N;
        s = 0.0f;
        for (int64_t j = threadIdx.x; j < pr.N; j += kLongThreads) {
            const float c = PxTraits<T>::cvt(x[j]) - mean;
            s = __fmaf_rn(c, c, s);
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, 0.0f).x / (float)pr.N + pr.eps);
        for (int64_t j = threadIdx.x; j < pr.N; j += kLongThreads) {
            const float xh = (PxTraits<T>::cvt(x[j]) - mean) * rstd;
            const float v = __fmaf_rn(xh, pr.w ? pr.w[at + j] : 1.0f, pr.b ? pr.b[at + j] : 0.0f);
            y[j] = to_out<T>(v);
            chk = __fmaf_rn(v, 0.0f, chk);
        }
        if (threadIdx.x == 0 && pr.mean) pr.mean[row] = mean;
        if (threadIdx.x == 0 && pr.rstd) pr.rstd[row] = rstd;
    }
    if (chk != chk && pr.status) atomicOr(pr.status, kStatusNonFinite);
}

// column sums of dy xh and dy over a range of the M positions: before dx, which may
// be written over x or dy
template <typename T>
__global__ void __launch_bounds__(kLongThreads) columns_long(const BwdParams pr) {
    follow_previous();
    const int64_t c = (int64_t)blockIdx.x * kLongThreads + threadIdx.x, C = pr.P * pr.N;
    if (c >= C) return;
    const int64_t p = c / pr.N;
    const int64_t m0 = pr.M * blockIdx.y / gridDim.y, m1 = pr.M * (blockIdx.y + 1) / gridDim.y;
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

template <typename T>
__global__ void __launch_bounds__(kLongThreads) dx_long(const BwdParams pr) {
    follow_previous();
    float chk = 0.0f;
    for (int64_t row = blockIdx.x; row < pr.M * pr.P; row += gridDim.x) {
        const T* x = static_cast<const T*>(pr.x) + row * pr.N;
        const T* dy = static_cast<const T*>(pr.dy) + row * pr.N;
        T* dx = static_cast<T*>(pr.dx) + row * pr.N;
        const int64_t at = (row % pr.P) * pr.N;
        const float mean = pr.mean[row], rstd = pr.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t j = threadIdx.x; j < pr.N; j += kLongThreads) {
            const float xh = (PxTraits<T>::cvt(x[j]) - mean) * rstd;
            const float d = PxTraits<T>::cvt(dy[j]) * (pr.w ? pr.w[at + j] : 1.0f);
            s1 += d;
            s2 = __fmaf_rn(d, xh, s2);
        }
        const float2 t = block_sum(s1, s2);
        const float m1 = t.x / (float)pr.N, m2 = t.y / (float)pr.N;
        for (int64_t j = threadIdx.x; j < pr.N; j += kLongThreads) {
            const float xh = (PxTraits<T>::cvt(x[j]) - mean) * rstd;
            const float d = PxTraits<T>::cvt(dy[j]) * (pr.w ? pr.w[at + j] : 1.0f);
            const float v = rstd * (d - m1 - xh * m2);
            dx[j] = to_out<T>(v);
            chk = __fmaf_rn(v, 0.0f, chk);
        }
    }
    if (chk != chk) atomicOr(pr.status, kStatusNonFinite);
}

// The blocks' partial sums added up: lane = column, each warp every sixteenth partial in order,
// then the warps in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) reduce_kernel(const float* part, int parts, float* dw, float* db,
                                                                int64_t C) {
    __shared__ float acc[kSumWarps][32];
    follow_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // of 2 C columns
    float s = 0.0f;
    if (c < 2 * C)
#pragma unroll 4
        for (int q = warp; q < parts; q += kSumWarps) s += part[(int64_t)q * 2 * C + c];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * C) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) s += acc[w][lane];
        float* to = c < C ? dw : db;
        if (to) to[c < C ? c : c - C] = s;
    }
}

// ---- launches -------------------------------------------------------------------
// Partial sums of the columns that a backward call may use: at most this many, and at
// most about 16 MB of them (one at least).
constexpr int kMaxParts = 1184;
int64_t max_parts(int64_t M, int64_t C) {
    const int64_t fit = (int64_t(16) << 20) / (8 * C);
    return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(M, kMaxParts), fit));
}

namespace {

struct Plan {
    int vec, each;  // values per access and per thread; 0: rows of any length
    int most;  // threads that the kernel is compiled for
    int tpr, threads, pb, gpp, npc;
};

int pow2_at_least(int64_t n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// Values per thread: as many as a warp needs to hold the row, 8 to 64 of bfloat16 and 8 to 32
// of float32, so that short and middle rows need no block barrier (32768x3x2048 bfloat16, on earlier code:
// 152 us with 64 values and a warp per row, 270 with 8 and a block); past 8192 columns, where the weights in
// shared memory leave one block to an SM, 32 and so 512 threads (16384x1x16384 bfloat16 270 us; 437
// with 64 and 256 threads).  With few rows the smaller count leaves more threads to each of
// them.  The backward pass, which holds two column sums for each value, has 8, or 16 past 256
// columns (32768x3x2048 bfloat16: 249 us with 16, 289 with 8).  A row of 256 bytes or more needs no
// neighbours: the block's rows then share one parameter row.
Plan plan_of(int64_t M, int64_t P, int64_t N, int esz, bool by16, bool by4, bool forward, int sms) {
    Plan p{};
    p.vec = by16 ? 16 / esz : (esz == 2 && by4) ? 2 : 1;
    if (N > 16384) return Plan{};
    const int most = !forward ? 16 : esz == 2 && p.vec > 1 && N <= 8192 ? 64 : 32;
    p.each = 8;
    if (forward) {
        while (p.each < most && p.each * 32 < N && (double)M * P * N >= 768.0 * sms * p.each) p.each *= 2;
        while (p.each < most && p.each * 1024 < N) p.each *= 2;
    } else if (N > 256) {
        p.each = 16;
    }
    p.tpr = pow2_at_least((N + p.each - 1) / p.each);
    p.threads = p.most = std::max(p.tpr, 256);
    const int groups = p.threads / p.tpr;
    p.pb = N * esz >= 256 ? 1 : (int)std::min<int64_t>(P, groups);
    p.gpp = groups / p.pb;
    p.npc = (int)((P + p.pb - 1) / p.pb);
    return p;
}

// calls f with the values per access, the accesses per thread and the threads as types
template <typename T, bool kForward, class F>
void with_shape(const Plan& p, F f) {
#define PARARNN_LN(V, E, B) \
    if (p.vec == V && p.each == E && p.most == B)  \
        return f(std::integral_constant<int, V>{}, std::integral_constant<int, E / V>{}, std::integral_constant<int, B>{});
#define PARARNN_LN_ALL(V) \
    PARARNN_LN(V, 8, 256) PARARNN_LN(V, 16, 256) PARARNN_LN(V, 16, 512) PARARNN_LN(V, 16, 1024)          \
    if constexpr (kForward) {                                                                             \
        PARARNN_LN(V, 8, 512) PARARNN_LN(V, 8, 1024) PARARNN_LN(V, 32, 256) PARARNN_LN(V, 32, 512)        \
        if constexpr (sizeof(T) == 2 && V > 1) {                                                          \
            PARARNN_LN(V, 64, 256)                                                                        \
        }                                                                                                 \
    }
    constexpr int full = 16 / sizeof(T);
    PARARNN_LN_ALL(full)
    if constexpr (sizeof(T) == 2) {
        PARARNN_LN_ALL(2)
    }
    PARARNN_LN_ALL(1)
#undef PARARNN_LN_ALL
#undef PARARNN_LN
}

// Blocks: as many as are resident at `threads_per_sm` threads per SM, or as there are rows
// for; `slots` ranges of positions for each range of parameter rows.
int64_t slots_for(const Plan& p, int64_t M, int sms, int threads_per_sm) {
    const int64_t want = std::max<int64_t>(1, (int64_t)sms * (threads_per_sm / p.threads) / p.npc);
    return std::max<int64_t>(1, std::min<int64_t>(want, (M + p.gpp - 1) / p.gpp));
}

template <typename T>
pararnn_status launch_forward(const char* who, Params pr, cudaStream_t st) {
    const int sms = abi::sm_count();
    if (sms <= 0) return abi::cuda_fail(who, "device query failed");
    const bool by16 = (pr.N * sizeof(T)) % 16 == 0 && !abi::misaligned(pr.x, 16) && !abi::misaligned(pr.y, 16);
    const bool by4 = (pr.N * sizeof(T)) % 4 == 0 && !abi::misaligned(pr.x, 4) && !abi::misaligned(pr.y, 4);
    const Plan p = plan_of(pr.M, pr.P, pr.N, sizeof(T), by16, by4, true, sms);
    if (!p.vec) {
        return abi::launch(who, forward_long<T>, dim3((unsigned)std::min<int64_t>(pr.M * pr.P, sms * 4)), kLongThreads, 0,
                           st, 1, pr);
    }
    pr.tpr = p.tpr, pr.pb = p.pb, pr.gpp = p.gpp, pr.npc = p.npc;
    const int64_t blocks = slots_for(p, pr.M, sms, p.most == 256 ? 768 : p.most) * p.npc;
    pararnn_status s = PARARNN_EINVAL;
    with_shape<T, true>(p, [&](auto v, auto k, auto big) {
        constexpr int V = decltype(v)::value, K = decltype(k)::value, most = decltype(big)::value;
        auto kern = forward_rows<T, V, K, most>;
        constexpr int words = words_of<T, V, K>;
        constexpr size_t ring = kRing<T, V, K, most, true> ? (size_t)most * words * batch_of(words) * 4 : 0;
        const size_t smem = (p.each > 16 ? (size_t)p.tpr * p.each * 2 * sizeof(float) : 0) + ring;
        constexpr size_t largest = (V * K > 16 ? (size_t)most * V * K * 2 * sizeof(float) : 0) + ring;
        static std::atomic<uint64_t> done{0};
        s = abi::prepare_kernel(kern, largest, done)
                ? abi::launch(who, kern, dim3((unsigned)blocks), p.threads, smem, st, 1, pr)
                : abi::cuda_fail(who, "kernel attributes not accepted");
    });
    return s;
}

template <typename T>
pararnn_status launch_backward(const char* who, BwdParams pr, float* dw, float* db, cudaStream_t st) {
    const int sms = abi::sm_count();
    if (sms <= 0) return abi::cuda_fail(who, "device query failed");
    const int64_t C = pr.P * pr.N;
    const bool sums = dw || db;
    auto ok = [&](size_t a) {
        return (pr.N * sizeof(T)) % a == 0 && !abi::misaligned(pr.x, a) && !abi::misaligned(pr.dy, a) &&
               !abi::misaligned(pr.dx, a);
    };
    const Plan p = plan_of(pr.M, pr.P, pr.N, sizeof(T), ok(16), ok(4), false, sms);
    if (!sums) pr.part = nullptr;
    int64_t parts;
    pararnn_status s = PARARNN_OK;
    if (!p.vec) {
        parts = std::min<int64_t>(max_parts(pr.M, C), 64);
        const dim3 cols((unsigned)((C + kLongThreads - 1) / kLongThreads), (unsigned)parts);
        if (sums) s = abi::launch(who, columns_long<T>, cols, kLongThreads, 0, st, 1, pr);
        if (s == PARARNN_OK)
            s = abi::launch(who, dx_long<T>, dim3((unsigned)std::min<int64_t>(pr.M * pr.P, sms * 4)), kLongThreads, 0, st,
                            1, pr);
    } else {
        pr.tpr = p.tpr, pr.pb = p.pb, pr.gpp = p.gpp, pr.npc = p.npc;
        parts = slots_for(p, pr.M, sms, p.most == 256 ? 512 : p.most);
        if (sums) parts = std::min<int64_t>(parts, max_parts(pr.M, C));
        with_shape<T, false>(p, [&](auto v, auto k, auto big) {
            constexpr int V = decltype(v)::value, K = decltype(k)::value, most = decltype(big)::value;
            auto kern = backward_rows<T, V, K, most>;
            constexpr size_t ring =
                kRing<T, V, K, most, false> ? (size_t)most * words_of<T, V, K> * kBackRows<T, V, K, most> * 8 : 0;
            constexpr size_t columns = (size_t)V * K * most * sizeof(float2);
            const size_t smem = sums ? std::max(columns, ring) : ring;
            static std::atomic<uint64_t> done{0};
            if (!abi::prepare_kernel(kern, std::max(columns, ring), done)) {
                s = abi::cuda_fail(who, "kernel attributes not accepted");
                return;
            }
            s = abi::launch(who, kern, dim3((unsigned)(parts * p.npc)), p.threads, smem, st, 1, pr);
        });
    }
    if (s != PARARNN_OK || !sums) return s;
    return abi::launch(who, reduce_kernel, dim3((unsigned)((2 * C + 31) / 32)), kSumWarps * 32, 0, st, 1,
                       (const float*)pr.part, (int)parts, dw, db, C);
}

}  // namespace

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
    return kHeaderBytes + (size_t)(ln::max_parts(M, P * N) * P * N) * 2 * sizeof(float);
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
    return dtype == PARARNN_F32 ? ln::launch_forward<float>(who, pr, st) : ln::launch_forward<ln::bf16>(who, pr, st);
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
    return dtype == PARARNN_F32 ? ln::launch_backward<float>(who, pr, dL_dweight, dL_dbias, st)
                                : ln::launch_backward<ln::bf16>(who, pr, dL_dweight, dL_dbias, st);
}

}  // extern "C"
