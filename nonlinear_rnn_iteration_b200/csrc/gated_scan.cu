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

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "abi_util.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "pararnn_b200.h"
#include "tma.cuh"

namespace pararnn {
// pararnn_abi.cu: a tensor map over (B, T, inner, D), box (1, rows, gates, W), zero fill outside
pararnn_status encode_steps_map(CUtensorMap* map, const void* base, bool bf16, int64_t D, int inner, int64_t T, int64_t B,
                                int W, int gates, int rows);

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
    int64_t nCG, nCk;  // channel groups; checkpoints per batch row
    int ranks;         // blocks per cluster
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
    float* part;  // (B * ranks, D)
    float* dh0;   // (B,D) or null
    unsigned* status;
    int64_t B, T, D;
    int64_t nCG, nCk;
    int ranks;
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

// ---- forward ------------------------------------------------------------------
// A block owns 64 channels of one batch row and walks T in tiles of L steps; with
// few channels a cluster of up to 16 blocks takes that many neighbouring tiles
// at once.  Lane l of every warp holds channels 2l, 2l+1, and warp w holds R consecutive
// steps of the tile, so a warp's scan needs no shuffles: each thread evaluates its R steps
// into registers (a_t, u_t), composes them into (prod a, B), and the warps' totals
// meet in shared memory.  With a cluster each block writes its tile's element into
// every block's shared memory, one cluster barrier per tile, and every block
// forms the state after all of the cluster's tiles itself.  Then each
// thread walks its R steps from the state before them and stores H.  Every
// pre-activation is read once, by tensor copies two tiles ahead.
constexpr int kW = 64;  // channels per block
constexpr int kNW = 8;  // warps per block
constexpr int kMaxRanks = 16;
constexpr int kStages = 2;
constexpr uint64_t kWaitNs = 2000000000ull;

template <typename T>
struct Tile {
    static constexpr int R = Ck<T>::kSteps;
    static constexpr int L = kNW * R;
    static constexpr uint32_t kBytes = (uint32_t)(L * 3 * kW * sizeof(T));
};

// an affine map h -> P h + B of two channels
struct Elem {
    f2 P, B;
};
struct alignas(16) Totals {
    float P[kW], B[kW];
};

template <typename T>
struct FwdSmem {
    alignas(128) T px[kStages][Tile<T>::L][3][kW];
    Totals warp[2][kNW];         // each warp's element, two tiles in turn
    Totals rank[2][kMaxRanks];   // each of the cluster's tiles, two rounds in turn
    unsigned warp_new[2][kNW];   // whether a marked step lies in the warp's steps
    unsigned rank_new[2][kMaxRanks];
    uint64_t bar[kStages];
};

__device__ __forceinline__ f2 ld2(const float* p) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    return f2{v.x, v.y};
}
__device__ __forceinline__ f2 ld2(const bf16* p) {
    const unsigned v = *reinterpret_cast<const unsigned*>(p);
    return f2{__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
}
__device__ __forceinline__ void st2(float* p, f2 v) { *reinterpret_cast<float2*>(p) = make_float2(v.x, v.y); }
__device__ __forceinline__ void st2(bf16* p, f2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}

__device__ __forceinline__ void st2_cluster(float* local, uint32_t rank, f2 v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st1_cluster(unsigned* local, uint32_t rank, unsigned v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}

// the box of L steps and all gates of 64 channels of one batch row
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// waits for a staged tile; after one wait that ran out of time the others are short
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity, bool& late) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns(), limit = late ? 1000000ull : kWaitNs;
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit) {
            late = true;
            return false;
        }
    return true;
}

// Two channels' decay a, and m = 1 - a, from z = y / 2 (kWide false: every y < 1):
// m(z) = z (1 - z/2 + z^2/6 - ...) to z^8 / 8! (the next term is below 1.1e-8 of
// it at z = 1/2), then 1 - e^-2z = m(z) (2 - m(z)).  kWide: y >= 1/2 takes the exponential as in
// decay_of.
template <bool kWide>
__device__ __forceinline__ void decay2(f2 z, f2& a, f2& m) {
    f2 s = fma2(z, splat2(-1.0f / 40320.0f), splat2(1.0f / 5040.0f));
    s = fma2(z, s, splat2(-1.0f / 720.0f));
    s = fma2(z, s, splat2(1.0f / 120.0f));
    s = fma2(z, s, splat2(-1.0f / 24.0f));
    s = fma2(z, s, splat2(1.0f / 6.0f));
    s = fma2(z, s, splat2(-0.5f));
    s = fma2(z, s, splat2(1.0f));
    s = mul2(z, s);
    m = mul2(s, sub2(splat2(2.0f), s));
    a = sub2(splat2(1.0f), m);
    if constexpr (kWide) {
        const f2 e = ex2_2(mul2(z, splat2(-2.0f * kLog2e)));
        if (z.x >= 0.25f) a.x = e.x, m.x = 1.0f - e.x;
        if (z.y >= 0.25f) a.y = e.y, m.y = 1.0f - e.y;
    }
}

// a and u = sqrt(1 - a^2) sig(p_i) x.  With v = 1 - a^2 and d = 1 + e^{-p_i},
// u = x v / sqrt(v d^2): one reciprocal square root for the root and the
// gate's reciprocal.  d is capped at 2^62 so that d^2 stays finite, and 2^-123
// keeps the root's argument above zero where v = 0.
template <bool kWide>
__device__ __forceinline__ void eval2(f2 pr, f2 pi, f2 x, f2 khalf, f2& a, f2& u) {
    const f2 z = mul2(khalf, sigmoid2(pr));
    f2 m;
    decay2<kWide>(z, a, m);
    const f2 v = mul2(m, sub2(splat2(2.0f), m));
    const f2 d = sig_den2(pi);
    const f2 q = fma2(mul2(v, d), d, splat2(9.4e-38f));
    u = mul2(mul2(x, v), f2{rsqrt_approx(q.x), rsqrt_approx(q.y)});
}

template <typename T, bool kTma, bool kCluster>
__global__ void __launch_bounds__(kNW * 32, 2) forward_kernel(const Params pr, const __grid_constant__ CUtensorMap map) {
    constexpr int R = Tile<T>::R, L = Tile<T>::L;
    extern __shared__ unsigned char raw[];
    FwdSmem<T>& sm = *reinterpret_cast<FwdSmem<T>*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = kCluster ? cluster_ctarank() : 0u;
    const int C = kCluster ? pr.ranks : 1;
    const int64_t group = (int64_t)blockIdx.x / C;
    const int64_t b = group / pr.nCG;
    const int d0 = (int)(group - b * pr.nCG) * kW, d = d0 + 2 * lane;
    const bool in0 = d < pr.D, in1 = d + 1 < pr.D;
    const int64_t row0 = b * pr.T;  // the batch row's first step in (B T)
    const int tiles = (int)((pr.T + L - 1) / L), rounds = (tiles + C - 1) / C;
    const T* px = static_cast<const T*>(pr.px) + row0 * 3 * pr.D;
    T* H = static_cast<T*>(pr.H) + row0 * pr.D + d;

    if (kTma && tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&sm.bar[i], 1);
        mbar_fence_init();
    }
    f2 khalf{0.0f, 0.0f}, carry{0.0f, 0.0f};
    if (in0) khalf.x = 0.5f * pr.decay * softplus_f(pr.lam[d]);
    if (in1) khalf.y = 0.5f * pr.decay * softplus_f(pr.lam[d + 1]);
    if (pr.h0 && in0) carry.x = pr.h0[b * pr.D + d];
    if (pr.h0 && in1) carry.y = pr.h0[b * pr.D + d + 1];
    const bool wide = __any_sync(0xffffffffu, !(khalf.x <= 0.5f && khalf.y <= 0.5f));
    // every block has begun, and has read h0 (h_last may be the same buffer), before a peer writes
    if constexpr (kCluster) {
        cluster_arrive_release();
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    auto issue = [&](int round) {
        const int t0 = (round * C + (int)rank) * L;
        if (round < rounds && t0 < pr.T) {
            uint64_t* bar = &sm.bar[round % kStages];
            mbar_arrive_expect_tx(bar, Tile<T>::kBytes);
            tma_load_4d(sm.px[round % kStages], &map, bar, d0, 0, t0, (int)b);
        }
    };
    if (kTma && tid == 0)
        for (int i = 0; i < kStages; ++i) issue(i);
    // lane j of a warp reads the mark of the warp's step j, a round ahead
    auto marks_of = [&](int round) -> unsigned {
        const int64_t t = (int64_t)(round * C + (int)rank) * L + warp * R + lane;
        return (pr.reset && lane < R && round < rounds && t < pr.T) ? pr.reset[row0 + t] : 0u;
    };
    unsigned mark = marks_of(0);
    bool late = false, timeout = false;
    f2 chk{0.0f, 0.0f};  // becomes NaN once a state is not finite

    for (int round = 0; round < rounds; ++round) {
        const int par = round & 1, st = round % kStages;
        const int tile0 = (round * C + (int)rank) * L;  // may be past T
        const int t0 = tile0 + warp * R;
        const unsigned marks = __ballot_sync(0xffffffffu, mark != 0);
        mark = marks_of(round + 1);
        f2 a[R], u[R];
        const bool live = tile0 < pr.T;
        if (live) {
            if constexpr (kTma) {
                timeout |= !wait_stage(&sm.bar[st], (round / kStages) & 1, late);
            } else {
                for (int i = tid; i < L * 3 * kW; i += kNW * 32) {
                    const int row = i / (3 * kW), g = (i / kW) % 3, c = i % kW;
                    const int64_t t = tile0 + row;
                    sm.px[0][row][g][c] = (t < pr.T && d0 + c < pr.D) ? px[(t * 3 + g) * pr.D + d0 + c] : T(0.0f);
                }
                __syncthreads();
            }
        }
        if (live && t0 < pr.T) {
            const T* p = &sm.px[kTma ? st : 0][warp * R][0][2 * lane];
            if (wide) {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    eval2<true>(ld2(p + j * 3 * kW), ld2(p + (j * 3 + 1) * kW), ld2(p + (j * 3 + 2) * kW), khalf, a[j], u[j]);
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    eval2<false>(ld2(p + j * 3 * kW), ld2(p + (j * 3 + 1) * kW), ld2(p + (j * 3 + 2) * kW), khalf, a[j], u[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j) a[j] = splat2(1.0f), u[j] = splat2(0.0f);
        }
        Elem e{a[0], u[0]};
        if (marks == 0) {
#pragma unroll
            for (int j = 1; j < R; ++j) {
                e.B = fma2(a[j], e.B, u[j]);
                e.P = mul2(a[j], e.P);
            }
        } else {
#pragma unroll
            for (int j = 1; j < R; ++j) e.B = (marks >> j & 1) ? u[j] : fma2(a[j], e.B, u[j]);
        }
        st2(&sm.warp[par][warp].P[2 * lane], e.P);
        st2(&sm.warp[par][warp].B[2 * lane], e.B);
        if (lane == 0) sm.warp_new[par][warp] = marks;
        __syncthreads();
        if (kTma && tid == 0) issue(round + kStages);

        f2 h;
        if constexpr (kCluster) {
            // the element of the warps before this one, and of the whole tile
            Elem pre{splat2(1.0f), splat2(0.0f)}, all = pre;
            unsigned pre_new = 0, all_new = 0;
#pragma unroll
            for (int w = 0; w < kNW; ++w) {
                if (w == warp) pre = all, pre_new = all_new;
                const f2 P = ld2(&sm.warp[par][w].P[2 * lane]), B = ld2(&sm.warp[par][w].B[2 * lane]);
                const unsigned nw = sm.warp_new[par][w];
                all.B = nw ? B : fma2(P, all.B, B);
                all.P = mul2(P, all.P);
                all_new |= nw;
            }
            for (int r = warp; r < C; r += kNW) {
                st2_cluster(&sm.rank[par][rank].P[2 * lane], r, all.P);
                st2_cluster(&sm.rank[par][rank].B[2 * lane], r, all.B);
                if (lane == 0) st1_cluster(&sm.rank_new[par][rank], r, all_new);
            }
            cluster_arrive_release();
            cluster_wait_acquire();
            f2 c = carry, mine = carry;
            for (int r = 0; r < C; ++r) {
                if (r == (int)rank) mine = c;
                const f2 P = ld2(&sm.rank[par][r].P[2 * lane]), B = ld2(&sm.rank[par][r].B[2 * lane]);
                c = sm.rank_new[par][r] ? B : fma2(P, c, B);
            }
            carry = c;
            h = pre_new ? pre.B : fma2(pre.P, mine, pre.B);
        } else {
            f2 c = carry;
            h = carry;
#pragma unroll
            for (int w = 0; w < kNW; ++w) {
                if (w == warp) h = c;
                const f2 P = ld2(&sm.warp[par][w].P[2 * lane]), B = ld2(&sm.warp[par][w].B[2 * lane]);
                c = sm.warp_new[par][w] ? B : fma2(P, c, B);
            }
            carry = c;
        }
        if (t0 >= pr.T) continue;
        if (pr.ck) {
            float* o = pr.ck + (b * pr.nCk + t0 / R) * pr.D + d;
            if (in0) o[0] = h.x;
            if (in1) o[1] = h.y;
        }
        T* o = H + (int64_t)t0 * pr.D;
        const int n = (int)min((int64_t)R, pr.T - t0);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (j < n) {
                h = (marks >> j & 1) ? u[j] : fma2(a[j], h, u[j]);
                chk = fma2(h, splat2(0.0f), chk);
                if constexpr (kTma) {
                    if (in0) st2(o, h);
                } else {
                    if (in0) o[0] = to_out<T>(h.x);
                    if (in1) o[1] = to_out<T>(h.y);
                }
            }
            o += pr.D;
        }
        if (pr.last && t0 + n == pr.T) {
            float* q = pr.last + b * pr.D + d;
            if (in0) q[0] = h.x;
            if (in1) q[1] = h.y;
        }
    }
    if (pr.status) {
        const bool bad = (in0 && chk.x != chk.x) || (in1 && chk.y != chk.y);
        const unsigned bits = (__any_sync(0xffffffffu, bad) ? kStatusNonFinite : 0u) |
                              (__any_sync(0xffffffffu, timeout) ? kStatusTimeout : 0u);
        if (bits && lane == 0) atomicOr(pr.status, bits);
    }
}

// ---- adjoint --------------------------------------------------------------------
// The forward's tiles in reversed time.  The scan runs on mu_t = a_t l_t, l_t =
// g_t + mu_{t+1}, whose elements need p_r and g only: pass 1 forms z = y / 2
// and the element of each thread's R steps and frees those arrays' stage.
// With the carry, each thread walks its steps backwards for l, then
// forwards from the checkpoint, the state before its first step, for h_{t-1} and
// the gradients: no state is read but one in R, and the forward's
// scan is not repeated.  p_r and g have one stage, p_i and x two, so that the
// next tile's copies all start after pass 1; 96 KB a block, two blocks per SM.
template <typename T>
struct BwdSmem {
    alignas(128) T pr[Tile<T>::L][kW];
    alignas(128) T g[Tile<T>::L][kW];
    alignas(128) T ix[kStages][Tile<T>::L][2][kW];
    Totals warp[2][kNW];
    Totals rank[2][kMaxRanks];
    unsigned warp_new[2][kNW];
    unsigned rank_new[2][kMaxRanks];
    float sum[kNW][kW];
    uint64_t bar_a, bar_b[kStages];
};

struct BwdMaps {
    CUtensorMap pr, ix, g;  // boxes of one gate, of two gates, and of dL/dH
};

// the gradients of one step of two channels; h is h_{t-1} in and h_t out
template <bool kWide>
__device__ __forceinline__ void grads2(f2 z, f2 l, f2 pi, f2 x, f2 kinv, bool first, f2& h, f2& dpr, f2& dpi, f2& dx, f2& w) {
    f2 a, m;
    decay2<kWide>(z, a, m);
    const f2 v = mul2(m, sub2(splat2(2.0f), m));
    // 1 / b; the addend keeps the root's argument above zero, and where v = 0 so is z, which scales the result
    const f2 va = add2(v, splat2(1e-37f));
    const f2 rs{rsqrt_approx(va.x), rsqrt_approx(va.y)};
    const f2 i = rcp_2(sig_den2(pi));
    const f2 ib = mul2(rs, i);          // i / b
    const f2 bi = mul2(v, ib);          // b i
    const f2 e = mul2(ib, x);           // i x / b
    if (first) h = splat2(0.0f);
    const f2 ah = mul2(a, h);
    dx = mul2(l, bi);
    dpi = mul2(mul2(dx, x), sub2(splat2(1.0f), i));
    w = mul2(mul2(add2(z, z), l), sub2(mul2(mul2(a, a), e), ah));
    dpr = mul2(w, sub2(splat2(1.0f), mul2(z, kinv)));
    h = fma2(v, e, ah);
}

template <typename T, bool kTma, bool kCluster>
__global__ void __launch_bounds__(kNW * 32, 2) backward_kernel(const BwdParams pr, const __grid_constant__ BwdMaps maps) {
    constexpr int R = Tile<T>::R, L = Tile<T>::L;
    extern __shared__ unsigned char raw[];
    BwdSmem<T>& sm = *reinterpret_cast<BwdSmem<T>*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = kCluster ? cluster_ctarank() : 0u;
    const int C = kCluster ? pr.ranks : 1;
    const int64_t group = (int64_t)blockIdx.x / C;
    const int64_t b = group / pr.nCG;
    const int d0 = (int)(group - b * pr.nCG) * kW, d = d0 + 2 * lane;
    const bool in0 = d < pr.D, in1 = d + 1 < pr.D;
    const int64_t row0 = b * pr.T;
    const int tiles = (int)((pr.T + L - 1) / L), rounds = (tiles + C - 1) / C;
    const T* px = static_cast<const T*>(pr.px) + row0 * 3 * pr.D;
    const T* dH = static_cast<const T*>(pr.dH) + row0 * pr.D;
    T* dpx = static_cast<T*>(pr.dpx) + row0 * 3 * pr.D + d;

    if (kTma && tid == 0) {
        mbar_init(&sm.bar_a, 1);
        for (int i = 0; i < kStages; ++i) mbar_init(&sm.bar_b[i], 1);
        mbar_fence_init();
    }
    f2 khalf{0.0f, 0.0f}, carry{0.0f, 0.0f};
    if (in0) khalf.x = 0.5f * pr.decay * softplus_f(pr.lam[d]);
    if (in1) khalf.y = 0.5f * pr.decay * softplus_f(pr.lam[d + 1]);
    if (pr.dlast && in0) carry.x = pr.dlast[b * pr.D + d];
    if (pr.dlast && in1) carry.y = pr.dlast[b * pr.D + d + 1];
    // r = z / khalf; a khalf this small gives no gradient to p_r (w is below 2^-60 l)
    const f2 kinv{khalf.x > 1e-37f ? 1.0f / khalf.x : 0.0f, khalf.y > 1e-37f ? 1.0f / khalf.y : 0.0f};
    const bool wide = __any_sync(0xffffffffu, !(khalf.x <= 0.5f && khalf.y <= 0.5f));
    if constexpr (kCluster) {
        cluster_arrive_release();
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    // round q takes the cluster's tiles from the last ones on; only round 0 may have tiles past T
    auto tile_of = [&](int q) { return (rounds - 1 - q) * C + (int)rank; };
    const int q0 = tile_of(0) < tiles ? 0 : 1;
    auto issue = [&](int q) {
        if (q >= rounds) return;
        const int t0 = tile_of(q) * L, sb = (q - q0) % kStages;
        mbar_arrive_expect_tx(&sm.bar_a, (uint32_t)(L * 2 * kW * sizeof(T)));
        tma_load_4d(sm.pr, &maps.pr, &sm.bar_a, d0, 0, t0, (int)b);
        tma_load_4d(sm.g, &maps.g, &sm.bar_a, d0, 0, t0, (int)b);
        mbar_arrive_expect_tx(&sm.bar_b[sb], (uint32_t)(L * 2 * kW * sizeof(T)));
        tma_load_4d(sm.ix[sb], &maps.ix, &sm.bar_b[sb], d0, 1, t0, (int)b);
    };
    if (kTma && tid == 0) issue(q0);
    auto marks_of = [&](int q) -> unsigned {
        if (q >= rounds) return 0u;
        const int64_t t = (int64_t)tile_of(q) * L + warp * R + lane;
        return (pr.reset && lane < R && t < pr.T) ? pr.reset[row0 + t] : 0u;
    };
    unsigned mark = marks_of(0);
    bool late = false, timeout = false;
    f2 chk{0.0f, 0.0f}, sum{0.0f, 0.0f};

    for (int q = 0; q < rounds; ++q) {
        const int par = q & 1, n_in = q - q0, sb = kTma ? n_in % kStages : 0;
        const int tile0 = tile_of(q) * L, t0 = tile0 + warp * R;
        const unsigned marks = __ballot_sync(0xffffffffu, mark != 0);
        mark = marks_of(q + 1);
        const bool live = q >= q0;
        const int n = live ? (int)max((int64_t)0, min((int64_t)R, pr.T - t0)) : 0;  // this warp's steps
        if (live) {
            if constexpr (kTma) {
                timeout |= !wait_stage(&sm.bar_a, n_in & 1, late);
            } else {
                __syncthreads();  // the tile before has been read
                for (int i = tid; i < L * 4 * kW; i += kNW * 32) {
                    const int row = i / (4 * kW), g = (i / kW) % 4, c = i % kW;
                    const int64_t t = tile0 + row;
                    T val = T(0.0f);
                    if (t < pr.T && d0 + c < pr.D) val = g < 3 ? px[(t * 3 + g) * pr.D + d0 + c] : dH[t * pr.D + d0 + c];
                    T* to = g == 0 ? &sm.pr[row][c] : g == 3 ? &sm.g[row][c] : &sm.ix[0][row][g - 1][c];
                    *to = val;
                }
                __syncthreads();
            }
        }
        // pass 1: z, g and the element of mu over the warp's steps
        f2 z[R], l[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            z[j] = l[j] = splat2(0.0f);
            if (j < n) {
                z[j] = mul2(khalf, sigmoid2(ld2(&sm.pr[warp * R + j][2 * lane])));
                l[j] = ld2(&sm.g[warp * R + j][2 * lane]);
            }
        }
        Elem e{splat2(1.0f), splat2(0.0f)};
        auto compose = [&](auto w) {
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                f2 a, m;
                decay2<decltype(w)::value>(z[j], a, m);
                e.B = mul2(a, add2(l[j], e.B));
                e.P = mul2(a, e.P);
                if (marks >> j & 1) e.B = splat2(0.0f);
            }
        };
        if (wide)
            compose(std::true_type{});
        else
            compose(std::false_type{});
        st2(&sm.warp[par][warp].P[2 * lane], e.P);
        st2(&sm.warp[par][warp].B[2 * lane], e.B);
        if (lane == 0) sm.warp_new[par][warp] = marks;
        __syncthreads();
        if (kTma && live && tid == 0) issue(q + 1);

        f2 mu;
        if constexpr (kCluster) {
            Elem pre{splat2(1.0f), splat2(0.0f)}, all = pre;
            unsigned pre_new = 0, all_new = 0;
#pragma unroll
            for (int w = kNW - 1; w >= 0; --w) {
                if (w == warp) pre = all, pre_new = all_new;
                const f2 P = ld2(&sm.warp[par][w].P[2 * lane]), B = ld2(&sm.warp[par][w].B[2 * lane]);
                const unsigned nw = sm.warp_new[par][w];
                all.B = nw ? B : fma2(P, all.B, B);
                all.P = mul2(P, all.P);
                all_new |= nw;
            }
            for (int r = warp; r < C; r += kNW) {
                st2_cluster(&sm.rank[par][rank].P[2 * lane], r, all.P);
                st2_cluster(&sm.rank[par][rank].B[2 * lane], r, all.B);
                if (lane == 0) st1_cluster(&sm.rank_new[par][rank], r, all_new);
            }
            cluster_arrive_release();
            cluster_wait_acquire();
            f2 c = carry, mine = carry;
            for (int r = C - 1; r >= 0; --r) {
                if (r == (int)rank) mine = c;
                const f2 P = ld2(&sm.rank[par][r].P[2 * lane]), B = ld2(&sm.rank[par][r].B[2 * lane]);
                c = sm.rank_new[par][r] ? B : fma2(P, c, B);
            }
            carry = c;
            mu = pre_new ? pre.B : fma2(pre.P, mine, pre.B);
        } else {
            f2 c = carry;
            mu = carry;
#pragma unroll
            for (int w = kNW - 1; w >= 0; --w) {
                if (w == warp) mu = c;
                const f2 P = ld2(&sm.warp[par][w].P[2 * lane]), B = ld2(&sm.warp[par][w].B[2 * lane]);
                c = sm.warp_new[par][w] ? B : fma2(P, c, B);
            }
            carry = c;
        }
        if (kTma && live) timeout |= !wait_stage(&sm.bar_b[sb], (n_in / kStages) & 1, late);
        if (n == 0) continue;
        // pass 2: l backwards, then the gradients forwards from the checkpoint
        f2 h{0.0f, 0.0f};
        const float* ck = pr.ck + (b * pr.nCk + t0 / R) * pr.D + d;
        if (in0) h.x = ck[0];
        if (in1) h.y = ck[1];
        T* o = dpx + (int64_t)t0 * 3 * pr.D;
        f2 part{0.0f, 0.0f};
        auto finish = [&](auto w) {
            constexpr bool kWide = decltype(w)::value;
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                f2 a, m;
                decay2<kWide>(z[j], a, m);
                l[j] = add2(l[j], mu);
                mu = mul2(a, l[j]);
                if (marks >> j & 1) mu = splat2(0.0f);
            }
            const T* s = &sm.ix[sb][warp * R][0][2 * lane];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (j < n) {
                    // evaluated again from z: a and m of all R steps would not stay in registers
                    asm volatile("" : "+f"(z[j].x), "+f"(z[j].y));
                    f2 dpr, dpi, dx, ww;
                    grads2<kWide>(z[j], l[j], ld2(s + j * 2 * kW), ld2(s + (j * 2 + 1) * kW), kinv, marks >> j & 1, h, dpr,
                                  dpi, dx, ww);
                    part = add2(part, ww);
                    chk = fma2(dx, splat2(0.0f), chk);
                    if constexpr (kTma) {
                        if (in0) {
                            st2(o, dpr);
                            st2(o + pr.D, dpi);
                            st2(o + 2 * pr.D, dx);
                        }
                    } else {
                        if (in0) o[0] = to_out<T>(dpr.x), o[pr.D] = to_out<T>(dpi.x), o[2 * pr.D] = to_out<T>(dx.x);
                        if (in1) o[1] = to_out<T>(dpr.y), o[pr.D + 1] = to_out<T>(dpi.y), o[2 * pr.D + 1] = to_out<T>(dx.y);
                    }
                }
                o += 3 * pr.D;
            }
        };
        if (wide)
            finish(std::true_type{});
        else
            finish(std::false_type{});
        sum = add2(sum, part);
        if (t0 == 0 && pr.dh0) {
            float* q = pr.dh0 + b * pr.D + d;
            if (in0) q[0] = mu.x;
            if (in1) q[1] = mu.y;
        }
    }
    // the warps' sums of w in order; a sum that is not finite stands for a dL/dp_r that is not
    st2(&sm.sum[warp][2 * lane], sum);
    __syncthreads();
    if (tid < kW && d0 + tid < pr.D) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) s += sm.sum[w][tid];
        pr.part[(b * C + rank) * pr.D + d0 + tid] = s;
    }
    chk = fma2(sum, splat2(0.0f), chk);
    const bool bad = (in0 && chk.x != chk.x) || (in1 && chk.y != chk.y);
    const unsigned bits = (__any_sync(0xffffffffu, bad) ? kStatusNonFinite : 0u) |
                          (__any_sync(0xffffffffu, timeout) ? kStatusTimeout : 0u);
    if (bits && lane == 0) atomicOr(pr.status, bits);
}

// dL/dlambda = sig(lambda) / softplus(lambda) * the sum of the blocks' partial
// sums: lane = channel, each warp every sixteenth row in order, then the warps in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) dlam_kernel(const float* part, const float* lam, float* dlam, int64_t rows,
                                                              int64_t D) {
    __shared__ float acc[kSumWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t d = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (d < D)
#pragma unroll 4
        for (int64_t r = warp; r < rows; r += kSumWarps) s += part[r * D + d];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && d < D) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) s += acc[w][lane];
        const float l = lam[d];
        // softplus(l) is sig(l) to within e^l for very negative l
        const float ratio = l < -20.0f ? 1.0f : 1.0f / ((1.0f + expf(-l)) * softplus_f(l));
        dlam[d] = ratio * s;
    }
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
    return B < 0 || T < 0 || D < 0 || B >= (int64_t(1) << 31) || T > (int64_t(1) << 30) || B * T >= (int64_t(1) << 31) ||
           D >= (int64_t(1) << 31) || (double)B * T * D > 4.0e12 || (double)B * D > 1.0e11;
}
int64_t n_checkpoints(int64_t T, pararnn_dtype dt) {
    const int s = dt == PARARNN_F32 ? Ck<float>::kSteps : Ck<bf16>::kSteps;
    return (T + s - 1) / s;
}

// ---- launches -------------------------------------------------------------------
// Blocks per cluster: the smallest power of two that fills the device's SMs twice
// (two blocks are resident per SM), as far as there are tiles for them.
int ranks_for(int64_t groups, int64_t tiles, int sms) {
    int c = 1;
    while (c < kMaxRanks && c < tiles && groups * c * 2 <= 2 * (int64_t)sms) c *= 2;
    return c;
}

// A kernel's attributes are set once per device; `done` holds a bit per device.
template <class Kern>
bool prepare_kernel(Kern kern, size_t smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

int sm_count() {
    static thread_local int dev_of = -1, sms = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev != dev_of) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        dev_of = dev;
    }
    return sms;
}

template <auto kern, class P, class Map>
pararnn_status launch_clusters(const char* who, const P& pr, const Map& map, int64_t blocks, int ranks,
                               size_t smem, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (!prepare_kernel(kern, smem, done)) return abi::cuda_fail(who, "kernel attributes not accepted");
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(kNW * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ranks;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, pr, map) == cudaSuccess ? PARARNN_OK
                                                                  : abi::cuda_fail(who, "kernel launch failed");
}

template <typename T>
pararnn_status launch_backward(const char* who, BwdParams pr, float* dlam, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return abi::cuda_fail(who, "device query failed");
    constexpr int L = Tile<T>::L;
    pr.nCG = (pr.D + kW - 1) / kW;
    pr.nCk = n_checkpoints(pr.T, sizeof(T) == 4 ? PARARNN_F32 : PARARNN_BF16);
    const int64_t groups = pr.B * pr.nCG, tiles = (pr.T + L - 1) / L;
    pr.ranks = ranks_for(groups, tiles, sms);
    if (groups * pr.ranks >= (int64_t(1) << 31)) return abi::fail(who, "too many channel groups");
    const bool tma = (pr.D * sizeof(T)) % 16 == 0 && !abi::misaligned(pr.px, 16) && !abi::misaligned(pr.dH, 16) &&
                     !abi::misaligned(pr.dpx, 16);
    BwdMaps maps;
    memset(&maps, 0, sizeof maps);
    if (tma) {
        const bool bf = sizeof(T) == 2;
        pararnn_status s = encode_steps_map(&maps.pr, pr.px, bf, pr.D, 3, pr.T, pr.B, kW, 1, L);
        if (s == PARARNN_OK) s = encode_steps_map(&maps.ix, pr.px, bf, pr.D, 3, pr.T, pr.B, kW, 2, L);
        if (s == PARARNN_OK) s = encode_steps_map(&maps.g, pr.dH, bf, pr.D, 1, pr.T, pr.B, kW, 1, L);
        if (s != PARARNN_OK) return s;
    }
    const size_t smem = sizeof(BwdSmem<T>) + 128;
    const int64_t blocks = groups * pr.ranks;
    pararnn_status s;
    if (pr.ranks > 1)
        s = tma ? launch_clusters<backward_kernel<T, true, true>>(who, pr, maps, blocks, pr.ranks, smem, st)
                : launch_clusters<backward_kernel<T, false, true>>(who, pr, maps, blocks, pr.ranks, smem, st);
    else
        s = tma ? launch_clusters<backward_kernel<T, true, false>>(who, pr, maps, blocks, 1, smem, st)
                : launch_clusters<backward_kernel<T, false, false>>(who, pr, maps, blocks, 1, smem, st);
    if (s != PARARNN_OK || !dlam) return s;
    dlam_kernel<<<(unsigned)((pr.D + 31) / 32), kSumWarps * 32, 0, st>>>(pr.part, pr.lam, dlam, pr.B * pr.ranks, pr.D);
    return abi::launched(who);
}

template <typename T>
pararnn_status launch_forward(const char* who, Params pr, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return abi::cuda_fail(who, "device query failed");
    pr.nCG = (pr.D + kW - 1) / kW;
    pr.nCk = n_checkpoints(pr.T, sizeof(T) == 4 ? PARARNN_F32 : PARARNN_BF16);
    const int64_t groups = pr.B * pr.nCG, tiles = (pr.T + Tile<T>::L - 1) / Tile<T>::L;
    pr.ranks = ranks_for(groups, tiles, sms);
    if (groups * pr.ranks >= (int64_t(1) << 31)) return abi::fail(who, "too many channel groups");
    const bool tma = (pr.D * sizeof(T)) % 16 == 0 && !abi::misaligned(pr.px, 16) && !abi::misaligned(pr.H, 16);
    CUtensorMap map;
    memset(&map, 0, sizeof map);
    if (tma) {
        const pararnn_status s = encode_steps_map(&map, pr.px, sizeof(T) == 2, pr.D, 3, pr.T, pr.B, kW, 3, Tile<T>::L);
        if (s != PARARNN_OK) return s;
    }
    const size_t smem = sizeof(FwdSmem<T>) + 128;
    const int64_t blocks = groups * pr.ranks;
    if (pr.ranks > 1)
        return tma ? launch_clusters<forward_kernel<T, true, true>>(who, pr, map, blocks, pr.ranks, smem, st)
                   : launch_clusters<forward_kernel<T, false, true>>(who, pr, map, blocks, pr.ranks, smem, st);
    return tma ? launch_clusters<forward_kernel<T, true, false>>(who, pr, map, blocks, 1, smem, st)
               : launch_clusters<forward_kernel<T, false, false>>(who, pr, map, blocks, 1, smem, st);
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
    // a partial sum of dL/dlambda from each block of a cluster of up to 16
    return kHeaderBytes + (size_t)(B * D) * gs::kMaxRanks * sizeof(float);
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
    return dtype == PARARNN_F32 ? gs::launch_forward<float>(who, pr, st) : gs::launch_forward<gs::bf16>(who, pr, st);
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
    return dtype == PARARNN_F32 ? gs::launch_backward<float>(who, pr, dL_dlambda, st)
                                : gs::launch_backward<gs::bf16>(who, pr, dL_dlambda, st);
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
