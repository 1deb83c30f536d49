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

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "abi_util.cuh"
#include "bulk.cuh"
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
// steps between two states that the forward keeps for the adjoint: a warp's share of a tile
constexpr int kCkSteps = 8;

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
    int nCG, nCk;          // channel groups; checkpoints per batch row
    int ranks;             // blocks per cluster
    int segs, seg_rounds;  // ranges of T, and the rounds of one
    float4* elems;         // (B, segs + 1, nCG, 32): the state before the first range, and the ranges' elements
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
    float* part;  // (B * segs * ranks, D)
    float* dh0;   // (B,D) or null
    unsigned* status;
    int64_t B, T, D;
    int nCG, nCk;
    int ranks;
    int segs, seg_rounds;
    float4* elems;  // the ranges' elements, and the state behind the last range
    float decay;
};

__device__ __forceinline__ float softplus_f(float x) { return x > 20.0f ? x : log1pf(expf(x)); }
// k = c softplus(lambda), so that y = k r; finite for a finite lambda, as 0 k has to be 0
__device__ __forceinline__ float scale_of(float decay, float lambda) {
    const float k = decay * softplus_f(lambda);
    return k > FLT_MAX ? FLT_MAX : k;
}

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
// A block owns 64 channels of one batch row and walks T in tiles of 8 R steps; with
// few channels a cluster of up to 8 blocks takes that many neighbouring tiles
// at once (a round).  Lane l of every warp holds channels 2l, 2l+1, and warp w holds R
// consecutive steps of the tile, so a warp's scan needs no shuffles: each thread evaluates
// its R steps into registers (a_t, u_t), composes them into h -> P h + B, and after one block
// barrier per tile applies the elements of the warps before it to the carry and walks its
// steps.  The last warp forms the carry of the next tile.  In a cluster the last warp
// first sends the tile's element into every block's shared memory, where an
// mbarrier counts the bytes: no block waits for more than the data it needs.
// Where even clusters of 8 leave most of the device idle, T is cut into ranges: a first
// launch (kSum) forms each range's element, and in the second each range's blocks start
// from those of the ranges before it.  That reads the pre-activations twice, on many times the SMs.
// Otherwise every pre-activation is read once, by tensor copies two tiles ahead; where rows or
// buffers are not multiples of 16 bytes (kTma false) each warp copies the 16-byte granules that
// hold its rows' pieces (RowRing), or reads them directly.
//
// Measured: 4x32768x1024 float32 320 us, 6.7 TB/s (with checkpoints 367), bound by HBM; bfloat16, which has
// half the bytes for the same arithmetic, 8x4096x2048 115 us, 4.7 TB/s, and 1x131072x4096 in clusters 955 us, 4.5 TB/s,
// bound by instructions, the special-function unit and the tile's phases, which overlap only between
// the two blocks of an SM.  16 steps a thread halve what a tile costs beside its steps (1x131072x4096, on
// earlier code: 1.07 times its time with 12, 1.23 with 8).
constexpr int kW = 64;  // channels per block
constexpr int kMaxRanks = 8;

template <typename T, bool kForward, bool kTma>
struct Tile {
    // the forward of bfloat16 has the registers and the stages for 16 steps a thread
    static constexpr int R = kForward && kTma && sizeof(T) == 2 ? 16 : kCkSteps;
    static constexpr int NW = 8;  // warps per block
    static constexpr int L = NW * R;
};

// An affine map h -> P h + B of two channels.  P is a product of decays, 0 to
// 1; P = -1 stands for a map through a marked step, which is h -> B for every h.
struct Elem {
    f2 P, B;
};
__device__ __forceinline__ float4 pack(const Elem& e) { return make_float4(e.P.x, e.P.y, e.B.x, e.B.y); }
__device__ __forceinline__ Elem unpack(float4 v) { return Elem{f2{v.x, v.y}, f2{v.z, v.w}}; }
template <bool kCuts>
__device__ __forceinline__ f2 apply(const Elem& e, f2 h) {
    const f2 to = fma2(e.P, h, e.B);
    if (kCuts && e.P.x < 0.0f) return e.B;
    return to;
}
// first `e`, then `f`
template <bool kCuts>
__device__ __forceinline__ Elem then(const Elem& e, const Elem& f) {
    Elem o{mul2(f.P, e.P), fma2(f.P, e.B, f.B)};
    if (kCuts && f.P.x < 0.0f) o = f;
    if (kCuts && e.P.x < 0.0f) o.P = splat2(-1.0f);
    return o;
}

// Rows that do not start on 16 bytes: each warp keeps a ring of its own pieces, kN of
// them a round (its steps' gates), each the 16-byte granules that hold 64 channels,
// brought by one bulk copy of one lane.  A round with a piece whose granules reach over the ends
// of its array is marked and read from global memory directly.  8x2000x2051 bfloat16: forward
// 109 us, adjoint 212; float32 adjoint of 16x1000x1001 146 us.  On earlier code: the former 107 and 213,
// with direct loads alone 146 and 268, as two 2-byte loads stand for one of 4; the latter 150, direct 159, but the
// float32 forward 67.6, direct 65.5, so that pass has no ring.
template <typename T, int kN>
struct RowRing {
    static constexpr int kSlots = sizeof(T) == 2 ? 2 : 1, kPitch = kW * (int)sizeof(T) + 16;
    alignas(16) unsigned char piece[kSlots][kN][kPitch];
    uint64_t bar[kSlots];
};
struct NoRing {};
template <typename T, bool kForward, bool kTma>
constexpr bool kHasRing = !kTma && !(kForward && sizeof(T) == 4);

template <typename T, bool kTma>
struct FwdSmem {
    static constexpr int kStages = kTma ? 2 : 0;
    alignas(128) T px[kTma ? kStages : 1][kTma ? Tile<T, true, kTma>::L : 1][3][kW];
    std::conditional_t<kHasRing<T, true, kTma>, RowRing<T, 3 * kCkSteps>, NoRing> ring[Tile<T, true, kTma>::NW];
    float4 warp[2][Tile<T, true, kTma>::NW][32];  // each warp's element, two rounds in turn
    float4 rank[2][kMaxRanks][32];  // each of the cluster's tiles
    float2 carry[2][32];            // the state before the round
    uint64_t bar[kStages + 1], rank_bar[2];
};

__device__ __forceinline__ f2 ld2(const float* p) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    return f2{v.x, v.y};
}
__device__ __forceinline__ f2 ld2(const bf16* p) {
    const unsigned v = *reinterpret_cast<const unsigned*>(p);
    return f2{__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
}
template <typename T>
__device__ __forceinline__ f2 load_pair(const T* p, bool in0, bool in1) {
    return f2{in0 ? PxTraits<T>::cvt(p[0]) : 0.0f, in1 ? PxTraits<T>::cvt(p[1]) : 0.0f};
}
__device__ __forceinline__ void st2(float* p, f2 v) { *reinterpret_cast<float2*>(p) = make_float2(v.x, v.y); }
__device__ __forceinline__ void st2(bf16* p, f2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// 16 bytes to the same place of block `rank` of the cluster, counted on its mbarrier
__device__ __forceinline__ void send16(float4* local, uint64_t* local_bar, uint32_t rank, float4 v) {
    uint32_t to, bar;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(local_bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(to),
                 "r"(bar), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// the box of a tile's steps, of some gates and 64 channels of one batch row
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// a box from shared memory, a group of its own; parts of it outside the tensor are not written
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// the thread's stores have read their shared memory
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <typename T, int kN>
struct RingState {
    static constexpr int kSlots = RowRing<T, kN>::kSlots;
    RowRing<T, kN>& ring;
    unsigned marked = 0, phase = 0;  // a bit for each slot

    __device__ __forceinline__ explicit RingState(RowRing<T, kN>& r, int lane) : ring(r) {
        if (lane == 0) {
            for (int i = 0; i < RowRing<T, kN>::kSlots; ++i) mbar_init(&ring.bar[i], 1);
            mbar_fence_init();
        }
        __syncwarp();
    }
    // lane l brings piece l: `bytes` from src, of an array [begin, end); nothing where bytes is 0
    __device__ __forceinline__ void fill(int slot, int lane, const void* src, int bytes, const void* begin, const void* end) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(src), lo = at & ~uintptr_t(15);
        const unsigned n = bytes ? (unsigned)((at - lo + bytes + 15) & ~uintptr_t(15)) : 0u;
        const bool over = n && (lo < reinterpret_cast<uintptr_t>(begin) || lo + n > reinterpret_cast<uintptr_t>(end));
        if (__any_sync(0xffffffffu, over)) {
            marked |= 1u << slot;
            return;
        }
        marked &= ~(1u << slot);
        const unsigned all = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) mbar_arrive_expect_tx(&ring.bar[slot], all);
        __syncwarp();
        if (n) bulk_load(ring.piece[slot][lane], lo, n, &ring.bar[slot]);
    }
    // whether the slot's round is to be read from global memory; else waits for it
    __device__ __forceinline__ bool direct(int slot, bool& late) {
        if (marked >> slot & 1) return true;
        wait_bar<false>(&ring.bar[slot], phase >> slot & 1, late);
        phase ^= 1u << slot;
        return false;
    }
    // channels 2 lane, 2 lane + 1 of piece i, which begins at src
    __device__ __forceinline__ f2 read(int slot, int i, const T* src, int lane) const {
        const T* p = reinterpret_cast<const T*>(ring.piece[slot][i] + (reinterpret_cast<uintptr_t>(src) & 15)) + 2 * lane;
        return f2{PxTraits<T>::cvt(p[0]), PxTraits<T>::cvt(p[1])};
    }
};

struct NoRingState {
    static constexpr int kSlots = 0;
    __device__ __forceinline__ NoRingState(NoRing&, int) {}
};
template <typename T, bool kForward, bool kTma>
using RingOf =
    std::conditional_t<kHasRing<T, kForward, kTma>, RingState<T, (kForward ? 3 : 4) * kCkSteps>, NoRingState>;

// Two channels' decay a = e^-y and m = 1 - a.  For y <= 1 m is y times a polynomial of
// degree 5 for (1 - e^-y) / y, exact at 0 and fitted to [0, 1] by reweighted least squares: off by at
// most 9.7e-8 of it there, 4e-9 below y = 1e-3.  a is 1 - m, rounded to nearest: an error
// of a that leans to one side would add up over a memory of 1/m steps, as that of an
// approximate exponential does.  kWide, for decays that reach past 1: there a is the
// exponential, which keeps the digits of a small a.  kTiny keeps 1 - a^2 above zero where
// y is zero (its root, 3e-19, stands for zero then).
constexpr float kTiny = 1e-37f;
template <bool kWide>
__device__ __forceinline__ void decay2(f2 y, f2& a, f2& m) {
    f2 s = fma2(y, splat2(-9.14316508e-4f), splat2(7.84359034e-3f));
    s = fma2(y, s, splat2(-4.14267108e-2f));
    s = fma2(y, s, splat2(1.66614130e-1f));
    s = fma2(y, s, splat2(-4.99996185e-1f));
    s = fma2(y, s, splat2(1.0f));
    m = fma2(y, s, splat2(kTiny));
    a = sub2(splat2(1.0f), m);
    if constexpr (kWide) {
        const f2 e = ex2_2(mul2(y, splat2(-kLog2e)));
        if (y.x > 1.0f) a.x = e.x, m.x = 1.0f - e.x;
        if (y.y > 1.0f) a.y = e.y, m.y = 1.0f - e.y;
        // a NaN decay takes the polynomial, which keeps it
    }
}
__device__ __forceinline__ f2 exp_neg2(f2 x) { return ex2_2(mul2(x, splat2(-kLog2e))); }

// u = sqrt(v) sig(p_i) x, v = 1 - a^2, the root and the gate each by itself
__device__ __forceinline__ f2 input_of(f2 v, f2 pi, f2 x) {
    return mul2(mul2(x, sigmoid2(pi)), mul2(v, f2{rsqrt_approx(v.x), rsqrt_approx(v.y)}));
}
__device__ __forceinline__ f2 input2(f2 y, f2 pi, f2 x) {
    f2 a, m;
    decay2<true>(y, a, m);
    return input_of(fma2(m, a, m), pi, x);
}
// a and u = sqrt(1 - a^2) sig(p_i) x from y.  With v = 1 - a^2 = m (1 + a) and d = 1 + e^{-p_i},
// u = x v / sqrt(q), q = v d^2: one reciprocal square root for the root and the gate's reciprocal.  Below
// p_i = -44 q can overflow, and u is 0 then, though x may be large enough to make up for the gate: `over`
// becomes NaN with a q that is not finite, and the caller takes input2's u for such steps.  That is one packed
// instruction of about 54: 8x4096x2048 bfloat16 114.9 us, 113.0 without.  (One for two steps, of the product of
// their q, is no faster: 115.1.)  kApart has no q: its u is input_of's.
template <bool kWide, bool kApart>
__device__ __forceinline__ void eval2(f2 y, f2 pi, f2 x, f2& a, f2& u, f2& over) {
    f2 m;
    decay2<kWide>(y, a, m);
    const f2 v = fma2(m, a, m);
    if constexpr (kApart) {
        u = input_of(v, pi, x);
    } else {
        const f2 d = add2(exp_neg2(pi), splat2(1.0f));
        const f2 q = mul2(mul2(v, d), d);
        over = fma2(q, splat2(0.0f), over);
        u = mul2(mul2(x, v), f2{rsqrt_approx(q.x), rsqrt_approx(q.y)});
    }
}

template <typename T, bool kTma, bool kCluster, bool kCuts, bool kSum>
__global__ void __launch_bounds__(Tile<T, true, kTma>::NW * 32, 2)
    forward_kernel(const Params pr, const __grid_constant__ CUtensorMap map) {
    typedef Tile<T, true, kTma> Tl;
    constexpr int kStages = FwdSmem<T, kTma>::kStages, R = Tl::R, L = Tl::L, kNW = Tl::NW;
    // Where rows are read from global memory directly, by blocks of their own, the gate has its own reciprocal
    // (8x2000x2051 float32 110.2 us, with the look at q 114.5); clusters, with a few blocks that wait for
    // one another, are slower with that (1x100000x63 float32 59.9, 58.4), and so are rings (8x2000x2051
    // bfloat16 113.1, 107.1).
    constexpr bool kApart = !kTma && !kHasRing<T, true, kTma> && !kCluster;
    extern __shared__ unsigned char raw[];
    FwdSmem<T, kTma>& sm = *reinterpret_cast<FwdSmem<T, kTma>*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // one value for the warp
    const uint32_t rank = kCluster ? cluster_ctarank() : 0u;
    const int C = kCluster ? pr.ranks : 1;
    const int group = (int)(blockIdx.x / C), range = group / pr.nCG, cg = group - range * pr.nCG;
    const int b = range / pr.segs, seg = range - b * pr.segs;
    const int d0 = cg * kW, d = d0 + 2 * lane;
    float4* elems = pr.elems + ((int64_t)(b * (pr.segs + 1)) * pr.nCG + cg) * 32 + lane;  // of this group, nCG * 32 apart
    if (kSum && seg == pr.segs - 1) return;  // nothing starts from the last range
    const int T_ = (int)pr.T, D = (int)pr.D;
    const bool in0 = d < D, in1 = d + 1 < D;
    const int first = seg * pr.seg_rounds;  // the range's first round
    const int rounds = min(pr.seg_rounds, ((T_ + L - 1) / L + C - 1) / C - first);
    const T* px = static_cast<const T*>(pr.px) + (int64_t)b * T_ * 3 * D;

    auto issue = [&](int round) {
        if constexpr (kTma) {
            const int t0 = ((first + round) * C + (int)rank) * L;
            if (round < rounds && t0 < T_) {
                uint64_t* bar = &sm.bar[round % kStages];
                mbar_arrive_expect_tx(bar, (uint32_t)(L * 3 * kW * sizeof(T)));
                tma_load_4d(sm.px[round % kStages], &map, bar, d0, 0, t0, b);
            }
        }
    };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&sm.bar[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.rank_bar[i], 1);
        mbar_fence_init();
    }
    constexpr int kSlots = RingOf<T, true, kTma>::kSlots;
    RingOf<T, true, kTma> ring(sm.ring[warp], lane);
    follow_previous();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) issue(i);  // under way while the rest is set up
        if (kCluster)
            for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&sm.rank_bar[i], C * (uint32_t)sizeof sm.rank[0][0]);
    }
    f2 k{0.0f, 0.0f};
    if (in0) k.x = scale_of(pr.decay, pr.lam[d]);
    if (in1) k.y = scale_of(pr.decay, pr.lam[d + 1]);
    const bool wide = __any_sync(0xffffffffu, !(k.x <= 1.0f && k.y <= 1.0f));
    if (warp == 0) {
        f2 h{0.0f, 0.0f};
        if (pr.segs == 1 || kSum) {
            if (pr.h0 && in0) h.x = pr.h0[(int64_t)b * D + d];
            if (pr.h0 && in1) h.y = pr.h0[(int64_t)b * D + d + 1];
            // h_last may be h0's buffer: the second launch reads this copy
            if (kSum && seg == 0 && rank == 0) *elems = make_float4(0.0f, 0.0f, h.x, h.y);
        } else {
            h = unpack(*elems).B;
#pragma unroll 4
            for (int i = 0; i < seg; ++i) h = apply<kCuts>(unpack(elems[(int64_t)(i + 1) * pr.nCG * 32]), h);
        }
        sm.carry[0][lane] = make_float2(h.x, h.y);
    }
    // every block has begun, and has read h0 (h_last may be the same buffer)
    if constexpr (kCluster) {
        cluster_arrive_release();
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    // lane j of a warp reads the mark of the warp's step j, a round ahead
    auto marks_of = [&](int round) -> unsigned {
        const int t = ((first + round) * C + (int)rank) * L + warp * R + lane;
        return (lane < R && round < rounds && t < T_) ? pr.reset[(int64_t)b * T_ + t] : 0u;
    };
    unsigned mark = kCuts ? marks_of(0) : 0u;
    bool late = false, bad = false;
    auto put = [&](T* o, f2 h) {
        if constexpr (kTma) {
            if (in0) st2(o, h);
        } else {
            if (in0) o[0] = to_out<T>(h.x);
            if (in1) o[1] = to_out<T>(h.y);
        }
    };
    auto keep = [&](int i, f2 h) {
        float* o = pr.ck + ((int64_t)b * pr.nCk + i) * D + d;
        if constexpr (kTma) {
            if (in0) st2(o, h);
        } else {
            if (in0) o[0] = h.x;
            if (in1) o[1] = h.y;
        }
    };
    int t0 = (first * C + (int)rank) * L + warp * R;  // the warp's first step
    auto piece = [&](int t, int j, int g) { return px + ((int64_t)(t + j) * 3 + g) * D + d0; };
    auto fill = [&](int round) {
        if constexpr (kHasRing<T, true, kTma>) {
            const int t = ((first + round) * C + (int)rank) * L + warp * R;
            if (round >= rounds || t >= T_) return;
            const bool mine = lane < 3 * R && t + lane / 3 < T_;
            const T* from = static_cast<const T*>(pr.px);
            ring.fill(round % kSlots, lane, piece(t, lane / 3, lane % 3), mine ? min(kW, D - d0) * (int)sizeof(T) : 0, from,
                      from + pr.B * T_ * 3 * D);
        }
    };
    for (int i = 0; i < kSlots; ++i) fill(i);
    Elem sum{splat2(1.0f), splat2(0.0f)};  // kSum: of the range, in the last warp
    T* H = static_cast<T*>(pr.H) + ((int64_t)b * T_ + t0) * D;

    for (int round = 0; round < rounds; ++round) {
        const int par = round & 1, tile0 = t0 - warp * R;
        int st = 0;
        if constexpr (kTma) st = round % kStages;
        unsigned marks = 0;
        if constexpr (kCuts) {
            marks = __ballot_sync(0xffffffffu, mark != 0);
            mark = marks_of(round + 1);
        }
        if constexpr (kTma)
            if (tile0 < T_) wait_bar<false>(&sm.bar[st], (round / kStages) & 1, late);
        f2 a[R], u[R];
        Elem e{splat2(1.0f), splat2(0.0f)};
        if (t0 < T_) {
            // at(j, g): gate g of step j
            auto evaluate = [&](auto at) {
                f2 over{0.0f, 0.0f};
                if (!wide) {
#pragma unroll
                    for (int j = 0; j < R; ++j)
                        eval2<false, kApart>(mul2(k, sigmoid2(at(j, 0))), at(j, 1), at(j, 2), a[j], u[j], over);
                } else {
#pragma unroll
                    for (int j = 0; j < R; ++j)
                        eval2<true, kApart>(mul2(k, sigmoid2(at(j, 0))), at(j, 1), at(j, 2), a[j], u[j], over);
                }
                if (!kApart && ((in0 && over.x != over.x) || (in1 && over.y != over.y))) {
#pragma unroll 1
                    for (int j = 0; j < R; ++j) {  // rolled up: this needs no registers of its own
                        const f2 y = mul2(k, sigmoid2(at(j, 0))), pi = at(j, 1), x = at(j, 2);
                        f2 aj, uj, own{0.0f, 0.0f};
                        eval2<true, false>(y, pi, x, aj, uj, own);
                        const f2 other = input2(y, pi, x);
                        // only where this step's own q asks for it: a ring has no values for steps past T
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            if (i == j && own.x != own.x) u[i].x = other.x;
                            if (i == j && own.y != own.y) u[i].y = other.y;
                        }
                    }
                }
            };
            if constexpr (kTma) {
                evaluate([&](int j, int g) { return ld2(&sm.px[st][warp * R + j][g][2 * lane]); });
            } else {
                auto load = [&](int j, int g) {
                    return load_pair(piece(t0, j, g) + 2 * lane, in0 && t0 + j < T_, in1 && t0 + j < T_);
                };
                if constexpr (kHasRing<T, true, kTma>) {
                    const int slot = round % kSlots;
                    if (ring.direct(slot, late))
                        evaluate(load);
                    else
                        evaluate([&](int j, int g) { return ring.read(slot, 3 * j + g, piece(t0, j, g), lane); });
                    __syncwarp();
                    fill(round + kSlots);
                } else {
                    evaluate(load);
                }
            }
            e = Elem{a[0], u[0]};
            if (!kCuts || marks == 0) {
#pragma unroll
                for (int j = 1; j < R; ++j) {
                    e.B = fma2(a[j], e.B, u[j]);
                    e.P = mul2(a[j], e.P);
                }
            } else {
#pragma unroll
                for (int j = 1; j < R; ++j) e.B = (marks >> j & 1) ? u[j] : fma2(a[j], e.B, u[j]);
                e.P = splat2(-1.0f);
            }
        }
        sm.warp[par][warp][lane] = pack(e);
        __syncthreads();
        if (kTma && tid == 0) issue(round + kStages);  // every warp has read this round's stage

        f2 h;
        if constexpr (kCluster) {
            Elem pre{splat2(1.0f), splat2(0.0f)};
            float4 of[kNW - 1];
#pragma unroll
            for (int w = 0; w < kNW - 1; ++w) of[w] = sm.warp[par][w][lane];
#pragma unroll
            for (int w = 0; w < kNW - 1; ++w)
                if (w < warp) pre = then<kCuts>(pre, unpack(of[w]));
            if (warp == kNW - 1) {
                const float4 all = pack(then<kCuts>(pre, e));
                for (int r = 0; r < C; ++r) send16(&sm.rank[par][rank][lane], &sm.rank_bar[par], r, all);
            }
            wait_bar<true>(&sm.rank_bar[par], (round >> 1) & 1, late);
            if (tid == 0) mbar_arrive_expect_tx(&sm.rank_bar[par], C * (uint32_t)sizeof sm.rank[0][0]);
            if constexpr (kSum) {
                if (warp == kNW - 1 && rank == 0)
                    for (int r = 0; r < C; ++r) sum = then<kCuts>(sum, unpack(sm.rank[par][r][lane]));
                t0 += C * L;
                continue;
            }
            h = ld2(&sm.carry[par][lane].x);
            for (int r = 0; r < (int)rank; ++r) h = apply<kCuts>(unpack(sm.rank[par][r][lane]), h);
            if (warp == kNW - 1) {
                f2 c = h;
                for (int r = (int)rank; r < C; ++r) c = apply<kCuts>(unpack(sm.rank[par][r][lane]), c);
                sm.carry[par ^ 1][lane] = make_float2(c.x, c.y);
            }
            h = apply<kCuts>(pre, h);
        } else {
            h = ld2(&sm.carry[par][lane].x);
            // the elements are read at once: the last warp, whose chain of them is the longest, is
            // what the next block barrier waits for
            float4 of[kNW - 1];
#pragma unroll
            for (int w = 0; w < kNW - 1; ++w) of[w] = sm.warp[par][w][lane];
#pragma unroll
            for (int w = 0; w < kNW - 1; ++w)
                if (w < warp) h = apply<kCuts>(unpack(of[w]), h);
            if (warp == kNW - 1) {
                const f2 c = apply<kCuts>(e, h);
                sm.carry[par ^ 1][lane] = make_float2(c.x, c.y);
            }
        }
        if (t0 < T_) {
            if (pr.ck) keep(t0 / kCkSteps, h);
            const int n = min(R, T_ - t0);
            T* o = H + d;
            if ((!kCuts || marks == 0) && n == R) {
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    if (j && j % kCkSteps == 0 && pr.ck) keep((t0 + j) / kCkSteps, h);
                    h = fma2(a[j], h, u[j]);
                    put(o, h);
                    o += D;
                }
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (j < n) {
                        if (j && j % kCkSteps == 0 && pr.ck) keep((t0 + j) / kCkSteps, h);
                        if (kCuts && (marks >> j & 1)) {
                            bad |= (in0 && !isfinite(h.x)) || (in1 && !isfinite(h.y));
                            h = u[j];
                        } else {
                            h = fma2(a[j], h, u[j]);
                        }
                        put(o, h);
                        o += D;
                    }
            }
            // without a marked step a state that is not finite stays so
            bad |= (in0 && !isfinite(h.x)) || (in1 && !isfinite(h.y));
            if (pr.last && t0 + n == T_) {
                float* q = pr.last + (int64_t)b * D + d;
                if (in0) q[0] = h.x;
                if (in1) q[1] = h.y;
            }
        }
        t0 += C * L;
        H += (int64_t)C * L * D;
    }
    if (kSum && warp == kNW - 1 && rank == 0) elems[(int64_t)(seg + 1) * pr.nCG * 32] = pack(sum);
    if (pr.status) {
        const unsigned bits = (__any_sync(0xffffffffu, bad) ? kStatusNonFinite : 0u) |
                              (__any_sync(0xffffffffu, late) ? kStatusTimeout : 0u);
        if (bits && lane == 0) atomicOr(pr.status, bits);
    }
    // no block leaves while a peer's element may be on its way to it
    if constexpr (kCluster) {
        cluster_arrive_release();
        cluster_wait_acquire();
    }
}

// ---- adjoint --------------------------------------------------------------------
// The forward's tiles in reversed time.  The scan runs on mu_t = a_t l_t, l_t =
// g_t + mu_{t+1}, whose elements need p_r and g only: a round first forms y and
// the elements and frees those arrays' stage.  With the carry, each thread walks its
// steps backwards for l, then forwards from the checkpoint, the state before its
// first step, for h_{t-1} and the gradients: of the states one in R is read, and the
// forward's scan is not repeated.
//
// Measured: 4x32768x1024 float32 614 us, 6.1 TB/s, bound by HBM; bfloat16 8x4096x2048 176 us, 5.3 TB/s,
// 1x131072x4096 in clusters 1.59 ms, 4.7 TB/s, bound as the forward is.  With marks on 1 step in 500 674 us, 196 us and
// 2.06 ms.  The instance for float32 rows off 16 bytes in clusters spills 100 bytes, with marks 176, the
// aligned one with marks 16; the others up to 4.
template <typename T, bool kTma>
struct BwdSmem {
    static constexpr int kA = kTma ? 4 / sizeof(T) : 0, kB = kTma ? 2 : 0;  // stages of p_r and g, of p_i and x
    static constexpr int kRows = kTma ? Tile<T, false, kTma>::L : 1;
    // the gradients of bfloat16 leave by tensor copies, a warp's steps at a time (8x4096x2048, on
    // earlier code: 180 us, 190 with the threads' own stores of two channels); float32 has no room for it
    static constexpr bool kOut = kTma && sizeof(T) == 2;
    alignas(128) T pr[kA + !kTma][kRows][kW];
    alignas(128) T g[kA + !kTma][kRows][kW];
    alignas(128) T ix[kB + !kTma][kRows][2][kW];
    alignas(128) T out[kOut ? Tile<T, false, kTma>::NW : 1][kOut ? kCkSteps : 1][kOut ? 3 : 1][kOut ? kW : 1];
    std::conditional_t<kHasRing<T, false, kTma>, RowRing<T, 4 * kCkSteps>, NoRing> ring[Tile<T, false, kTma>::NW];
    float4 warp[2][Tile<T, false, kTma>::NW][32];
    float4 rank[2][kMaxRanks][32];
    float2 carry[2][32];
    uint64_t bar_a[kA + 1], bar_b[kB + 1], rank_bar[2];
};

struct BwdMaps {
    CUtensorMap pr, ix, g, out;  // boxes of one gate, of two gates, of dL/dH, and of a warp's dL/dpx
};

// the gradients of one step of two channels; h is h_{t-1} in and h_t out
__device__ __forceinline__ void grads2(f2 y, f2 a, f2 m, f2 l, f2 pi, f2 x, f2 kinv, f2& h, f2& dpr, f2& dpi, f2& dx,
                                       f2& w) {
    const f2 v = fma2(m, a, m);
    const f2 i = sigmoid2(pi);
    const f2 ib = mul2(f2{rsqrt_approx(v.x), rsqrt_approx(v.y)}, i);  // i / b
    const f2 e = mul2(ib, x);
    const f2 ah = mul2(a, h);
    dx = mul2(l, mul2(v, ib));
    // in an order in which no partial product is much larger than its factors and the whole: y may be as large as a
    // float can be, and a, and with it the difference, is 0 then
    dpi = mul2(dx, mul2(x, sub2(splat2(1.0f), i)));
    w = mul2(l, mul2(y, sub2(mul2(mul2(a, a), e), ah)));
    dpr = mul2(w, sub2(splat2(1.0f), mul2(y, kinv)));
    h = fma2(v, e, ah);
}

template <typename T, bool kTma, bool kCluster, bool kCuts, bool kSum>
__global__ void __launch_bounds__(Tile<T, false, kTma>::NW * 32, 2)
    backward_kernel(const BwdParams pr, const __grid_constant__ BwdMaps maps) {
    typedef Tile<T, false, kTma> Tl;
    constexpr int kA = BwdSmem<T, kTma>::kA, kB = BwdSmem<T, kTma>::kB, R = Tl::R, L = Tl::L, kNW = Tl::NW;
    static_assert(R == kCkSteps, "a thread's steps begin at a checkpoint");
    extern __shared__ unsigned char raw[];
    BwdSmem<T, kTma>& sm = *reinterpret_cast<BwdSmem<T, kTma>*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = kCluster ? cluster_ctarank() : 0u;
    const int C = kCluster ? pr.ranks : 1;
    const int group = (int)(blockIdx.x / C), range = group / pr.nCG, cg = group - range * pr.nCG;
    const int b = range / pr.segs, seg = range - b * pr.segs;
    const int d0 = cg * kW, d = d0 + 2 * lane;
    float4* elems = pr.elems + ((int64_t)(b * (pr.segs + 1)) * pr.nCG + cg) * 32 + lane;  // of this group, nCG * 32 apart
    if (kSum && seg == 0) return;  // nothing starts from the first range
    const int T_ = (int)pr.T, D = (int)pr.D;
    const bool in0 = d < D, in1 = d + 1 < D;
    const int first = seg * pr.seg_rounds;  // the range's first round in time
    const int tiles = (T_ + L - 1) / L, rounds = min(pr.seg_rounds, (tiles + C - 1) / C - first);
    const T* px = static_cast<const T*>(pr.px) + (int64_t)b * T_ * 3 * D;
    const T* dH = static_cast<const T*>(pr.dH) + (int64_t)b * T_ * D;

    // round q takes the cluster's tiles from the last ones on; only round 0 may have tiles past T
    auto tile_of = [&](int q) { return (first + rounds - 1 - q) * C + (int)rank; };
    const int q0 = tile_of(0) < tiles ? 0 : 1;  // the block's first tile is of this round
    auto issue_a = [&](int i) {
        if constexpr (!kTma) return;
        if (q0 + i >= rounds) return;
        const int t0 = tile_of(q0 + i) * L, st = kTma ? i % (kA + !kTma) : 0;
        mbar_arrive_expect_tx(&sm.bar_a[st], (uint32_t)(L * 2 * kW * sizeof(T)));
        tma_load_4d(sm.pr[st], &maps.pr, &sm.bar_a[st], d0, 0, t0, b);
        tma_load_4d(sm.g[st], &maps.g, &sm.bar_a[st], d0, 0, t0, b);
    };
    auto issue_b = [&](int i) {
        if constexpr (!kTma) return;
        if (q0 + i >= rounds) return;
        const int t0 = tile_of(q0 + i) * L, st = kTma ? i % (kB + !kTma) : 0;
        mbar_arrive_expect_tx(&sm.bar_b[st], (uint32_t)(L * 2 * kW * sizeof(T)));
        tma_load_4d(sm.ix[st], &maps.ix, &sm.bar_b[st], d0, 1, t0, b);
    };
    if (tid == 0) {
        for (int i = 0; i < kA; ++i) mbar_init(&sm.bar_a[i], 1);
        for (int i = 0; i < kB; ++i) mbar_init(&sm.bar_b[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.rank_bar[i], 1);
        mbar_fence_init();
    }
    constexpr int kSlots = RingOf<T, false, kTma>::kSlots;
    RingOf<T, false, kTma> ring(sm.ring[warp], lane);
    follow_previous();
    if (tid == 0) {
        for (int i = 0; i < kA; ++i) issue_a(i);
        for (int i = 0; i < (kSum ? 0 : kB); ++i) issue_b(i);
        if (kCluster)
            for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&sm.rank_bar[i], C * (uint32_t)sizeof sm.rank[0][0]);
    }
    f2 k{0.0f, 0.0f};
    if (in0) k.x = scale_of(pr.decay, pr.lam[d]);
    if (in1) k.y = scale_of(pr.decay, pr.lam[d + 1]);
    // r = y / k; a k this small gives no gradient to p_r (w is below 2^-60 l)
    const f2 kinv{k.x > 1e-37f ? 1.0f / k.x : 0.0f, k.y > 1e-37f ? 1.0f / k.y : 0.0f};
    const bool wide = __any_sync(0xffffffffu, !(k.x <= 1.0f && k.y <= 1.0f));
    if (warp == 0) {
        f2 mu{0.0f, 0.0f};
        if (pr.dlast && in0) mu.x = pr.dlast[(int64_t)b * D + d];
        if (pr.dlast && in1) mu.y = pr.dlast[(int64_t)b * D + d + 1];
        if (!kSum)
#pragma unroll 4
            for (int i = pr.segs - 1; i > seg; --i) mu = apply<kCuts>(unpack(elems[(int64_t)i * pr.nCG * 32]), mu);
        sm.carry[0][lane] = make_float2(mu.x, mu.y);
    }
    if constexpr (kCluster) {
        cluster_arrive_release();
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    auto marks_of = [&](int q) -> unsigned {
        if (q >= rounds) return 0u;
        const int t = tile_of(q) * L + warp * R + lane;
        return (lane < R && t < T_) ? pr.reset[(int64_t)b * T_ + t] : 0u;
    };
    unsigned mark = kCuts ? marks_of(0) : 0u;
    bool late = false;
    // chk becomes NaN with a dL/dp_i that is not finite, and so with such a dL/dx, a factor of it
    f2 sum{0.0f, 0.0f}, chk{0.0f, 0.0f};
    Elem whole{splat2(1.0f), splat2(0.0f)};  // kSum: of the range, in warp 0

    constexpr bool kOut = BwdSmem<T, kTma>::kOut;
    // bfloat16, which waits for instructions and latency, reads the checkpoint and the warps'
    // elements ahead (8x4096x2048, on earlier code: 181 us, 210 without); float32, which waits for HBM, has no
    // registers for that (4x32768x1024: 650 us with, 613 without)
    constexpr bool kEarly = sizeof(T) == 2;
    // pieces 4 j .. 4 j + 3: the gates and dL/dH of step j
    auto piece = [&](int t, int j, int g) {
        return g < 3 ? px + ((int64_t)(t + j) * 3 + g) * D + d0 : dH + (int64_t)(t + j) * D + d0;
    };
    auto fill = [&](int q) {
        if constexpr (!kTma) {
            if (q < q0 || q >= rounds) return;
            const int t = tile_of(q) * L + warp * R, g = lane & 3;
            if (t >= T_) return;
            const bool mine = t + lane / 4 < T_ && (!kSum || g == 0 || g == 3);
            const T* from = static_cast<const T*>(g < 3 ? pr.px : pr.dH);
            ring.fill((q - q0) % kSlots, lane, piece(t, lane / 4, g), mine ? min(kW, D - d0) * (int)sizeof(T) : 0, from,
                      from + pr.B * T_ * D * (g < 3 ? 3 : 1));
        }
    };
    for (int i = 0; i < kSlots; ++i) fill(q0 + i);

    auto put = [&](int j, T* o, f2 dpr, f2 dpi, f2 dx) {
        if constexpr (kOut) {
            T* to = &sm.out[warp][j][0][2 * lane];
            st2(to, dpr);
            st2(to + kW, dpi);
            st2(to + 2 * kW, dx);
        } else if constexpr (kTma) {
            if (in0) {
                st2(o, dpr);
                st2(o + D, dpi);
                st2(o + 2 * (int64_t)D, dx);
            }
        } else {
            if (in0) o[0] = to_out<T>(dpr.x), o[D] = to_out<T>(dpi.x), o[2 * (int64_t)D] = to_out<T>(dx.x);
            if (in1) o[1] = to_out<T>(dpr.y), o[D + 1] = to_out<T>(dpi.y), o[2 * (int64_t)D + 1] = to_out<T>(dx.y);
        }
    };

    for (int q = 0; q < rounds; ++q) {
        const int par = q & 1, i = q - q0;
        const int tile0 = tile_of(q) * L, t0 = tile0 + warp * R;
        const int n = max(0, min(R, T_ - t0));  // this warp's steps
        const int sa = kTma && i >= 0 ? i % (kA + !kTma) : 0, sb = kTma && i >= 0 ? i % (kB + !kTma) : 0;
        unsigned marks = 0;
        if constexpr (kCuts) {
            marks = __ballot_sync(0xffffffffu, mark != 0);
            mark = marks_of(q + 1);
        }
        // the state before the warp's steps
        f2 h{0.0f, 0.0f};
        auto read_state = [&]() {
            const float* ck = pr.ck + ((int64_t)b * pr.nCk + t0 / R) * D + d;
            if constexpr (kTma) {
                if (in0) h = ld2(ck);
            } else {
                h = load_pair(ck, in0, in1);
            }
        };
        if (kEarly && n > 0 && !kSum) read_state();
        if constexpr (kTma)
            if (i >= 0) wait_bar<false>(&sm.bar_a[sa], (i / kA) & 1, late);
        // p_r, g, p_i and x of step j
        int slot = 0;
        bool direct = false;
        if constexpr (!kTma)
            if (n > 0) {
                slot = i % kSlots;
                direct = ring.direct(slot, late);
            }
        auto from_ring = [&](int j, int g) -> f2 {
            if constexpr (!kTma) {
                if (!direct) return ring.read(slot, 4 * j + g, piece(t0, j, g), lane);
                return load_pair(piece(t0, j, g) + 2 * lane, in0, in1);
            }
            return f2{0.0f, 0.0f};
        };
        auto at_r = [&](int j) -> f2 {
            if constexpr (kTma) return ld2(&sm.pr[sa][warp * R + j][2 * lane]);
            return from_ring(j, 0);
        };
        auto at_g = [&](int j) -> f2 {
            if constexpr (kTma) return ld2(&sm.g[sa][warp * R + j][2 * lane]);
            return from_ring(j, 3);
        };
        auto at_ix = [&](int j, int g) -> f2 {
            if constexpr (kTma) return ld2(&sm.ix[sb][warp * R + j][g][2 * lane]);
            return from_ring(j, 1 + g);
        };
        // y, g and the element of mu over the warp's steps; steps past T keep mu (y = 0, g = 0)
        f2 y[R], l[R], m[R];  // m only where every decay is within 1
        Elem e{splat2(1.0f), splat2(0.0f)};
        const bool plain = n == R && (!kCuts || marks == 0) && !wide;
        if (plain) {
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                y[j] = mul2(k, sigmoid2(at_r(j)));
                l[j] = at_g(j);
                f2 a;
                decay2<false>(y[j], a, m[j]);
                e.B = mul2(a, add2(l[j], e.B));
                e.P = mul2(a, e.P);
            }
        } else {
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                y[j] = l[j] = splat2(0.0f);
                if (j < n) {
                    y[j] = mul2(k, sigmoid2(at_r(j)));
                    l[j] = at_g(j);
                    f2 a, none;
                    decay2<true>(y[j], a, none);
                    e.B = (marks >> j & 1) ? splat2(0.0f) : mul2(a, add2(l[j], e.B));
                    e.P = mul2(a, e.P);
                }
            }
            if (marks) e.P = splat2(-1.0f);
        }
        sm.warp[par][warp][lane] = pack(e);
        __syncthreads();
        if (kTma && tid == 0 && i >= 0) {
            // this round's p_r and g have been read, and the round before is finished
            issue_a(i + kA);
            if (i >= 1 && !kSum) issue_b(i - 1 + kB);
        }
        f2 mu;
        if constexpr (kCluster) {
            Elem pre{splat2(1.0f), splat2(0.0f)};
            if constexpr (kEarly) {
                float4 of[kNW];
#pragma unroll
                for (int w = 1; w < kNW; ++w) of[w] = sm.warp[par][w][lane];
#pragma unroll
                for (int w = kNW - 1; w > 0; --w)
                    if (w > warp) pre = then<kCuts>(pre, unpack(of[w]));
            } else {
#pragma unroll 1
                for (int w = kNW - 1; w > warp; --w) pre = then<kCuts>(pre, unpack(sm.warp[par][w][lane]));
            }
            if (warp == 0) {
                const float4 all = pack(then<kCuts>(pre, e));
                for (int r = 0; r < C; ++r) send16(&sm.rank[par][rank][lane], &sm.rank_bar[par], r, all);
            }
            wait_bar<true>(&sm.rank_bar[par], (q >> 1) & 1, late);
            if (tid == 0) mbar_arrive_expect_tx(&sm.rank_bar[par], C * (uint32_t)sizeof sm.rank[0][0]);
            if constexpr (kSum) {
                if (warp == 0 && rank == 0)
                    for (int r = C - 1; r >= 0; --r) whole = then<kCuts>(whole, unpack(sm.rank[par][r][lane]));
                __syncwarp();
                if (i >= 0) fill(q + kSlots);
                continue;
            }
            mu = ld2(&sm.carry[par][lane].x);
            for (int r = C - 1; r > (int)rank; --r) mu = apply<kCuts>(unpack(sm.rank[par][r][lane]), mu);
            if (warp == 0) {
                f2 c = mu;
                for (int r = (int)rank; r >= 0; --r) c = apply<kCuts>(unpack(sm.rank[par][r][lane]), c);
                sm.carry[par ^ 1][lane] = make_float2(c.x, c.y);
            }
            mu = apply<kCuts>(pre, mu);
        } else {
            mu = ld2(&sm.carry[par][lane].x);
            if constexpr (kEarly) {
                float4 of[kNW];
#pragma unroll
                for (int w = 1; w < kNW; ++w) of[w] = sm.warp[par][w][lane];
#pragma unroll
                for (int w = kNW - 1; w > 0; --w)
                    if (w > warp) mu = apply<kCuts>(unpack(of[w]), mu);
            } else {
#pragma unroll 1
                for (int w = kNW - 1; w > warp; --w) mu = apply<kCuts>(unpack(sm.warp[par][w][lane]), mu);
            }
            if (warp == 0) {
                const f2 c = apply<kCuts>(e, mu);
                sm.carry[par ^ 1][lane] = make_float2(c.x, c.y);
            }
        }
        if constexpr (kTma)
            if (i >= 0) wait_bar<false>(&sm.bar_b[sb], (i / kB) & 1, late);
        if (n == 0) {
            if (i >= 0) fill(q + kSlots);
            continue;
        }
        // l backwards from mu, then the gradients forwards from the checkpoint
        if constexpr (kOut) {
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
        }
        if (!kEarly) read_state();
        f2 part{0.0f, 0.0f}, dpr, dpi, dx, w;
        T* o = static_cast<T*>(pr.dpx) + ((int64_t)b * T_ + t0) * 3 * D + d;
        if (plain) {
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                l[j] = add2(l[j], mu);
                mu = mul2(sub2(splat2(1.0f), m[j]), l[j]);
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                grads2(y[j], sub2(splat2(1.0f), m[j]), m[j], l[j], at_ix(j, 0), at_ix(j, 1), kinv, h, dpr, dpi, dx, w);
                part = add2(part, w);
                chk = fma2(dpi, splat2(0.0f), chk);
                put(j, o, dpr, dpi, dx);
                o += 3 * (int64_t)D;
            }
        } else {
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                f2 a, none;
                decay2<true>(y[j], a, none);
                l[j] = add2(l[j], mu);
                mu = (marks >> j & 1) ? splat2(0.0f) : mul2(a, l[j]);
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (j < n) {
                    if (marks >> j & 1) h = splat2(0.0f);
                    f2 a, mm;
                    decay2<true>(y[j], a, mm);
                    grads2(y[j], a, mm, l[j], at_ix(j, 0), at_ix(j, 1), kinv, h, dpr, dpi, dx, w);
                    part = add2(part, w);
                    chk = fma2(dpi, splat2(0.0f), chk);
                    put(j, o, dpr, dpi, dx);
                }
                o += 3 * (int64_t)D;
            }
        }
        __syncwarp();
        fill(q + kSlots);
        if constexpr (kOut) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) tma_store_4d(&maps.out, sm.out[warp], d0, 0, t0, b);
        }
        sum = add2(sum, part);
        if (t0 == 0 && pr.dh0) {
            float* to = pr.dh0 + (int64_t)b * D + d;
            if (in0) to[0] = mu.x;
            if (in1) to[1] = mu.y;
        }
    }
    if constexpr (kSum) {
        if (warp == 0 && rank == 0) elems[(int64_t)seg * pr.nCG * 32] = pack(whole);
        const unsigned bits = __any_sync(0xffffffffu, late) ? kStatusTimeout : 0u;
        if (bits && lane == 0) atomicOr(pr.status, bits);
        if constexpr (kCluster) {
            cluster_arrive_release();
            cluster_wait_acquire();
        }
        return;
    }
    if (kOut && lane == 0) tma_store_wait_read();
    // the warps' sums of w in order; a sum that is not finite stands for a dL/dp_r that is not
    __syncthreads();  // the last round's elements have been read
    sm.warp[0][warp][lane] = make_float4(sum.x, sum.y, 0.0f, 0.0f);
    __syncthreads();
    if (warp == 0) {
        f2 t{0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kNW; ++w) t = add2(t, unpack(sm.warp[0][w][lane]).P);
        float* o = pr.part + ((int64_t)range * C + rank) * D + d;
        if (in0) o[0] = t.x;
        if (in1) o[1] = t.y;
    }
    chk = fma2(sum, splat2(0.0f), chk);
    const bool bad = (in0 && chk.x != chk.x) || (in1 && chk.y != chk.y);
    const unsigned bits = (__any_sync(0xffffffffu, bad) ? kStatusNonFinite : 0u) |
                          (__any_sync(0xffffffffu, late) ? kStatusTimeout : 0u);
    if (bits && lane == 0) atomicOr(pr.status, bits);
    if constexpr (kCluster) {
        cluster_arrive_release();
        cluster_wait_acquire();
    }
}

// dL/dlambda = sig(lambda) / softplus(lambda) * the sum of the blocks' partial
// sums: lane = channel, each warp every sixteenth row in order, then the warps in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32)
    dlam_kernel(const float* part, const float* lam, float* dlam, int64_t rows, int64_t D) {
    __shared__ float acc[kSumWarps][32];
    follow_previous();
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

// A block takes one row and 256 V channels; it is bound by the latency of its loads for
// few rows and by HBM for many.  Rows that name the same slot must be taken in order:
// the block of the first of them takes them all, each with the state that the one before left,
// and the others' blocks end.  Every block looks through the slots for that, N
// words that the L2 cache holds, while its own loads are on their way.  Replayed from a graph:
// 1x4096 bfloat16 2.8 us, 250x2048 float32 4.9, 1500x2048 bfloat16 16.7 (12.4 without slots to look through).
constexpr int kStepThreads = 256;
constexpr int kStepRows = 8192;  // rows of one launch

template <typename T, int V>
__device__ __forceinline__ void step_load(const T* p, float (&o)[V]) {
    if constexpr (V == 4 && sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
    } else if constexpr (V == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        o[0] = __uint_as_float(v.x << 16), o[1] = __uint_as_float(v.x & 0xffff0000u);
        o[2] = __uint_as_float(v.y << 16), o[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
        o[0] = PxTraits<T>::cvt(p[0]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void step_store(T* p, const float (&v)[V]) {
    if constexpr (V == 4 && sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else if constexpr (V == 4) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
        p[0] = to_out<T>(v[0]);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const StepParams pr) {
    __shared__ unsigned more[kStepRows / 32];  // rows behind this one that name its slot
    __shared__ unsigned found;                 // 1: a row before it names the slot, 2: one behind it
    const int n0 = (int)blockIdx.x, N = (int)pr.N, tid = threadIdx.x;
    const int64_t D = pr.D, d = ((int64_t)blockIdx.y * kStepThreads + tid) * V;
    const bool in = d < D;
    follow_previous();
    const int64_t slot = pr.slots ? pr.slots[n0] : n0;
    if (slot < 0 || slot >= pr.n_slots) {
        if (slot >= 0 && pr.status && tid == 0) atomicOr(pr.status, kStatusBadIndex);
        return;
    }
    const T* px = static_cast<const T*>(pr.px) + (int64_t)n0 * 3 * D + d;
    float* state = pr.state + slot * D + d;
    float p[3][V], h[V], k[V];
    if (in) {
#pragma unroll
        for (int g = 0; g < 3; ++g) step_load<T, V>(px + g * D, p[g]);
        step_load<float, V>(state, h);
        step_load<float, V>(pr.lam + d, k);
    }
    bool chain = false;
    if (pr.slots) {
        for (int i = tid; i < (N + 31) / 32; i += kStepThreads) more[i] = 0;
        if (tid == 0) found = 0;
        __syncthreads();
        auto look = [&](int j, int32_t other) {
            if (other == (int32_t)slot && j != n0) {
                if (j > n0) atomicOr(&more[j >> 5], 1u << (j & 31));
                atomicOr(&found, j < n0 ? 1u : 2u);
            }
        };
        const int quads = (reinterpret_cast<uintptr_t>(pr.slots) & 15) == 0 ? N / 4 : 0;
#pragma unroll 4
        for (int j = tid; j < quads; j += kStepThreads) {
            const int4 q = reinterpret_cast<const int4*>(pr.slots)[j];
            look(4 * j, q.x);
            look(4 * j + 1, q.y);
            look(4 * j + 2, q.z);
            look(4 * j + 3, q.w);
        }
        for (int j = 4 * quads + tid; j < N; j += kStepThreads) look(j, pr.slots[j]);
        __syncthreads();
        if (found & 1) return;
        chain = found & 2;
    }
    if (!in) return;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) k[i] = scale_of(pr.decay, k[i]);
    for (int n = n0;;) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Row g = gates(p[0][i], p[1][i], p[2][i], k[i]);
            h[i] = __fmaf_rn(g.a, h[i], sqrtf(g.v) * g.i * g.x);
            bad |= !isfinite(h[i]);
        }
        step_store<T, V>(static_cast<T*>(pr.y) + (int64_t)n * D + d, h);
        if (!chain) break;
        do ++n;
        while (n < N && !(more[n >> 5] >> (n & 31) & 1));
        if (n == N) break;
#pragma unroll
        for (int g = 0; g < 3; ++g) step_load<T, V>(static_cast<const T*>(pr.px) + ((int64_t)n * 3 + g) * D + d, p[g]);
    }
    step_store<float, V>(state, h);
    if (bad && pr.status) atomicOr(pr.status, kStatusNonFinite);
}

bool bad_sizes(int64_t B, int64_t T, int64_t D) {
    return B < 0 || T < 0 || D < 0 || B >= (int64_t(1) << 31) || T > (int64_t(1) << 30) || B * T >= (int64_t(1) << 31) ||
           D > (int64_t(1) << 29) || (double)B * T * D > 4.0e12 || (double)B * D > 1.0e11;
}
int64_t n_checkpoints(int64_t T) { return (T + kCkSteps - 1) / kCkSteps; }

// ---- launches -------------------------------------------------------------------
namespace {

// Blocks per cluster: the smallest power of two that fills the device's SMs twice
// (two blocks are resident per SM), as far as there are tiles for them.  Its bound without the
// device, which has 148 of the kMostSms SMs that the clusters are made for, sizes the workspace.
constexpr int kMostSms = 256;
int ranks_for(int64_t groups, int64_t tiles, int sms) {
    sms = std::min(sms, kMostSms);
    int c = 1;
    while (c < kMaxRanks && c < tiles && groups * c * 2 <= 2 * (int64_t)sms) c *= 2;
    return c;
}

template <auto kern, int kThreadCount, class P, class Map>
pararnn_status launch_clusters(const char* who, const P& pr, const Map& map, int64_t blocks, int ranks,
                               size_t smem, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (!abi::prepare_kernel(kern, smem, done)) return abi::cuda_fail(who, "kernel attributes not accepted");
    return abi::launch(who, kern, dim3((unsigned)blocks), kThreadCount, smem, st, ranks, pr, map);
}

constexpr std::true_type yes{};
constexpr std::false_type no{};

// calls f with two truth values as types
template <class F>
void choose(bool a, bool b, F f) {
    auto one = [&](auto x) { b ? f(x, std::true_type{}) : f(x, std::false_type{}); };
    a ? one(std::true_type{}) : one(std::false_type{});
}

// two blocks share an SM's 228 KB, of which each gives 1 KB to the system
constexpr size_t kHalfSm = (228 * 1024) / 2 - 1024;
static_assert(sizeof(FwdSmem<float, true>) + 128 <= kHalfSm && sizeof(FwdSmem<bf16, true>) + 128 <= kHalfSm);
static_assert(sizeof(BwdSmem<float, true>) + 128 <= kHalfSm && sizeof(BwdSmem<bf16, true>) + 128 <= kHalfSm);

// Ranges of T: only up to kSegGroups channel groups (which bounds the workspace whatever the device
// is), as many as bring two blocks to each SM with clusters of 8, of two rounds at least; with
// fewer than three the second reading costs what the SMs gain.
constexpr int kSegGroups = 16, kMaxSegs = 32, kMinSegs = 3;
int64_t groups_of(int64_t B, int64_t D) { return B * ((D + kW - 1) / kW); }
size_t elems_bytes(int64_t B, int64_t D) {
    const int64_t groups = groups_of(B, D);
    return groups <= kSegGroups ? (size_t)(groups * (kMaxSegs + 1)) * 32 * sizeof(float4) : 0;
}
// The adjoint's partial sums: a row for each block of a channel group, as many as plan() can come to.  (Eight
// for each would be 2 GB, of which it used 0.3, for 65536 sequences of 32 steps and 1024 channels.)
size_t part_bytes(int64_t B, int64_t T, int64_t D) {
    typedef Tile<float, false, false> Tl;  // of L steps for every type
    const int64_t tiles = (T + Tl::L - 1) / Tl::L;
    const int ranks = ranks_for(groups_of(B, D), tiles, kMostSms);
    const bool cut = elems_bytes(B, D) && tiles > (2 * kMinSegs - 1) * kMaxRanks;
    return (size_t)(B * D * (cut ? kMaxSegs : 1)) * ranks * sizeof(float);
}

// the grid of either kernel: channel groups, ranges of T, and blocks for each of them
template <class P>
bool plan(P& pr, int L, bool may_cut, int64_t& blocks) {
    const int sms = abi::sm_count();
    pr.nCG = (int)((pr.D + kW - 1) / kW);
    pr.nCk = (int)n_checkpoints(pr.T);
    const int64_t groups = pr.B * pr.nCG, tiles = (pr.T + L - 1) / L;
    pr.ranks = ranks_for(groups, tiles, sms);
    const int rounds = (int)((tiles + pr.ranks - 1) / pr.ranks);
    int segs = 1;
    if (may_cut && groups <= kSegGroups && pr.ranks == kMaxRanks) {
        segs = (int)std::min<int64_t>(std::min<int64_t>(2 * sms / (groups * pr.ranks), rounds / 2), kMaxSegs);
        if (segs < kMinSegs) segs = 1;
    }
    pr.seg_rounds = (rounds + segs - 1) / segs;
    pr.segs = (rounds + pr.seg_rounds - 1) / pr.seg_rounds;
    blocks = groups * pr.segs * pr.ranks;
    return sms > 0 && blocks < (int64_t(1) << 31);
}

template <typename T, bool kTma>
pararnn_status launch_backward(const char* who, BwdParams pr, float* dlam, cudaStream_t st) {
    typedef Tile<T, false, kTma> Tl;
    constexpr bool bf = sizeof(T) == 2;
    int64_t blocks;
    if (!plan(pr, Tl::L, true, blocks)) return abi::cuda_fail(who, "device query failed, or too many channel groups");
    BwdMaps maps;
    memset(&maps, 0, sizeof maps);
    pararnn_status s = PARARNN_OK;
    if (kTma) {
        s = encode_steps_map(&maps.pr, pr.px, bf, pr.D, 3, pr.T, pr.B, kW, 1, Tl::L);
        if (s == PARARNN_OK) s = encode_steps_map(&maps.ix, pr.px, bf, pr.D, 3, pr.T, pr.B, kW, 2, Tl::L);
        if (s == PARARNN_OK) s = encode_steps_map(&maps.g, pr.dH, bf, pr.D, 1, pr.T, pr.B, kW, 1, Tl::L);
        if (s == PARARNN_OK) s = encode_steps_map(&maps.out, pr.dpx, bf, pr.D, 3, pr.T, pr.B, kW, 3, Tl::R);
        if (s != PARARNN_OK) return s;
    }
    auto launch_pass = [&](auto c, auto m, auto sum) {
        s = launch_clusters<backward_kernel<T, kTma, decltype(c)::value, decltype(m)::value, decltype(sum)::value>,
                            Tl::NW * 32>(who, pr, maps, blocks, pr.ranks, sizeof(BwdSmem<T, kTma>) + 128, st);
    };
    if (pr.segs > 1) pr.reset ? launch_pass(yes, yes, yes) : launch_pass(yes, no, yes);
    if (s == PARARNN_OK) choose(pr.ranks > 1, pr.reset != nullptr, [&](auto c, auto m) { launch_pass(c, m, no); });
    if (s != PARARNN_OK || !dlam) return s;
    return abi::launch(who, dlam_kernel, dim3((unsigned)((pr.D + 31) / 32)), kSumWarps * 32, 0, st, 1,
                       (const float*)pr.part, pr.lam, dlam, pr.B * pr.segs * pr.ranks, pr.D);
}

template <typename T, bool kTma>
pararnn_status launch_forward(const char* who, Params pr, cudaStream_t st) {
    typedef Tile<T, true, kTma> Tl;
    int64_t blocks;
    if (!plan(pr, Tl::L, pr.elems != nullptr, blocks))
        return abi::cuda_fail(who, "device query failed, or too many channel groups");
    CUtensorMap map;
    memset(&map, 0, sizeof map);
    pararnn_status s = PARARNN_OK;
    if (kTma) s = encode_steps_map(&map, pr.px, sizeof(T) == 2, pr.D, 3, pr.T, pr.B, kW, 3, Tl::L);
    if (s != PARARNN_OK) return s;
    auto launch_pass = [&](auto c, auto m, auto sum) {
        s = launch_clusters<forward_kernel<T, kTma, decltype(c)::value, decltype(m)::value, decltype(sum)::value>,
                            Tl::NW * 32>(who, pr, map, blocks, pr.ranks, sizeof(FwdSmem<T, kTma>) + 128, st);
    };
    if (pr.segs > 1) pr.reset ? launch_pass(yes, yes, yes) : launch_pass(yes, no, yes);
    if (s == PARARNN_OK) choose(pr.ranks > 1, pr.reset != nullptr, [&](auto c, auto m) { launch_pass(c, m, no); });
    return s;
}

template <typename T>
pararnn_status launch(const char* who, const Params& pr, cudaStream_t st) {
    const bool tma = (pr.D * sizeof(T)) % 16 == 0 && !abi::misaligned(pr.px, 16) && !abi::misaligned(pr.H, 16) &&
                     !abi::misaligned(pr.ck, 8);
    return tma ? launch_forward<T, true>(who, pr, st) : launch_forward<T, false>(who, pr, st);
}
template <typename T>
pararnn_status launch(const char* who, const BwdParams& pr, float* dlam, cudaStream_t st) {
    const bool tma = (pr.D * sizeof(T)) % 16 == 0 && !abi::misaligned(pr.px, 16) && !abi::misaligned(pr.dH, 16) &&
                     !abi::misaligned(pr.dpx, 16) && !abi::misaligned(pr.ck, 8);
    return tma ? launch_backward<T, true>(who, pr, dlam, st) : launch_backward<T, false>(who, pr, dlam, st);
}

template <typename T>
pararnn_status launch_step(const char* who, StepParams pr, cudaStream_t st) {
    const bool quads = pr.D % 4 == 0 && !abi::misaligned(pr.px, 4 * sizeof(T)) && !abi::misaligned(pr.y, 4 * sizeof(T)) &&
                       !abi::misaligned(pr.lam, 16) && !abi::misaligned(pr.state, 16);
    const int64_t per = kStepThreads * (quads ? 4 : 1), chunks = (pr.D + per - 1) / per;
    if (chunks > 65535) return abi::fail(who, "too many channels");
    const int64_t N = pr.N;
    // rows of a later launch come after those of an earlier one, as the order of rows wants it
    for (int64_t n = 0; n < N; n += kStepRows) {
        pr.N = N - n < kStepRows ? N - n : kStepRows;
        const dim3 grid((unsigned)pr.N, (unsigned)chunks);
        const pararnn_status s =
            abi::launch(who, quads ? step_kernel<T, 4> : step_kernel<T, 1>, grid, kStepThreads, 0, st, 1, pr);
        if (s != PARARNN_OK) return s;
        pr.px = static_cast<const T*>(pr.px) + kStepRows * 3 * pr.D;
        pr.y = static_cast<T*>(pr.y) + kStepRows * pr.D;
        if (pr.slots)
            pr.slots += kStepRows;
        else
            pr.state += kStepRows * pr.D, pr.n_slots -= kStepRows;
    }
    return PARARNN_OK;
}

}  // namespace
}  // namespace gs
}  // namespace pararnn

using namespace pararnn;

extern "C" {

size_t pararnn_gated_scan_checkpoint_bytes(int64_t B, int64_t T, int64_t D, pararnn_dtype dtype) {
    if (gs::bad_sizes(B, T, D) || abi::bad_dtype(dtype)) return 0;
    return (size_t)(B * gs::n_checkpoints(T) * D) * sizeof(float);
}

size_t pararnn_gated_scan_workspace_bytes(int64_t B, int64_t T, int64_t D) {
    if (gs::bad_sizes(B, T, D)) return 0;
    if (B == 0 || T == 0 || D == 0) return kHeaderBytes;
    return kHeaderBytes + gs::elems_bytes(B, D) + gs::part_bytes(B, T, D);
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
    const size_t elems = gs::elems_bytes(B, D);
    if (elems && workspace && ws_bytes >= kHeaderBytes + elems)
        pr.elems = reinterpret_cast<float4*>(static_cast<char*>(workspace) + kHeaderBytes);
    pr.status = static_cast<unsigned*>(workspace);
    pr.B = B;
    pr.T = T;
    pr.D = D;
    pr.decay = decay;
    return dtype == PARARNN_F32 ? gs::launch<float>(who, pr, st) : gs::launch<gs::bf16>(who, pr, st);
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
    pr.elems = reinterpret_cast<float4*>(static_cast<char*>(workspace) + kHeaderBytes);
    pr.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeaderBytes + gs::elems_bytes(B, D));
    pr.dh0 = dL_dh0;
    pr.status = static_cast<unsigned*>(workspace);
    pr.B = B;
    pr.T = T;
    pr.D = D;
    pr.decay = decay;
    return dtype == PARARNN_F32 ? gs::launch<float>(who, pr, dL_dlambda, st)
                                : gs::launch<gs::bf16>(who, pr, dL_dlambda, st);
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
    return dtype == PARARNN_F32 ? gs::launch_step<float>(who, pr, st) : gs::launch_step<gs::bf16>(who, pr, st);
}

}  // extern "C"
