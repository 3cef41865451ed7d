// kda_glr_common.cuh -- what the kernels of the gated linear recurrence share: its step, a warp's tiles of tokens and channels,
// the sequences that start and end among a warp's tokens, and the exchange between the blocks of a cluster.
//
//   h_t = a_t h_{t-1} + s_t x_t,   a_t = exp(g_t) or 1 / (1 + exp(-g_t)),   s_t = 1 or 1 - a_t
//
// The step is taken with n_t = a_t - 1, h_t = h_{t-1} + n_t h_{t-1} + s_t x_t (an fma and an addition).  A decay near 1 is what
// gives a channel its memory of 1 / -n tokens: a rounded to fp32 is off by 2^-25, which the memory multiplies to 2^-25 / -n of the
// state, while n itself is held to 2^-20 of its value.  Below a decay of 1/2 this form is off by 2^-25 of the state before, more than a
// rounding of the little that is left of it: the single token takes a_t h_{t-1} there, a stretch is no better than its N (next).
// Tokens i..j together are a pair (N, H): h_j = h_{i-1} + N h_{i-1} + H, where N = a_i .. a_j - 1 grows by N += n (1 + N).  Where little
// of h_{i-1} is left, N's roundings near -1 are what stands for it, 2^-25 of h_{i-1}: relative to the states of the stretch, 128 tokens at most.
// The product of the decays beside N would be good to 2^-24 of what is left, for a third operation a join and registers that are not there.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "kda_gdn_ptx.cuh"
#include "kda_glr_internal.h"
#include "kda_glr_room.h"

namespace kda {

constexpr int kGlrWarps = 8;  // of a block: consecutive stretches of time; a cluster's blocks have consecutive chunks of it
constexpr int kGlrThreads = 32 * kGlrWarps;

// ------------------------------------------------------- a thread's channels --
// V channels beside each other, and their arithmetic in fp32: two at once in one instruction (fma, mul and add of f32x2 take
// one issue slot for two, and issue is what these kernels run out of beside HBM), held as the register pair that it takes.
template <int V>
struct Lanes;
template <>
struct Lanes<1> {
    float p;
};
template <>
struct Lanes<2> {
    uint64_t p;
};
__device__ __forceinline__ Lanes<2> lanes_of(float x, float y) {
    Lanes<2> r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.p) : "f"(x), "f"(y));
    return r;
}
// f of each channel, or of each channel of two
template <typename F>
__device__ __forceinline__ Lanes<1> each(const Lanes<1>& a, const F& f) { return {f(a.p)}; }
template <typename F>
__device__ __forceinline__ Lanes<2> each(const Lanes<2>& a, const F& f) {
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.p));
    return lanes_of(f(x), f(y));
}
template <typename F>
__device__ __forceinline__ Lanes<1> each(const Lanes<1>& a, const Lanes<1>& b, const Lanes<1>& c, const F& f) { return {f(a.p, b.p, c.p)}; }
template <typename F>
__device__ __forceinline__ Lanes<2> each(const Lanes<2>& a, const Lanes<2>& b, const Lanes<2>& c, const F& f) {
    float x[3], y[3];
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x[0]), "=f"(y[0]) : "l"(a.p));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x[1]), "=f"(y[1]) : "l"(b.p));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x[2]), "=f"(y[2]) : "l"(c.p));
    return lanes_of(f(x[0], x[1], x[2]), f(y[0], y[1], y[2]));
}
template <int V>
__device__ __forceinline__ Lanes<V> lanes(float x) {
    if constexpr (V == 1) return {x};
    else return lanes_of(x, x);
}
__device__ __forceinline__ Lanes<2> fma(const Lanes<2>& a, const Lanes<2>& b, const Lanes<2>& c) {
    Lanes<2> r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.p) : "l"(a.p), "l"(b.p), "l"(c.p));
    return r;
}
__device__ __forceinline__ Lanes<2> mul(const Lanes<2>& a, const Lanes<2>& b) {
    Lanes<2> r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.p) : "l"(a.p), "l"(b.p));
    return r;
}
__device__ __forceinline__ Lanes<2> add(const Lanes<2>& a, const Lanes<2>& b) {
    Lanes<2> r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.p) : "l"(a.p), "l"(b.p));
    return r;
}
__device__ __forceinline__ Lanes<1> fma(const Lanes<1>& a, const Lanes<1>& b, const Lanes<1>& c) { return {fmaf(a.p, b.p, c.p)}; }
__device__ __forceinline__ Lanes<1> mul(const Lanes<1>& a, const Lanes<1>& b) { return {__fmul_rn(a.p, b.p)}; }
__device__ __forceinline__ Lanes<1> add(const Lanes<1>& a, const Lanes<1>& b) { return {__fadd_rn(a.p, b.p)}; }

__device__ __forceinline__ float glr_f32(float x) { return x; }
__device__ __forceinline__ float glr_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void glr_round(float& d, float x) { d = x; }
__device__ __forceinline__ void glr_round(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
// The channels of a row as they are in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) GlrVec {
    T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Lanes<V> wide(const GlrVec<T, V>& x) {
    if constexpr (V == 1) return {glr_f32(x.e[0])};
    else return lanes_of(glr_f32(x.e[0]), glr_f32(x.e[1]));
}
// The same with the signs turned over.
template <typename T, int V>
__device__ __forceinline__ Lanes<V> wide_negative(const GlrVec<T, V>& x) {
    if constexpr (V == 2 && sizeof(T) == 2) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&x) ^ 0x80008000u;
        return wide(*reinterpret_cast<const GlrVec<T, V>*>(&u));
    } else {
        return each(wide(x), [](float y) { return -y; });
    }
}
template <typename T, int V>
__device__ __forceinline__ GlrVec<T, V> narrow(const Lanes<V>& x) {
    GlrVec<T, V> r;
    if constexpr (V == 1) {
        glr_round(r.e[0], x.p);
    } else {
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.p));
        if constexpr (sizeof(T) == 2) {
            const uint32_t u = pack_bf16(lo, hi);
            r = *reinterpret_cast<const GlrVec<T, V>*>(&u);
        } else {
            r.e[0] = lo;
            r.e[1] = hi;
        }
    }
    return r;
}
// fp32 states of V channels; zeros where there are none.
template <int V>
__device__ __forceinline__ Lanes<V> glr_state(const float* p, int64_t at, bool live) {
    if (!p || !live) return lanes<V>(0.f);
    return wide(*reinterpret_cast<const GlrVec<float, V>*>(p + at));
}
template <int V>
__device__ __forceinline__ void glr_put(float* p, int64_t at, const Lanes<V>& x) {
    *reinterpret_cast<GlrVec<float, V>*>(p + at) = narrow<float, V>(x);
}

// ------------------------------------------------------------------- gates ----
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <int V>
struct GlrGate {
    Lanes<V> n;      // a - 1
    Lanes<V> slope;  // da / dg (asked for by SLOPE)
    Lanes<V> e;      // e^g (with the sigmoid or SLOPE)
};
// The gates of a row.  Where e^g is corrected (below) they are held to where it is finite and what that loses is below fp32's normal range:
// -150 and, of the sigmoid, 88.  bf16 pairs in one instruction a bound.
template <bool SIGMOID, bool SLOPE, typename G, int V>
__device__ __forceinline__ Lanes<V> glr_gates(const GlrVec<G, V>& gate) {
    if constexpr (!SIGMOID && !SLOPE) {
        return wide(gate);
    } else if constexpr (V == 2 && sizeof(G) == 2) {
        uint32_t u = *reinterpret_cast<const uint32_t*>(&gate);
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0xc316c316u));
        if (SIGMOID) asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0x42b042b0u));
        return wide(*reinterpret_cast<const GlrVec<G, V>*>(&u));
    } else {
        return each(wide(gate), [](float x) {
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-150.f));
            if (SIGMOID) asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(88.f));
            return x;
        });
    }
}
// n and the slope are good to 2^-20 of their value, of what glr_gates gave.  The rounded product g log2(e) makes e^g off by |g| 2^-24 of its value:
// of e^g - 1 with g below 0 that is little (|g| e^g is below 0.4), and a log gate above 0 keeps it; the sigmoid, whose 1 - a is e^-g far
// above 0, and the slopes are given what the product lost (8192 x 4096 bf16, sigmoid: 56.4 us with cold caches, without 54.4).
template <bool SIGMOID, bool SLOPE, int V>
__device__ __forceinline__ GlrGate<V> glr_gate(const Lanes<V>& g) {
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kRest = -1.9046542e-9f;  // ln(2) is kLn2 + kRest
    GlrGate<V> r;
    const Lanes<V> t = mul(g, lanes<V>(-kLog2e));
    const Lanes<V> e = each(t, [](float x) { return ex2(-x); });
    if constexpr (SIGMOID || SLOPE) r.e = fma(e, fma(t, lanes<V>(kRest), fma(t, lanes<V>(kLn2), g)), e);  // 2^-t e^(g + t ln(2))
    if constexpr (SIGMOID) {
        r.n = each(fma(r.e, lanes<V>(-1.f), lanes<V>(-1.f)), [](float x) { return rcp(x); });
    } else {
        // expm1(g): below 1/4 the first six terms of its series (the seventh is 5e-8 of the sum)
        Lanes<V> p = fma(g, lanes<V>(1.f / 720), lanes<V>(1.f / 120));
        p = fma(g, p, lanes<V>(1.f / 24));
        p = fma(g, p, lanes<V>(1.f / 6));
        p = fma(g, p, lanes<V>(0.5f));
        p = fma(g, p, lanes<V>(1.f));
        r.n = each(g, mul(g, p), add(e, lanes<V>(-1.f)), [](float x, float near, float far) { return fabsf(x) < 0.25f ? near : far; });
    }
    if constexpr (SLOPE) r.slope = SIGMOID ? mul(mul(r.n, r.e), r.n) : r.e;  // a (1 - a), with a = e^g (1 - a)
    return r;
}

// ------------------------------------------------------------- (N, H) pairs ----
template <int V>
struct alignas(8 * V) GlrStretch {
    Lanes<V> n, h;
};
template <int V>
__device__ __forceinline__ Lanes<V> glr_step(const Lanes<V>& h, const Lanes<V>& n, const Lanes<V>& v) {
    return add(fma(n, h, h), v);
}
template <int V>
__device__ __forceinline__ Lanes<V> glr_join(const Lanes<V>& n, const Lanes<V>& next) {  // of two stretches' N
    return fma(next, add(n, lanes<V>(1.f)), n);
}
// The state behind a stretch of tokens from the one before it; `cut`: a sequence starts in the stretch (backwards: ends), so
// that nothing of the state before it is left, not even where that is not finite.
template <int V>
__device__ __forceinline__ Lanes<V> glr_through(const Lanes<V>& h, const GlrStretch<V>& s, bool cut) {
    const Lanes<V> through = glr_step(h, s.n, s.h);
    return {cut ? s.h.p : through.p};
}
// Pairs of a block's warps for 32 x V channels, and the stretches that are cut.  The cluster's blocks' are kept twice, by turns: another
// block may be a round ahead.
template <int V>
struct GlrExchange {
    GlrStretch<V> warp[kGlrWarps][32];
    int32_t warp_cut[kGlrWarps];
    int32_t flags[2][32];  // by turns as well: the blocks' cuts and, last, whether a wait of this block has expired
    uint64_t come[2];      // what the blocks send in a round has come
};
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Stores into another block of the cluster, counted in bytes on the barrier `bar` of that block.
__device__ __forceinline__ void cluster_send(uint32_t addr, uint32_t bar, const GlrStretch<2>& x) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(addr), "l"(x.n.p), "l"(x.h.p),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_send(uint32_t addr, uint32_t bar, const GlrStretch<1>& x) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(x.n.p), "f"(x.h.p),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_send(uint32_t addr, uint32_t bar, int32_t x) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.s32 [%0], %1, [%2];" ::"r"(addr), "r"(x), "r"(bar) : "memory");
}
// Before the first round; every thread of every block.  All have begun, and their barriers are set, before one sends to another.
template <int V>
__device__ __forceinline__ void glr_exchange_start(GlrExchange<V>& ex, int blocks) {
    if (threadIdx.x == 0) {
        mbar_init(&ex.come[0], 1);
        mbar_init(&ex.come[1], 1);
        fence_mbar_init();
    }
    if (threadIdx.x < 64) ex.flags[threadIdx.x >> 5][threadIdx.x & 31] = 0;
    __syncthreads();
    if (blocks > 1) cluster_sync();
}
// A warp's wait for a phase.  Where it expires the rounds end, for all of the block's warps at once: they read the flag of a round behind
// its second barrier, so it is set for a round whose first barrier is to come.
__device__ __forceinline__ void glr_wait(uint64_t* bar, uint32_t parity, int32_t (&flags)[32], int32_t* device_status) {
    if (__all_sync(~0u, mbar_wait_pipe(bar, parity))) return;
    if ((threadIdx.x & 31) == 0) {
        *reinterpret_cast<volatile int32_t*>(&flags[31]) = 1;
        if (device_status) atomicOr(device_status, KDA_DEV_TIMEOUT);
    }
}
// Behind the last round; whole warps: whether a wait expired.  A block whose has may still be sent to, so it stays until the cluster's others
// are here as well; rounds that went to their end leave nothing to wait for.
template <int V, typename F>
__device__ __forceinline__ void glr_exchange_end(const GlrExchange<V>& ex, int blocks, const F& drain) {
    const volatile int32_t* flags = &ex.flags[0][31];
    const bool stopped = __any_sync(~0u, (flags[0] | flags[32]) != 0);
    if (stopped) {
        drain();
        __syncwarp();
    }
    if (blocks == 1) return;
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (stopped) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The block's warps' pairs in the order of time: those before this warp together in `ahead`, all in `sum`.
template <int V, bool BACK, bool CUT>
__device__ __forceinline__ void glr_fold(const GlrExchange<V>& ex, GlrStretch<V>& ahead, GlrStretch<V>& sum, bool& ahead_cut, bool& any) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    sum = ahead = {lanes<V>(0.f), lanes<V>(0.f)};
    any = ahead_cut = false;
#pragma unroll
    for (int i = 0; i < kGlrWarps; ++i) {
        const int w = BACK ? kGlrWarps - 1 - i : i;
        if (w == warp) {
            ahead = sum;
            ahead_cut = any;
        }
        const GlrStretch<V> s = ex.warp[w][lane];
        const bool cut = CUT && ex.warp_cut[w] != 0;
        sum.h = CUT ? glr_through(sum.h, s, cut) : glr_step(sum.h, s.n, s.h);
        sum.n = glr_join(sum.n, s.n);
        any |= cut;
    }
}
// All warps of every block of the cluster, with the warp's pair and cut; BACK: time runs backwards, from the last warp and block
// to the first.  `carry` is the state before the whole round, and becomes the one behind it; `before` gets the state before this warp.
// `between()` runs where shared memory that the block's warps wrote before the call can be read, and is not written again.  A block that
// is here for round r + 2 has had what the others sent in round r + 1, so they have read what they had in round r.
// False, in all of the block's warps: a wait of theirs expired, for this round's tiles or in the round before.  Nothing is stored then, and
// the block leaves, so that it does not give up once a round.
template <uint32_t TILES, int V, bool BACK, typename F>
__device__ __forceinline__ bool glr_exchange(GlrExchange<V>& ex, int rank, int blocks, int32_t round, const GlrStretch<V>& pair, bool cut,
                                             Lanes<V>& carry, Lanes<V>& before, int32_t* device_status, const F& between) {
    extern __shared__ __align__(128) uint8_t tiles[];
    // the blocks' pairs stand behind the tiles, where they take as much as there are blocks
    GlrStretch<V>(*const block)[2][32] = reinterpret_cast<GlrStretch<V>(*)[2][32]>(tiles + TILES);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = round & 1;
    ex.warp[warp][lane] = pair;
    if (lane == 0) ex.warp_cut[warp] = cut;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&ex.come[turn], blocks * (32 * sizeof(GlrStretch<V>) + 4));
    const bool cuts = __syncthreads_or(cut);
    GlrStretch<V> ahead, sum;
    bool ahead_cut, any;
    if (cuts) glr_fold<V, BACK, true>(ex, ahead, sum, ahead_cut, any);
    else glr_fold<V, BACK, false>(ex, ahead, sum, ahead_cut, any);  // most stretches are not cut
    const auto send = [&](int to) {
        const uint32_t bar = cluster_address(smem_u32(&ex.come[turn]), to);
        cluster_send(cluster_address(smem_u32(&block[rank][turn][lane]), to), bar, sum);
        if (lane == 0) cluster_send(cluster_address(smem_u32(&ex.flags[turn][rank]), to), bar, static_cast<int32_t>(any));
    };
    static_assert(kGlrMaxCluster == 2 * kGlrWarps, "a warp sends to two blocks");
    if (warp < blocks) send(warp);
    if (warp + kGlrWarps < blocks) send(warp + kGlrWarps);
    between();
    __syncthreads();  // ex.warp has been read
    glr_wait(&ex.come[turn], round >> 1 & 1, ex.flags[turn ^ 1], device_status);
    const uint32_t block_cuts = __ballot_sync(~0u, *reinterpret_cast<volatile int32_t*>(&ex.flags[turn][lane]) != 0);
    if (block_cuts >> 31) return false;
    before = carry;  // the state before this block
    constexpr int kStep = BACK ? -1 : 1;
    GlrStretch<V> next = block[BACK ? blocks - 1 : 0][turn][lane];
    for (int i = 0; i < blocks; ++i) {
        const int b = BACK ? blocks - 1 - i : i;
        const GlrStretch<V> s = next;
        if (i + 1 < blocks) next = block[b + kStep][turn][lane];
        if (b == rank) before = carry;
        carry = block_cuts ? glr_through(carry, s, block_cuts >> b & 1) : glr_step(carry, s.n, s.h);
    }
    before = glr_through(before, ahead, ahead_cut);
    return true;
}

// --------------------------------------------------------------- sequences ----
// The sequences that start or end among tokens [t, t + L) of a warp: a bit for each token, and the sequence by token.
template <int L>
struct GlrMarks {
    int32_t start[kGlrWarps][L], end[kGlrWarps][L];
};
// Where a warp's last look at cu_seqlens ended: the last entry below its tokens, and the first that is not.
struct GlrPlace {
    int32_t below = INT32_MAX, next = INT32_MIN;
};
// Whole warp; rounds go up, or with BACK down, by more than L tokens.  Most tokens are far from a sequence's ends, which `place`
// tells without a look.  Entries of cu_seqlens that are out of order give other marks, none outside the tokens or the sequences.
template <int L, bool BACK>
__device__ __forceinline__ void glr_marks(GlrMarks<L>& marks, GlrPlace& place, const int32_t* __restrict__ cu, int32_t num_seqs,
                                          int32_t t, uint32_t* starts, uint32_t* ends) {
    *starts = *ends = 0;
    if (BACK ? place.below < t : place.next > t + L) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncwarp();
    // the first entry that is not below t, of entries 0..num_seqs: 32 of them looked at in a round
    int32_t lo = 0, left = num_seqs + 1;  // it is one of [lo, lo + left], lo + left where those before are all below t
    while (left > 32) {
        const int32_t step = left / 32;
        const uint32_t below = __ballot_sync(~0u, __ldg(cu + lo + (lane + 1) * step - 1) < t);
        const int skip = __popc(below);  // of sorted entries: the first `skip`
        lo += skip * step;
        left = skip == 32 ? left - 32 * step : step - 1;
    }
    {
        const bool in = lane < left;
        const int32_t v = in ? __ldg(cu + lo + lane) : 0;
        lo += __popc(__ballot_sync(~0u, in && v < t));
    }
    place.below = lo > 0 ? __ldg(cu + lo - 1) : INT32_MIN;
    place.next = lo <= num_seqs ? __ldg(cu + lo) : INT32_MAX;
    uint32_t s = 0, e = 0;
    for (;;) {
        const int32_t m = lo + lane;
        const int32_t v = m <= num_seqs ? __ldg(cu + m) : INT32_MAX;
        const bool near = v >= t && v <= t + L;
        if (near && v < t + L && m < num_seqs && __ldg(cu + m + 1) > v) {
            s |= 1u << (v - t);
            marks.start[warp][v - t] = m;
        }
        if (near && v > t && m > 0 && __ldg(cu + m - 1) < v) {
            e |= 1u << (v - t - 1);
            marks.end[warp][v - t - 1] = m - 1;
        }
        if (__ballot_sync(~0u, near) != ~0u) break;
        lo += 32;
    }
    *starts = __reduce_or_sync(~0u, s);
    *ends = __reduce_or_sync(~0u, e);
    __syncwarp();
}
// cu_seqlens is 0 .. total_tokens, nowhere falling: every thread of the grid looks at its share.
__device__ __forceinline__ void glr_check_sequences(const int32_t* __restrict__ cu, int32_t num_seqs, int32_t total_tokens,
                                                    int32_t* device_status) {
    if (!device_status) return;
    bool ok = true;
    for (int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; m <= num_seqs;
         m += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int32_t v = cu[m];
        ok &= m == 0 ? v == 0 : v >= cu[m - 1];
        if (m == num_seqs) ok &= v == total_tokens;
    }
    if (!ok) atomicOr(device_status, KDA_DEV_BAD_CU_SEQLENS);
}

// ------------------------------------------------------------------- tiles ----
// How a warp's L tokens x 32 V channels come and go.  TMA, where rows are whole multiples of 16 bytes apart: a ring in shared
// memory, a stage a tile of every tensor for all the block's warps; what is read behind the ends is zeros.  Else plain loads, a channel a thread.
// Results go from registers to memory: a tile is free again once it has been read.
struct GlrMaps {
    CUtensorMap in[3];
};
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}
// A block's ring: stage i % STAGES holds round i's tiles, `bytes` together.  One thread fills it.
template <int STAGES>
struct GlrRing {
    uint64_t full[STAGES];
    __device__ __forceinline__ void start() {  // before a barrier
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    // load(stage, barrier, round), once every warp has read what was there
    template <typename L>
    __device__ __forceinline__ void fill(uint8_t* base, uint32_t bytes, int32_t round, const L& load) {
        mbar_arrive_expect_tx(&full[round % STAGES], bytes);
        load(base + round % STAGES * bytes, &full[round % STAGES], round);
    }
    // What was begun, of rounds up to `filled`, has to be over before the block ends.  The thread that filled.
    __device__ __forceinline__ void drain(int32_t filled) {
        for (int32_t i = filled > STAGES ? filled - STAGES : 0; i < filled; ++i)
            (void)mbar_wait(&full[i % STAGES], i / STAGES & 1, kDrainLimit);
    }
};
// A thread's channel of a row in memory, read once; zero where there is none.
template <typename T>
__device__ __forceinline__ T glr_load(const T* p, bool in) {
    if (!in) return T(0.f);
    if constexpr (sizeof(T) == 4) {
        return __ldcs(p);
    } else {
        const uint16_t u = __ldcs(reinterpret_cast<const uint16_t*>(p));
        return *reinterpret_cast<const T*>(&u);
    }
}

// ------------------------------------------------------------------ launch ----
// Tile map of a [tokens, dim] tensor: boxes of `rows` tokens x 64 channels.
bool glr_map(CUtensorMap* m, const void* base, bool f32, int64_t tokens, int32_t dim, int32_t rows);
// Whether the rows of all its tensors are whole multiples of 16 bytes apart.
inline bool glr_tiled(const GlrKind& kind, int32_t dim) { return dim % (kind.x_f32 && kind.gate_f32 ? 4 : 8) == 0; }
// A kernel over `slices` slices of channels with a cluster of blocks on each: as many blocks as have tokens of their own, while all the
// clusters find room beside each other (a training step of 8192 tokens, 2560 channels: 7 blocks 114 us, 4 blocks 150; 64 channels: 16
// blocks 42, 8 blocks 61).  `smem`: bytes of tiles; V: channels of a thread.
template <typename K, typename... A>
inline cudaError_t glr_launch(K kernel, int64_t slices, int64_t tokens, int block_tokens, uint32_t smem, int V, GlrRooms& rooms,
                              cudaStream_t stream, const A&... args) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const auto shape = [&](int n) {
        cfg.gridDim = dim3(static_cast<unsigned>(slices * n));
        cfg.blockDim = dim3(kGlrThreads);
        cfg.dynamicSmemBytes = smem + static_cast<uint32_t>(n * 2 * 32 * 8 * V);
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = n;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    };
    GlrRoom room;
    err = rooms.get(dev, [&](GlrRoom* r) {
        shape(kGlrMaxCluster);
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        for (int n = 1; e == cudaSuccess && n <= kGlrMaxCluster; ++n) {
            shape(n);
            e = cudaOccupancyMaxActiveClusters(&r->clusters[n], kernel, &cfg);
        }
        return e;
    }, &room);
    if (err != cudaSuccess) return err;
    int blocks = static_cast<int>(std::min<int64_t>(kGlrMaxCluster, std::max<int64_t>(1, (tokens + block_tokens - 1) / block_tokens)));
    while (blocks > 1 && slices > room.clusters[blocks]) --blocks;
    shape(blocks);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Calls f<x type, gate type, sigmoid, complement>() of a call's kind.
#define KDA_GLR_BY_KIND(kind, F, ...)                                                                            \
    [&]() -> cudaError_t {                                                                                       \
        const bool sg = ((kind).flags & KDA_GLR_SIGMOID) != 0, cm = ((kind).flags & KDA_GLR_COMPLEMENT) != 0;    \
        using bf = __nv_bfloat16;                                                                                \
        if ((kind).x_f32)                                                                                        \
            return sg ? (cm ? F<float, float, true, true>(__VA_ARGS__) : F<float, float, true, false>(__VA_ARGS__)) \
                      : (cm ? F<float, float, false, true>(__VA_ARGS__) : F<float, float, false, false>(__VA_ARGS__)); \
        if ((kind).gate_f32)                                                                                     \
            return sg ? (cm ? F<bf, float, true, true>(__VA_ARGS__) : F<bf, float, true, false>(__VA_ARGS__))    \
                      : (cm ? F<bf, float, false, true>(__VA_ARGS__) : F<bf, float, false, false>(__VA_ARGS__)); \
        return sg ? (cm ? F<bf, bf, true, true>(__VA_ARGS__) : F<bf, bf, true, false>(__VA_ARGS__))              \
                  : (cm ? F<bf, bf, false, true>(__VA_ARGS__) : F<bf, bf, false, false>(__VA_ARGS__));           \
    }()

}  // namespace kda
