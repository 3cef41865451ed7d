// kda_glr.cu -- gated linear recurrence over packed sequences, and its single token.
//
//   h_t = a_t h_{t-1} + s_t x_t   for every channel by itself (kda_glr_common.cuh has the step and its rounding)
//
// Bound by HBM: x and the gates are read once and h is written once.  A cluster owns 32 V channels for all tokens and goes
// through them in rounds of (blocks x 8 warps x L) tokens, a thread V channels of L tokens: it takes them to
// registers, scans them from a zero state, and once the pairs of all warps and blocks before it are known (shared memory, then
// the cluster's) adds what comes in.  One pass, no second reading and no waiting on other clusters; sums are taken in a fixed
// order, so results are bitwise repeatable.  12345 tokens x 4096 channels, bf16 with fp32 gates: 84 us, 4.8 TB/s of 6.8; what is left is a
// round's chain (tile, gates, scan, exchange, outputs: 3.4 us with two blocks an SM) and that 256 blocks find 304 places.

#include <limits>

#include "kda_glr_common.cuh"

namespace kda {
namespace {

template <typename X, typename G, bool TMA>
struct Form {
    static constexpr int V = TMA ? 2 : 1;
    static constexpr int L = sizeof(X) + sizeof(G) == 8 ? 8 : 16;  // tokens of a thread in a round: as many as registers hold
    static constexpr int kBlockTokens = kGlrWarps * L;
    static constexpr uint32_t kTileX = kBlockTokens * 64 * sizeof(X), kTileG = kBlockTokens * 64 * sizeof(G), kStage = kTileX + kTileG;
    static constexpr int kStages = sizeof(X) + sizeof(G) == 6 ? 2 : 3;
    static constexpr uint32_t kSmem = TMA ? kStages * kStage : 0;
    static_assert(kBlockTokens % kGlrCheckpoint == 0 && kGlrCheckpoint % L == 0, "checkpoints stand before a warp's tokens");
};

template <typename X, typename G, bool TMA, bool SIGMOID, bool COMPLEMENT>
__global__ void __launch_bounds__(kGlrThreads, 2) kda_glr_prefill_kernel(const __grid_constant__ GlrMaps maps, const GlrArgs a) {
    using F = Form<X, G, TMA>;
    constexpr int V = F::V, L = F::L;
    extern __shared__ __align__(128) uint8_t tiles[];
    __shared__ GlrExchange<V> ex;
    __shared__ GlrMarks<L> marks;
    __shared__ GlrRing<F::kStages> ring;
    const int rank = cluster_rank(), blocks = cluster_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t T = a.total_tokens;
    const int64_t dim = a.dim, ch0 = static_cast<int64_t>(blockIdx.x / blocks) * 32 * V, ch = ch0 + lane * V;
    const bool live = ch < dim;  // V divides dim
    const int32_t step = blocks * F::kBlockTokens;
    const int32_t block_t = rank * F::kBlockTokens, t0 = block_t + warp * L;  // of the first round
    glr_check_sequences(a.cu_seqlens, a.num_seqs, T, a.device_status);
    if (TMA && threadIdx.x == 0) ring.start();
    glr_exchange_start(ex, blocks);
    const bool copies = TMA && warp == kGlrWarps - 1 && lane == 0;
    int32_t filled = 0;
    const auto load = [&](uint8_t* at, uint64_t* bar, int32_t round) {
        tma_load_2d(at, &maps.in[0], bar, static_cast<int32_t>(ch0), block_t + round * step);
        tma_load_2d(at + F::kTileX, &maps.in[1], bar, static_cast<int32_t>(ch0), block_t + round * step);
    };
    if (copies)
        for (; filled < F::kStages && filled * step < T; ++filled) ring.fill(tiles, F::kStage, filled, load);
    Lanes<V> carry = lanes<V>(0.f);
    GlrPlace place;
    for (int32_t round = 0, at = 0; at < T; ++round, at += step) {
        const int32_t t = t0 + at;
        uint32_t starts, ends;
        glr_marks<L, false>(marks, place, a.cu_seqlens, a.num_seqs, t, &starts, &ends);
        Lanes<V> n[L], h[L];  // a - 1 and the weighted input, then the pairs of the tokens up to and with each
        if constexpr (TMA) {
            glr_wait(&ring.full[round % F::kStages], round / F::kStages & 1, ex.flags[round & 1], a.device_status);
            const uint8_t* stage = tiles + round % F::kStages * F::kStage;
            const GlrVec<X, V>* tile = reinterpret_cast<const GlrVec<X, V>*>(stage) + warp * L * 32 + lane;
            const GlrVec<G, V>* gates = reinterpret_cast<const GlrVec<G, V>*>(stage + F::kTileX) + warp * L * 32 + lane;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                h[i] = COMPLEMENT ? wide_negative(tile[i * 32]) : wide(tile[i * 32]);
                n[i] = glr_gates<SIGMOID, false>(gates[i * 32]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool in = live && t + i < T;
                h[i].p = (COMPLEMENT ? -1.f : 1.f) * glr_f32(glr_load(static_cast<const X*>(a.x) + (t + i) * dim + ch, in));
                n[i] = glr_gates<SIGMOID, false>(GlrVec<G, 1>{glr_load(static_cast<const G*>(a.gate) + (t + i) * dim + ch, in)});
            }
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            n[i] = glr_gate<SIGMOID, false>(n[i]).n;
            if (COMPLEMENT) h[i] = mul(n[i], h[i]);  // its sign was turned over
        }
        // a sequence's first token takes its state from h0; then from a zero state
        if (starts) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool cut = starts >> i & 1;
                if (cut) h[i] = glr_step(glr_state<V>(a.h0, marks.start[warp][i] * dim + ch, live), n[i], h[i]);
                if (i > 0) {
                    h[i] = glr_through(h[i - 1], {n[i], h[i]}, cut);
                    n[i] = glr_join(n[i - 1], n[i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 1; i < L; ++i) {
                h[i] = glr_step(h[i - 1], n[i], h[i]);
                n[i] = glr_join(n[i - 1], n[i]);
            }
        }
        Lanes<V> before;
        if (!glr_exchange<F::kSmem, V, false>(ex, rank, blocks, round, {n[L - 1], h[L - 1]}, starts != 0, carry, before, a.device_status, [&] {
                if (copies && filled * step < T) ring.fill(tiles, F::kStage, filled++, load);
            }))
            break;
        if (a.checkpoints && live && t % kGlrCheckpoint == 0 && t < T) glr_put(a.checkpoints, t / kGlrCheckpoint * dim + ch, before);
        if (starts) {
            bool cut = false;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                cut |= starts >> i & 1;
                h[i] = glr_through(before, {n[i], h[i]}, cut);
            }
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) h[i] = glr_step(before, n[i], h[i]);
        }
        if (a.h && live) {
            X* to = static_cast<X*>(a.h) + t * dim + ch;
            if (t + L <= T) {
#pragma unroll
                for (int i = 0; i < L; ++i, to += dim) *reinterpret_cast<GlrVec<X, V>*>(to) = narrow<X, V>(h[i]);
            } else {
#pragma unroll
                for (int i = 0; i < L; ++i, to += dim)
                    if (t + i < T) *reinterpret_cast<GlrVec<X, V>*>(to) = narrow<X, V>(h[i]);
            }
        }
        if (ends && a.h_final && live) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (ends >> i & 1) glr_put(a.h_final, marks.end[warp][i] * dim + ch, h[i]);
        }
    }
    glr_exchange_end(ex, blocks, [&] {
        if (copies) ring.drain(filled);
    });
    // sequences without tokens
    if (a.h_final && live) {
        for (int64_t m = rank * kGlrWarps + warp; m < a.num_seqs; m += blocks * kGlrWarps)
            if (a.cu_seqlens[m + 1] == a.cu_seqlens[m]) glr_put(a.h_final, m * dim + ch, glr_state<V>(a.h0, m * dim + ch, true));
    }
}

// A row by 256 threads a stretch of it: one token of every sequence, states read and written in place.  Near a decay of 1 the step is as in a
// stretch; elsewhere, and for a state that is infinite, it is a h.
constexpr float kInfinity = std::numeric_limits<float>::infinity();
template <typename X, typename G, int V, bool SIGMOID, bool COMPLEMENT>
__global__ void __launch_bounds__(kGlrThreads) kda_glr_decode_kernel(const GlrDecodeArgs a, int32_t stretches) {
    const int64_t n = blockIdx.x / stretches, dim = a.dim;
    const int64_t ch = (static_cast<int64_t>(blockIdx.x % stretches) * kGlrThreads + threadIdx.x) * V;
    if (ch >= dim) return;
    const int64_t slot = a.state_indices ? __ldg(a.state_indices + n) : n;
    if (slot < 0 || slot >= a.num_slots) {
        if (ch == 0 && a.device_status) atomicOr(a.device_status, KDA_DEV_BAD_SLOT);
        return;
    }
    const GlrVec<X, V> x = *reinterpret_cast<const GlrVec<X, V>*>(static_cast<const X*>(a.x) + n * dim + ch);
    const GlrVec<G, V> g = *reinterpret_cast<const GlrVec<G, V>*>(static_cast<const G*>(a.gate) + n * dim + ch);
    GlrVec<float, V> s = *reinterpret_cast<const GlrVec<float, V>*>(a.state + slot * dim + ch);
    GlrVec<X, V> out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const GlrGate<1> d = glr_gate<SIGMOID, true>(glr_gates<SIGMOID, true>(GlrVec<G, 1>{g.e[j]}));
        const float xi = glr_f32(x.e[j]), v = COMPLEMENT ? d.n.p * -xi : xi, h = s.e[j];
        const float a = SIGMOID ? -d.n.p * d.e.p : fabsf(d.n.p) < kInfinity ? d.e.p : d.n.p;
        s.e[j] = fabsf(d.n.p) < 0.5f && fabsf(h) < kInfinity ? glr_step(Lanes<1>{h}, d.n, Lanes<1>{v}).p : fmaf(a, h, v);
        glr_round(out.e[j], s.e[j]);
    }
    *reinterpret_cast<GlrVec<float, V>*>(a.state + slot * dim + ch) = s;
    *reinterpret_cast<GlrVec<X, V>*>(static_cast<X*>(a.h) + n * dim + ch) = out;
}

template <typename X, typename G, bool TMA, bool SIGMOID, bool COMPLEMENT>
cudaError_t prefill_as(const GlrArgs& a, const GlrMaps& maps, cudaStream_t stream) {
    using F = Form<X, G, TMA>;
    static GlrRooms rooms;
    const int64_t slices = (a.dim + 32 * F::V - 1) / (32 * F::V);
    return glr_launch(kda_glr_prefill_kernel<X, G, TMA, SIGMOID, COMPLEMENT>, slices, a.total_tokens, F::kBlockTokens,
                      F::kSmem, F::V, rooms, stream, maps, a);
}
template <typename X, typename G, bool SIGMOID, bool COMPLEMENT>
cudaError_t prefill(const GlrArgs& a, bool tiled, cudaStream_t stream) {
    GlrMaps maps = {};
    if (!tiled) return prefill_as<X, G, false, SIGMOID, COMPLEMENT>(a, maps, stream);
    constexpr bool xf = sizeof(X) == 4, gf = sizeof(G) == 4;
    constexpr int rows = Form<X, G, true>::kBlockTokens;
    if (!glr_map(&maps.in[0], a.x, xf, a.total_tokens, a.dim, rows) || !glr_map(&maps.in[1], a.gate, gf, a.total_tokens, a.dim, rows))
        return cudaErrorUnknown;
    return prefill_as<X, G, true, SIGMOID, COMPLEMENT>(a, maps, stream);
}
template <typename X, typename G, bool SIGMOID, bool COMPLEMENT>
cudaError_t decode(const GlrDecodeArgs& a, cudaStream_t stream) {
    const int V = a.dim % 4 == 0 ? 4 : 1;
    const int32_t stretches = (a.dim + kGlrThreads * V - 1) / (kGlrThreads * V);
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.N) * stretches);
    if (V == 4)
        kda_glr_decode_kernel<X, G, 4, SIGMOID, COMPLEMENT><<<grid, kGlrThreads, 0, stream>>>(a, stretches);
    else
        kda_glr_decode_kernel<X, G, 1, SIGMOID, COMPLEMENT><<<grid, kGlrThreads, 0, stream>>>(a, stretches);
    return cudaGetLastError();
}

}  // namespace

bool glr_map(CUtensorMap* m, const void* base, bool f32, int64_t tokens, int32_t dim, int32_t rows) {
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(dim) * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(rows)}, steps[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
              steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
cudaError_t launch_glr_prefill(const GlrKind& kind, const GlrArgs& a, cudaStream_t stream) {
    const bool tiled = a.total_tokens > 0 && glr_tiled(kind, a.dim);
    return KDA_GLR_BY_KIND(kind, prefill, a, tiled, stream);
}
cudaError_t launch_glr_decode(const GlrKind& kind, const GlrDecodeArgs& a, cudaStream_t stream) {
    if (a.N == 0) return cudaSuccess;
    return KDA_GLR_BY_KIND(kind, decode, a, stream);
}

}  // namespace kda
