// kda_glr_backward.cu -- gradient of the gated linear recurrence.
//
// With L = <h, grad_h> + <h_final, grad_h_final>, lambda_t = dL/dh_t and mu_t = a_t lambda_t (what token t - 1 gets of it):
//   lambda_t = grad_h_t + mu_{t+1}   (a sequence's last token: grad_h_final in place of mu)
//   grad_x_t = s_t lambda_t,   da_t = lambda_t (h_{t-1} - [s_t = 1 - a_t] x_t),   grad_h0 = mu of the first token
//   grad_gate_t = a_t da_t (exp)  or  a_t (1 - a_t) da_t (sigmoid)
// mu is the same kind of recurrence, backwards: mu_t = (1 - c_t)(grad_h_t + mu_{t+1}), so tokens i..j together are a pair (C, M).
//
// Bound by HBM like the forward: x, gates and grad_h are read once, two gradients written once.  The rounds go from the last
// tokens to the first.  h_{t-1} is built again from the state before each kGlrCheckpoint tokens, which is what a block has in a
// round, so only mu has to go from block to block (kda_glr_common.cuh).  8192 tokens x 4096 channels, bf16: 100 us, 3.4 TB/s of 6.8, bound
// by a round's chain as the forward is, with issue slots 52 % taken.
#include <type_traits>

#include "kda_glr_common.cuh"

namespace kda {
namespace {

template <typename X, typename G, bool TMA>
struct Form {
    static constexpr int V = TMA ? 2 : 1;
    static constexpr int L = kGlrCheckpoint / kGlrWarps;  // tokens of a thread in a round
    static constexpr uint32_t kTileX = kGlrCheckpoint * 64 * sizeof(X), kTileG = kGlrCheckpoint * 64 * sizeof(G), kStage = 2 * kTileX + kTileG;
    static constexpr int kStages = sizeof(X) == 4 ? 2 : 3;
    static constexpr uint32_t kSmem = TMA ? kStages * kStage : 0;
};

template <typename X, typename G, bool TMA, bool SIGMOID, bool COMPLEMENT>
__global__ void __launch_bounds__(kGlrThreads, 2) kda_glr_backward_kernel(const __grid_constant__ GlrMaps maps, const GlrArgs a,
                                                                          const GlrBackwardArgs b) {
    using F = Form<X, G, TMA>;
    constexpr int V = F::V, L = F::L;
    extern __shared__ __align__(128) uint8_t tiles[];
    __shared__ GlrExchange<V> ex;
    __shared__ GlrMarks<L> marks;
    __shared__ GlrStretch<V> forward[kGlrWarps][32];
    __shared__ int32_t forward_cut[kGlrWarps];
    __shared__ GlrRing<F::kStages> ring;
    const int rank = cluster_rank(), blocks = cluster_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t T = a.total_tokens;
    const int64_t dim = a.dim, ch0 = static_cast<int64_t>(blockIdx.x / blocks) * 32 * V, ch = ch0 + lane * V;
    const bool live = ch < dim;  // V divides dim
    const int32_t step = blocks * kGlrCheckpoint, rounds = (T + step - 1) / step;
    const int32_t block_last = (rounds - 1) * step + rank * kGlrCheckpoint;  // the block's first token of the first round
    glr_check_sequences(a.cu_seqlens, a.num_seqs, T, a.device_status);
    if (TMA && threadIdx.x == 0) ring.start();
    glr_exchange_start(ex, blocks);
    const bool copies = TMA && warp == 0 && lane == 0;
    int32_t filled = 0;
    const auto load = [&](uint8_t* at, uint64_t* bar, int32_t round) {
        const int32_t c = static_cast<int32_t>(ch0), t = block_last - round * step;
        tma_load_2d(at, &maps.in[0], bar, c, t);
        tma_load_2d(at + F::kTileX, &maps.in[2], bar, c, t);
        tma_load_2d(at + 2 * F::kTileX, &maps.in[1], bar, c, t);
    };
    if (copies)
        for (; filled < F::kStages && filled < rounds; ++filled) ring.fill(tiles, F::kStage, filled, load);
    const auto checkpoint = [&](int32_t t) {
        return glr_state<V>(b.checkpoints, t / kGlrCheckpoint * dim + ch, live && t >= 0 && t < T);
    };
    Lanes<V> carry = lanes<V>(0.f), coming = checkpoint(block_last);
    GlrPlace place;
    for (int32_t round = 0; round < rounds; ++round) {
        const int32_t block_t = block_last - round * step, t = block_t + warp * L;
        uint32_t starts, ends;
        glr_marks<L, true>(marks, place, a.cu_seqlens, a.num_seqs, t, &starts, &ends);
        Lanes<V> n[L], slope[L], v[L], dh[L], state = coming;  // v: the weighted input
        GlrVec<X, V> xr[L];
        if constexpr (TMA) {
            glr_wait(&ring.full[round % F::kStages], round / F::kStages & 1, ex.flags[round & 1], a.device_status);
            const uint8_t* at = tiles + round % F::kStages * F::kStage;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                xr[i] = reinterpret_cast<const GlrVec<X, V>*>(at)[(warp * L + i) * 32 + lane];
                dh[i] = wide(reinterpret_cast<const GlrVec<X, V>*>(at + F::kTileX)[(warp * L + i) * 32 + lane]);
                n[i] = glr_gates<SIGMOID, true>(reinterpret_cast<const GlrVec<G, V>*>(at + 2 * F::kTileX)[(warp * L + i) * 32 + lane]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool in = live && t + i < T;
                xr[i].e[0] = glr_load(static_cast<const X*>(a.x) + (t + i) * dim + ch, in);
                dh[i].p = glr_f32(glr_load(static_cast<const X*>(b.grad_h) + (t + i) * dim + ch, in));
                n[i] = glr_gates<SIGMOID, true>(GlrVec<G, 1>{glr_load(static_cast<const G*>(a.gate) + (t + i) * dim + ch, in)});
            }
        }
        coming = checkpoint(block_t - step);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const GlrGate<V> g = glr_gate<SIGMOID, true>(n[i]);
            n[i] = g.n;
            slope[i] = g.slope;
            v[i] = COMPLEMENT ? mul(n[i], wide_negative(xr[i])) : wide(xr[i]);
        }
        // Most tokens are far from a sequence's ends and from the tensors': the loops over them are there with and without the questions.
        const bool plain = (starts | ends) == 0 && t + L <= T && ch0 + 32 * V <= dim;
        // The warp's pairs, both ways, from zero states.
        GlrStretch<V> fwd = {lanes<V>(0.f), lanes<V>(0.f)}, bwd = fwd;
        const auto scan = [&](auto marked) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (marked && (starts >> i & 1)) fwd.h = glr_state<V>(a.h0, marks.start[warp][i] * dim + ch, live);
                fwd.h = glr_step(fwd.h, n[i], v[i]);
                fwd.n = glr_join(fwd.n, n[i]);
            }
#pragma unroll
            for (int i = L - 1; i >= 0; --i) {
                if (marked && (ends >> i & 1)) bwd.h = glr_state<V>(b.grad_h_final, marks.end[warp][i] * dim + ch, live);
                const Lanes<V> lambda = add(dh[i], bwd.h);
                bwd.h = fma(n[i], lambda, lambda);
            }
            bwd.n = fwd.n;  // the same product of decays
        };
        if (plain) scan(std::false_type{});
        else scan(std::true_type{});
        forward[warp][lane] = fwd;
        if (lane == 0) forward_cut[warp] = starts != 0;
        Lanes<V> mu;
        if (!glr_exchange<F::kSmem, V, true>(ex, rank, blocks, round, bwd, ends != 0, carry, mu, a.device_status, [&] {
                if (copies && filled < rounds) ring.fill(tiles, F::kStage, filled++, load);
                for (int w = 0; w < warp; ++w) state = glr_through(state, forward[w][lane], forward_cut[w] != 0);
            }))
            break;
        const auto finish = [&](auto marked) {
            Lanes<V> before[L];  // the state before each token
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (marked && (starts >> i & 1)) state = glr_state<V>(a.h0, marks.start[warp][i] * dim + ch, live);
                before[i] = state;
                if (i + 1 < L) state = glr_step(state, n[i], v[i]);
            }
            const int64_t last = (t + L - 1) * dim + ch;
            X* to_x = static_cast<X*>(b.grad_x) + last;
            G* to_g = static_cast<G*>(b.grad_gate) + last;
#pragma unroll
            for (int i = L - 1; i >= 0; --i, to_x -= dim, to_g -= dim) {
                if (marked && (ends >> i & 1)) mu = glr_state<V>(b.grad_h_final, marks.end[warp][i] * dim + ch, live);
                const Lanes<V> lambda = add(dh[i], mu);
                const Lanes<V> from = COMPLEMENT ? add(before[i], wide_negative(xr[i])) : before[i];
                mu = fma(n[i], lambda, lambda);
                const GlrVec<X, V> dx = narrow<X, V>(COMPLEMENT ? mul(n[i], mul(lambda, lanes<V>(-1.f))) : lambda);
                const GlrVec<G, V> dg = narrow<G, V>(mul(slope[i], mul(lambda, from)));
                if (!marked || (live && t + i < T)) {
                    *reinterpret_cast<GlrVec<X, V>*>(to_x) = dx;
                    *reinterpret_cast<GlrVec<G, V>*>(to_g) = dg;
                }
                if (marked && (starts >> i & 1) && b.grad_h0 && live) glr_put(b.grad_h0, marks.start[warp][i] * dim + ch, mu);
            }
        };
        if (plain) finish(std::false_type{});
        else finish(std::true_type{});
    }
    glr_exchange_end(ex, blocks, [&] {
        if (copies) ring.drain(filled);
    });
    // sequences without tokens
    if (b.grad_h0 && live) {
        for (int64_t m = rank * kGlrWarps + warp; m < a.num_seqs; m += blocks * kGlrWarps)
            if (a.cu_seqlens[m + 1] == a.cu_seqlens[m])
                glr_put(b.grad_h0, m * dim + ch, glr_state<V>(b.grad_h_final, m * dim + ch, true));
    }
}

template <typename X, typename G, bool TMA, bool SIGMOID, bool COMPLEMENT>
cudaError_t backward_as(const GlrArgs& a, const GlrBackwardArgs& b, const GlrMaps& maps, cudaStream_t stream) {
    using F = Form<X, G, TMA>;
    static GlrRooms rooms;
    const int64_t slices = (a.dim + 32 * F::V - 1) / (32 * F::V);
    return glr_launch(kda_glr_backward_kernel<X, G, TMA, SIGMOID, COMPLEMENT>, slices, a.total_tokens, kGlrCheckpoint,
                      F::kSmem, F::V, rooms, stream, maps, a, b);
}
template <typename X, typename G, bool SIGMOID, bool COMPLEMENT>
cudaError_t backward(const GlrArgs& a, const GlrBackwardArgs& b, bool tiled, cudaStream_t stream) {
    GlrMaps maps = {};
    if (!tiled) return backward_as<X, G, false, SIGMOID, COMPLEMENT>(a, b, maps, stream);
    constexpr bool xf = sizeof(X) == 4, gf = sizeof(G) == 4;
    constexpr int rows = kGlrCheckpoint;
    if (!glr_map(&maps.in[0], a.x, xf, a.total_tokens, a.dim, rows) || !glr_map(&maps.in[1], a.gate, gf, a.total_tokens, a.dim, rows) ||
        !glr_map(&maps.in[2], b.grad_h, xf, a.total_tokens, a.dim, rows))
        return cudaErrorUnknown;
    return backward_as<X, G, true, SIGMOID, COMPLEMENT>(a, b, maps, stream);
}

}  // namespace

cudaError_t launch_glr_backward(const GlrKind& kind, const GlrArgs& a, const GlrBackwardArgs& b, cudaStream_t stream) {
    const bool tiled = a.total_tokens > 0 && glr_tiled(kind, a.dim);
    return KDA_GLR_BY_KIND(kind, backward, a, b, tiled, stream);
}

}  // namespace kda
