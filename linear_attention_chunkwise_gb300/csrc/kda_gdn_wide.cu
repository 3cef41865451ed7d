// kda_gdn_wide.cu -- the gated delta rule's scan on tcgen05: one CTA for all 128 columns of a (sequence, value
// head) pair, where there are too many pairs for the CTAs of 32 columns (scan_wide in kda_gdn_prefill.cu).
//
// Everything is kept transposed, rows = the 128 columns of the value head, so that every product has M = 128
// and an epilogue's thread has a row; the left operands are made in registers and go to TMEM, k, q, T and P
// are the right operands as they lie in shared memory:
//   D1 = S^T K^T  (S in two bf16 terms);  DQ = S^T Q^T  (the first term: the output is rounded to bf16 too)
//   R^T = b (V - e^g K S)^T  (two terms)
//   D2 = U^T = R^T T^T  (two terms each, without the product of the second ones)
//   D3 = (e^(gC - g) U)^T K  (two terms);  D4 = U^T P^T  (one term)
//   S^T <- e^gC S^T + D3,   O^T = e^g DQ + D4
// S^T is fp32 in the registers of the eight epilogue warps (warp w: rows 32 (w % 4), channels 64 (w / 4)).  The two
// halves of the channels are handed over by themselves, so that one half's products run beside the other
// half's epilogue.  O of a chunk is formed while the next chunk's second product runs.  One thread issues the
// products and another the copies.
// A chunk is three products and three epilogues one after the other: 3.2 us, of which the tensor pipe is busy 28%
// and the issue slots 40%; what bounds it is the chain of their latencies.  24571 tokens in eight sequences, the
// longest of 6825, x 32 heads: 344 us, 500 with prep and the tables; with two CTAs of 64 columns on mma.sync 489 and
// 632.  With the left operands in shared memory the call took 610 us (its bandwidth is what bounds then), with
// sixteen epilogue warps 533, with V read after the first product instead of during it 529; with the outputs on four
// warps of their own 552 (they are in the way all the time then, not while the second product runs).
// Every on-chip wait is bounded; when one expires KDA_DEV_TIMEOUT is set and the CTA winds down: the copying thread
// waits for its copies, the issuing one for its products, and then the CTA gives TMEM back.
#include "kda_gdn_walk.cuh"

namespace kda {
namespace {

using namespace gdn;

struct Wide {
    static constexpr uint32_t KQ = 0;                     // two blocks of 64 channels x [K 64; Q 64][128 B]
    static constexpr uint32_t IMG = 32768;                // T's two terms, P: [64][128 B] each
    static constexpr uint32_t VEC = IMG + 3 * kTileBytes;  // the image's vectors
    static constexpr uint32_t V = VEC + 1024;             // two blocks of 64 columns x [64][128 B]
    static constexpr uint32_t STAGE = V + 16384;
    static constexpr int ST = 3;
    static constexpr uint32_t BARS = ST * STAGE;
    static constexpr uint32_t TMEM_SLOT = BARS + 128;
    static constexpr uint32_t ABORT = TMEM_SLOT + 4;
    static constexpr uint32_t ALLOC = ABORT + 12 + 1024;
    static constexpr int kParts = 2;                      // epilogue warps to a row: 32 tokens, 64 channels each
    static constexpr int kWalk = 4 * kParts;              // epilogue warps; then the products' and the copies' warp
    static constexpr int kThreads = 32 * (kWalk + 2);
    // barriers: copies landed; four (S, by halves) or eight warps are past; products done
    static constexpr int B_FULL = 0, B_S = 3, B_R = 5, B_U = 6, B_D1 = 7, B_D2 = 8, B_D3 = 9, B_D4 = 11, B_FREE = 12;
    static constexpr int B_END = 14, N_BARS = 15;
    // TMEM columns; D3 takes D1's and D2's place, the first term of U that of S's last channels' second terms
    static constexpr uint32_t D1 = 0, D2 = 64, D3 = 0, DQ = 128, D4 = 256, SH = 320, SL = 384, UH = SL + 32, RH = 448,
                              RL = 480;
};
static_assert(Wide::ALLOC <= 232448 && Wide::N_BARS * 8 <= 128, "shared memory");
constexpr uint32_t kVecBytes = (3 * C + 4) * 4;

__global__ void __launch_bounds__(Wide::kThreads, 1)
    kda_gdn_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const GdnArgs p, const int32_t* __restrict__ co,
                        const int32_t* __restrict__ order, const uint8_t* __restrict__ images, int64_t chunk_slots) {
    using L = Wide;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sm + L::TMEM_SLOT);
    volatile int* const abort_s = reinterpret_cast<volatile int*>(sm + L::ABORT);
    if (tid == 0) {
        *abort_s = 0;
        for (int i = 0; i < L::N_BARS; ++i)
            mbar_init(&bars[i], i < L::B_S || i > L::B_U ? 1 : i < L::B_R ? L::kWalk / 2 : L::kWalk);
        fence_mbar_init();
    }
    grid_wait();  // the images, and the table and order, of the launches before
    WalkUnit u;
    if (!walk_unit<D>(p, co, order, chunk_slots, u)) return;
    if (warp == L::kWalk) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int Hv = p.Hv, nch = u.nch;
    const uint8_t* const img0 = images + (static_cast<size_t>(u.jb) * Hv + u.h) * kImgStrideTile;
    const size_t img_step = static_cast<size_t>(Hv) * kImgStrideTile;

    if (warp == L::kWalk + 1) {  // ---------------------------------------------------------------- copies ----
        if (lane == 0) {
            auto tok = [&](int c) { return static_cast<int32_t>(u.t_begin + static_cast<int64_t>(c) * C); };
            auto load = [&](int c) {
                uint64_t* const bar = &bars[L::B_FULL + c % L::ST];
                uint8_t* const st = sm + c % L::ST * L::STAGE;
                mbar_arrive_expect_tx(bar, 32768 + 3 * kTileBytes + kVecBytes + 16384);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tma_load_3d(st + L::KQ + h * 16384, &tm_k, bar, 64 * h, u.hk, tok(c));
                    tma_load_3d(st + L::KQ + h * 16384 + 8192, &tm_q, bar, 64 * h, u.hk, tok(c));
                    tma_load_3d(st + L::V + h * 8192, &tm_v, bar, 64 * h, u.h, tok(c));
                }
                bulk_g2s(st + L::IMG, img0 + c * img_step, 3 * kTileBytes + kVecBytes, bar);
            };
            int n = 0;  // chunks whose copies have been issued
            for (; n < min(L::ST, nch); ++n) load(n);
            // Chunk c's state products come after the outputs of chunk c - 1, the last that read its stage.  Two
            // barriers in turn: neither can pass this thread by.
            for (int c = 0; n < nch; ++c) {
                if (*abort_s || !mbar_wait_or_stop(&bars[L::B_FREE + (c & 1)], (c >> 1) & 1)) {
                    *abort_s = 1;
                    break;
                }
                if (c > 0) load(n++);
            }
            for (int c = max(0, n - L::ST); c < n; ++c)  // no copy is left in flight
                (void)mbar_wait(&bars[L::B_FULL + c % L::ST], (c / L::ST) & 1, kDrainLimit);
        }
    } else if (warp == L::kWalk) {  // ----------------------------------------------------------- products ----
        if (lane == 0) {
            constexpr uint32_t id = idesc_bf16_f32(128, 64, false, false), id_k = idesc_bf16_f32(128, 64, false, true);
            auto past = [&](int bar, uint32_t parity) {
                if (mbar_wait_or_stop(&bars[bar], parity)) {
                    tc_fence_after();
                    return true;
                }
                *abort_s = 1;
                return false;
            };
            auto steps = [&](uint32_t d, uint32_t a, uint64_t b, bool fresh) {  // 64 of K, b's rows K-major
#pragma unroll
                for (int s = 0; s < 4; ++s) mma_bf16_ta(tmem + d, tmem + a + 8 * s, b + 2 * s, id, s > 0 || !fresh);
            };
            // The same with T or P: tokens 16 s .. of K reach the columns from there on only, and the blocks above the
            // diagonal are not read.
            auto lower_steps = [&](uint32_t d, uint32_t a, uint64_t b, bool fresh) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_bf16_ta(tmem + d + 16 * s, tmem + a + 8 * s, b + 128 * s + 2 * s,
                                idesc_bf16_f32(128, 64 - 16 * s, false, false), s > 0 || !fresh);
            };
            for (int c = 0; c < nch; ++c) {
                const uint32_t par = c & 1, st = smem_u32(sm + c % L::ST * L::STAGE), dq = L::DQ + 64 * par;
                const uint64_t d_k = sdesc_sw128(st + L::KQ, 16, 1024), d_q = d_k + 512;
                const uint64_t d_t = sdesc_sw128(st + L::IMG, 16, 1024), d_p = d_t + 1024;
                if (!past(L::B_FULL + c % L::ST, (c / L::ST) & 1) || !past(L::B_S, par)) break;
                steps(L::D1, L::SH, d_k, true);
                steps(L::D1, L::SL, d_k, false);
                if (!past(L::B_S + 1, par)) break;
                steps(L::D1, L::SH + 32, d_k + 1024, false);
                steps(L::D1, L::SL + 32, d_k + 1024, false);
                mma_commit(&bars[L::B_D1]);
                steps(dq, L::SH, d_q, true);
                steps(dq, L::SH + 32, d_q + 1024, false);
                if (!past(L::B_R, par)) break;
                lower_steps(L::D2, L::RH, d_t, true);
                lower_steps(L::D2, L::RL, d_t, false);
                lower_steps(L::D2, L::RH, d_t + 512, false);
                mma_commit(&bars[L::B_D2]);
                if (!past(L::B_U, par)) break;
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {  // the state's channels 64 kh ..
#pragma unroll
                    for (int s = 0; s < 8; ++s)  // k as it lies: rows of tokens, 16 of them a step
                        mma_bf16_ta(tmem + L::D3 + 64 * kh, tmem + (s < 4 ? L::RH : L::RL) + 8 * (s & 3),
                                    d_k + 1024 * kh + 128 * (s & 3), id_k, s > 0);
                    if (kh == 0) {
                        mma_commit(&bars[L::B_D3]);
                        lower_steps(L::D4, L::UH, d_p, true);
                        mma_commit(&bars[L::B_D4]);
                    }
                }
                mma_commit(&bars[L::B_D3 + 1]);
                mma_commit(&bars[L::B_FREE + par]);
            }
            mma_commit(&bars[L::B_END]);  // every product has landed before the CTA gives its memory back
            (void)mbar_wait(&bars[L::B_END], 0, kDrainLimit);
        }
    } else {  // -------------------------------------------------------------------------- epilogues ----
        constexpr int NB = 4 / L::kParts, NT = 16 * NB, NC = 2 * NT;  // 16s of tokens, tokens, channels of a thread
        const int qw = warp & 3, part = warp >> 2, half = part / (L::kParts / 2);
        const int col = 32 * qw + lane;            // the row of S^T: a column of the value head
        const uint32_t tq = tmem + (static_cast<uint32_t>(32 * qw) << 16);
        const size_t state = ((static_cast<size_t>(u.seq) * Hv + u.h) * D + NC * part) * D + col;
        float S[NC];  // channels NC part ..
#pragma unroll
        for (int i = 0; i < NC; ++i) S[i] = p.S0 ? p.S0[state + static_cast<size_t>(i) * D] : 0.f;
        auto past = [&](int bar, uint32_t parity) {  // the whole warp
            const bool ok = mbar_wait_or_stop(&bars[bar], parity);
            if (__all_sync(0xffffffffu, ok)) return true;
            *abort_s = 1;
            return false;
        };
        auto arrive = [&](int bar) {  // this warp's TMEM reads and writes are done
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[bar]);
        };
        auto put8 = [&](uint32_t hi, uint32_t lo, const float (&x)[16]) {  // the two terms of 16 values of this row
            uint32_t h[8], l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) split2(x[2 * i], x[2 * i + 1], h[i], l[i]);
            tmem_st8(tq + hi, h);
            tmem_st8(tq + lo, l);
        };
        auto load8 = [](float (&x)[8], const float* from) {
            const float4 a = reinterpret_cast<const float4*>(from)[0], b = reinterpret_cast<const float4*>(from)[1];
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
            x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        };
        auto outputs = [&](int c) {  // O of chunk c: this thread's column, tokens NT part ..
            if (!past(L::B_D4, c & 1)) return false;
            tc_fence_after();
            const float* eg = reinterpret_cast<const float*>(sm + c % L::ST * L::STAGE + L::VEC) + kVecEg + NT * part;
            const int64_t t0 = u.t_begin + static_cast<int64_t>(c) * C + NT * part;
            const int n = static_cast<int>(u.t_end - t0 < NT ? u.t_end - t0 : NT);
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + (t0 * Hv + u.h) * D + col;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float x[16], y[16];
                tmem_ld16(tq + L::DQ + 64 * (c & 1) + NT * part + 16 * b, x);
                tmem_ld16(tq + L::D4 + NT * part + 16 * b, y);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float e[8];
                    load8(e, eg + 16 * b + 8 * h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (n >= NT || 16 * b + 8 * h + i < n) *o = __float2bfloat16_rn(fmaf(e[i], x[8 * h + i], y[8 * h + i]));
                        o += static_cast<int64_t>(Hv) * D;
                    }
                }
            }
            return true;
        };
        int c = 0;
        for (; c < nch; ++c) {
            const uint32_t par = c & 1;
            const int64_t rem = u.t_end - (u.t_begin + static_cast<int64_t>(c) * C);
            const int Lc = static_cast<int>(rem < C ? rem : C);
#pragma unroll
            for (int b = 0; b < 2 * NB; ++b) {
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = S[16 * b + i];
                put8(L::SH + NC / 2 * part + 8 * b, L::SL + NC / 2 * part + 8 * b, x);
            }
            uint8_t* const st = sm + c % L::ST * L::STAGE;
            if (Lc < C) {  // k rows behind the sequence's end meet zeros of U: they must be numbers
                if (!past(L::B_FULL + c % L::ST, (c / L::ST) & 1)) break;
                for (int e = tid; e < (C - Lc) * 16; e += 32 * L::kWalk)
                    *reinterpret_cast<uint4*>(st + L::KQ + (e & 1) * 16384 + sw128_chunk(Lc + (e >> 4), (e >> 1) & 7)) =
                        make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
            }
            arrive(L::B_S + half);
            const float* vec = reinterpret_cast<const float*>(st + L::VEC);
            if (!past(L::B_FULL + c % L::ST, (c / L::ST) & 1)) break;
            uint32_t v[NT / 2];  // this column's values, pairs of tokens, read while the product runs
            const uint8_t* const vt = st + L::V + (qw >> 1) * 8192 + NT * part * 128 + 2 * (col & 7);
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) {
                const uint32_t lo = *reinterpret_cast<const uint16_t*>(vt + sw128_chunk(2 * i, (col & 63) >> 3));
                const uint32_t hi = *reinterpret_cast<const uint16_t*>(vt + sw128_chunk(2 * i + 1, (col & 63) >> 3));
                v[i] = lo | hi << 16;
            }
            if (!past(L::B_D1, par)) break;
            tc_fence_after();
            float a[16], x[16];
#pragma unroll
            for (int b = 0; b < NB; ++b) {  // R^T
                const int t0 = NT * part + 16 * b;
                tmem_ld16(tq + L::D1 + t0, a);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float eg[8], be[8];
                    load8(eg, vec + kVecEg + t0 + 8 * h);
                    load8(be, vec + kVecB + t0 + 8 * h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t vv = v[(16 * b + 8 * h + i) / 2];
                        x[8 * h + i] = be[i] * fmaf(-eg[i], a[8 * h + i], __uint_as_float(i & 1 ? vv & 0xffff0000u : vv << 16));
                    }
                }
                if (Lc < C) {  // v behind the sequence's end may be anything
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (t0 + i >= Lc) x[i] = 0.f;
                }
                put8(L::RH + t0 / 2, L::RL + t0 / 2, x);
            }
            arrive(L::B_R);
            if (c > 0 && !outputs(c - 1)) break;  // before U(c) may replace what they come from
            if (!past(L::B_D2, par)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < NB; ++b) {  // U^T
                const int t0 = NT * part + 16 * b;
                tmem_ld16(tq + L::D2 + t0, a);
                tmem_ld_wait();
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = pack_bf16(a[2 * i], a[2 * i + 1]);
                tmem_st8(tq + L::UH + t0 / 2, h);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float eo[8];
                    load8(eo, vec + kVecEo + t0 + 8 * e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[8 * e + i] = eo[i] * a[8 * e + i];
                }
                put8(L::RH + t0 / 2, L::RL + t0 / 2, x);
            }
            arrive(L::B_U);
            const float gc = vec[kVecEc];
            if (!past(L::B_D3 + half, par)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2 * NB; ++b) {
                tmem_ld16(tq + L::D3 + NC * part + 16 * b, a);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) S[16 * b + i] = fmaf(gc, S[16 * b + i], a[i]);
            }
        }
        if (c == nch && nch > 0) (void)outputs(nch - 1);
        if (p.S_final && !*abort_s) {
#pragma unroll
            for (int i = 0; i < NC; ++i) p.S_final[state + static_cast<size_t>(i) * D] = S[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_s && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
    if (warp == L::kWalk) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_gdn_wide(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                            cudaStream_t stream) {
    static int configured[64];
    const cudaError_t err = set_smem(kda_gdn_wide_kernel, Wide::ALLOC, configured);
    if (err != cudaSuccess) return err;
    CUtensorMap tm_v;
    if (!make_tensor_map(&tm_v, a.v, a.Hv, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    return launch_dependent(kda_gdn_wide_kernel, static_cast<int64_t>(a.num_seqs) * a.Hv, Wide::kThreads, Wide::ALLOC, stream,
                            tm_q, tm_k, tm_v, a, w.table, w.order, w.images, w.chunks);
}

}  // namespace kda
