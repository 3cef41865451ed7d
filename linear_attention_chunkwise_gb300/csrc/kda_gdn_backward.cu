// kda_gdn_backward.cu -- gradient of the gated delta rule's chunkwise prefill (bf16 inputs).
//
// For L = <o, dO> + <S_final, dS_final>, with a chunk's quantities of kda_gdn_prefill.cu (g, G, A, T, P, U,
// start state S) and X the adjoint of the state at its end, e_i = exp(gC - g_i), b = beta:
//   dU = P^T dO + Diag(e) K X,   W = T^T dU,   dv = b W,
//   adjoint of the start state = e^gC X + K^T (-Diag(e^g b) W) + Q^T (Diag(e^g) dO)
//   dP = dO U^T, dA = -W U^T (below the diagonal), M = G dP, E = b G dA
//   dq = Diag(e^g) dO S^T + M K
//   dk = -Diag(e^g b) W S^T + Diag(e) U X^T + M^T Q + (E + E^T) K
//   db_i = (W_i . U_i) / b_i      (U_i / b_i are the rows that b multiplies)
// log_decay_t scales what passes from before token t to it or later: the pairs i >= t > j, the start state
// as tokens from t on read it, what tokens before t leave in the end state, and the start state there:
//   gradient of log_decay_t = sum_{i >= t > j} (dP P + dA A)_ij + sum_{i >= t} a_i + sum_{j < t} w_j + e^gC <X, S>,
//   a_i = q_i . (e^g dO S^T)_i - k_i . (e^g b W S^T)_i,   w_j = k_j . (e U X^T)_j.
// (As the sums, from t on, of one gradient for each g_i it would need a difference of large sums; here a
// decay of 0 gives exactly 0.)
//
// Kernels: the prefill's prep; a walk over the chunks (leaving S and U) and beside it one back (leaving X and
// W, writing dv and the start state's gradient); and the rest by (chunk, q/k head), the value heads of a group
// added up in registers.  Operands that are not raw bf16 inputs are two bf16 terms
// wherever the result is kept in fp32 (states, decays, b); M and E, which only reach the bf16 dq and dk,
// are one.
#include <algorithm>

#include "kda_gdn_walk.cuh"

namespace kda {
namespace {

using namespace gdn;

// ============================================================== walks ==
// Four warps walk forward and four back, each group with tiles and a copying thread of its own: a warp of
// either is a chain that leaves the SM's issue slots and tensor cores half idle, and the two do not wait for
// each other.  8192 tokens x 16/32 heads: 447 us, 3.5 us a chunk, 0.8 GB of records written; the tensor pipe is 51%
// busy, the back walk's chain is the longer one.  The copying warps' registers go to the walks': launched with 168 a
// thread, 3 x 168 = 216 + 248 + 40; five words spill at 32 columns, none at 64.
template <int NT>
struct BackCfg {
    static constexpr int ST = 2;
    static constexpr int kCols = 32 * NT;
    static constexpr uint32_t kVRow = 2 * kCols;  // bytes of a dO row
    static constexpr uint32_t K = 0, Q = 16384, IMG = 32768, V = IMG + 27648;
    static constexpr uint32_t STAGE = V + C * kVRow;
    static_assert(STAGE % 1024 == 0 && kImgStrideBwd <= 27648, "stages");
};
template <int NT>
struct WalksCfg {
    using F = ForwardCfg<NT, 4, 2, true>;
    using B = BackCfg<NT>;
    static constexpr int kThreads = 384;
    static constexpr uint32_t BACK = F::ST * F::STAGE;
    static constexpr uint32_t BARS = BACK + B::ST * B::STAGE;  // full, empty of each
    static constexpr uint32_t ABORT = BARS + 16 * (F::ST + B::ST);
    static constexpr uint32_t ALLOC = ABORT + 16 + 1024;
    static_assert(ALLOC <= 232448, "shared memory");
};

template <typename L>
__device__ __forceinline__ void back_copies(const WalkUnit& u, const WalkPipe& pipe, const GdnArgs& p,
                                            const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_do,
                                            const uint8_t* images) {
    pipe_copies<L::ST>(pipe, u.nch, [&](int i, int s) {  // step i takes chunk nch - 1 - i
        const int c = u.nch - 1 - i;
        uint8_t* st = pipe.sm + s * L::STAGE;
        uint64_t* bar = &pipe.full[s];
        const int32_t tok = static_cast<int32_t>(u.t_begin + static_cast<int64_t>(c) * C);
        mbar_arrive_expect_tx(bar, 32768 + static_cast<uint32_t>(kImgStrideBwd) + C * L::kVRow);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) tma_load_3d(st + L::K + kh * 8192, tm_k, bar, 64 * kh, u.hk, tok);
        tma_load_3d(st + L::V, tm_do, bar, u.col0, u.h, tok);
        bulk_g2s(st + L::IMG, images + (static_cast<size_t>(u.jb + c) * p.Hv + u.h) * kImgStrideBwd,
                 static_cast<uint32_t>(kImgStrideBwd), bar);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) tma_load_3d(st + L::Q + kh * 8192, tm_q, bar, 64 * kh, u.hk, tok);
    });
}

template <typename L, int NT>
__device__ __forceinline__ void walk_back(const WalkUnit& wu, const WalkPipe& pipe, const GdnArgs& p,
                                          const GdnBackwardArgs& gr, uint8_t* records, int warp, int lane) {
    constexpr int ST = L::ST;
    const int Hv = p.Hv;
    const int g = lane >> 2, t = lane & 3;
    const int wc = 8 * NT * warp;               // the warp's first column in the CTA's
    const int col = wu.col0 + wc + 2 * t;  // this thread's first column
    const size_t sbase = (static_cast<size_t>(wu.seq) * Hv + wu.h) * D * D;
    float X[8][NT][4];  // rows 16 m + g (+ 8), columns col + 8 n (+ 1)
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const size_t off = sbase + static_cast<size_t>(16 * m + g + 8 * e) * D + col + 8 * n;
                const float2 x =
                    gr.grad_S_final ? *reinterpret_cast<const float2*>(gr.grad_S_final + off) : make_float2(0.f, 0.f);
                X[m][n][2 * e] = x.x;
                X[m][n][2 * e + 1] = x.y;
            }
    // ldmatrix addresses: rows of tokens, and transposed [channels or columns][tokens] blocks
    const int lr = lane & 15, lc = lane >> 4;
    const int tr = (lane & 7) + ((lane >> 4) << 3), tc = (lane >> 3) & 1;
    const int lt = (lane & 7) | ((lane & 8) << 1) | ((lane & 16) >> 1);  // an image block's, transposed
    for (int i = 0; i < wu.nch; ++i) {
        const int s = i % ST, c = wu.nch - 1 - i;
        uint8_t* st = pipe.sm + s * L::STAGE;
        const bool landed = !*pipe.abort_s && mbar_wait_pipe(&pipe.full[s], (i / ST) & 1);
        if (!__all_sync(0xffffffffu, landed)) {  // a bounded wait expired, here or elsewhere
            *pipe.abort_s = 1;
            break;
        }
        const int64_t t0 = wu.t_begin + static_cast<int64_t>(c) * C;
        const int Lc = static_cast<int>(wu.t_end - t0 < C ? wu.t_end - t0 : C);
        if (Lc < C) {  // rows behind the sequence's end: no tokens (every warp clears all it reads)
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            for (int e = lane; e < (C - Lc) * 16; e += 32) {
                const uint32_t off = (e & 1) * 8192 + sw128_chunk(Lc + (e >> 4), (e >> 1) & 7);
                *reinterpret_cast<uint4*>(st + L::K + off) = z;
                *reinterpret_cast<uint4*>(st + L::Q + off) = z;
            }
            for (uint32_t e = Lc * L::kVRow + 16 * lane; e < C * L::kVRow; e += 512)
                *reinterpret_cast<uint4*>(st + L::V + e) = z;
            __syncwarp();
        }
        const uint32_t kb = smem_u32(st + L::K), qb = smem_u32(st + L::Q), ib = smem_u32(st + L::IMG) + 16 * lt;
        const float* gs = reinterpret_cast<const float*>(st + L::IMG + kImgG);
        uint8_t* const rec = records + (static_cast<size_t>(wu.jb + c) * Hv + wu.h) * kRecStride;
        const int rcol = (wu.col0 + wc) >> 3;  // matrices of 8 columns
        // K X
        float u[4][NT][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) u[m][n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            BTerms b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                put_record(X[k][n], rec + kRecX, 32768, 2 * k, rcol + n, lane);
                b[n] = b_terms(X[k][n]);
            }
            uint32_t a[4][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) ldsm4(a[m], kb + (k >> 2) * 8192 + sw128_chunk(16 * m + lr, 2 * (k & 3) + lc));
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], a[m], b[n].h0, b[n].h1);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], a[m], b[n].l0, b[n].l1);
        }
        // dO as B operand: [k][n] registers of tokens 16 k + 2 t (+ 1) and 16 k + 8 + 2 t (+ 1)
        uint32_t dob[4][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int row = 32 * hf + lane, piece = (wc >> 3) + n;
                uint32_t off;
                if constexpr (L::kVRow == 128) off = sw128_chunk(row, piece);
                else off = row * 64 + (((piece ^ (row >> 1)) & 3) << 4);  // 64-byte rows
                uint32_t f[4];
                ldsm4t(f, smem_u32(st + L::V) + off);
                dob[2 * hf][n][0] = f[0];
                dob[2 * hf][n][1] = f[1];
                dob[2 * hf + 1][n][0] = f[2];
                dob[2 * hf + 1][n][1] = f[3];
            }
        // dU = e K X + P^T dO, P in three terms: an entry's error is that of a whole row of W, and of b's
        // gradient with it
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float e0 = gs[kVecEo + 16 * m + g], e1 = gs[kVecEo + 16 * m + g + 8];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                u[m][n][0] *= e0;
                u[m][n][1] *= e0;
                u[m][n][2] *= e1;
                u[m][n][3] *= e1;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t ah[4][4], al[4][4], am[4][4];
#pragma unroll
            for (int m = 0; m <= k; ++m) {
                ldsm4t(ah[m], ib + kImgP + tri_blk(k, m));
                ldsm4t(al[m], ib + kImgPl + tri_blk(k, m));
                ldsm4t(am[m], ib + kImgPl2 + tri_blk(k, m));
            }
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], dob[k][n][0], dob[k][n][1]);
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], al[m], dob[k][n][0], dob[k][n][1]);
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], am[m], dob[k][n][0], dob[k][n][1]);
        }
        // W = T^T dU, T in two terms, dU in three
        float w[4][NT][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[m][n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            BTerms3 b3[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b3[n] = b_terms3(u[k][n]);
            uint32_t ah[4][4], al[4][4];
#pragma unroll
            for (int m = 0; m <= k; ++m) {
                ldsm4t(ah[m], ib + kImgTh + tri_blk(k, m));
                ldsm4t(al[m], ib + kImgTl + tri_blk(k, m));
            }
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(w[m][n], ah[m], b3[n].b.h0, b3[n].b.h1);
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(w[m][n], ah[m], b3[n].b.l0, b3[n].b.l1);
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(w[m][n], ah[m], b3[n].m0, b3[n].m1);
#pragma unroll
            for (int m = 0; m <= k; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(w[m][n], al[m], b3[n].b.h0, b3[n].b.h1);
        }
        // X <- e^gC X + K^T (-e^g b W) + Q^T (e^g dO)
        const float gc = gs[kVecEc];
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) X[m][n][e] *= gc;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r0 = 16 * k + g;
            const float z0 = -gs[kVecEg + r0] * gs[kVecB + r0], z1 = -gs[kVecEg + r0 + 8] * gs[kVecB + r0 + 8];
            const float2 ga = *reinterpret_cast<const float2*>(gs + kVecEg + 16 * k + 2 * t);
            const float2 gb = *reinterpret_cast<const float2*>(gs + kVecEg + 16 * k + 8 + 2 * t);
            BTerms b[NT], d[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float x[4] = {w[k][n][0] * z0, w[k][n][1] * z0, w[k][n][2] * z1, w[k][n][3] * z1};
                b[n] = b_terms(x);
                const float2 y0 = unpack_bf16(dob[k][n][0]), y1 = unpack_bf16(dob[k][n][1]);
                split2(y0.x * ga.x, y0.y * ga.y, d[n].h0, d[n].l0);
                split2(y1.x * gb.x, y1.y * gb.y, d[n].h1, d[n].l1);
            }
#pragma unroll
            for (int mh = 0; mh < 2; ++mh) {
                uint32_t a[4][4];
#pragma unroll
                for (int m = 0; m < 4; ++m) ldsm4t(a[m], kb + mh * 8192 + sw128_chunk(16 * k + tr, 2 * m + tc));
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(X[4 * mh + m][n], a[m], b[n].h0, b[n].h1);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(X[4 * mh + m][n], a[m], b[n].l0, b[n].l1);
#pragma unroll
                for (int m = 0; m < 4; ++m) ldsm4t(a[m], qb + mh * 8192 + sw128_chunk(16 * k + tr, 2 * m + tc));
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(X[4 * mh + m][n], a[m], d[n].h0, d[n].h1);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(X[4 * mh + m][n], a[m], d[n].l0, d[n].l1);
            }
        }
        float bs[4][2];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) bs[m][e] = gs[kVecB + 16 * m + g + 8 * e];
        if (Lc < C) fence_async_smem();  // the cleared rows, before the stage's next copies
        __syncwarp();
        if (lane == 0) mbar_arrive(&pipe.empty[s]);  // the warp has read all it takes of this stage
        __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(gr.grad_v) + (t0 * Hv + wu.h) * D + col;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int n = 0; n < NT; ++n) put_record(w[m][n], rec + kRecW, 16384, 2 * m, rcol + n, lane);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 16 * m + g + 8 * e;
                if (row < Lc) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<uint32_t*>(dv + static_cast<int64_t>(row) * Hv * D + 8 * n) =
                            pack_bf16(bs[m][e] * w[m][n][2 * e], bs[m][e] * w[m][n][2 * e + 1]);
                }
            }
        }
    }
    if (gr.grad_S0 && !*pipe.abort_s) {
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2*>(gr.grad_S0 + sbase + static_cast<size_t>(16 * m + g + 8 * e) * D + col +
                                               8 * n) = make_float2(X[m][n][2 * e], X[m][n][2 * e + 1]);
    }
}

template <int NT>
__global__ void __launch_bounds__(WalksCfg<NT>::kThreads, 1)
    kda_gdn_walks_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const GdnArgs p,
                         const GdnBackwardArgs gr, const int32_t* __restrict__ co, const int32_t* __restrict__ order,
                         const uint8_t* __restrict__ images, int64_t chunk_slots, uint8_t* records) {
    using L = WalksCfg<NT>;
    using F = typename L::F;
    using B = typename L::B;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
    volatile int* const abort_s = reinterpret_cast<volatile int*>(sm + L::ABORT);
    const WalkPipe fwd{sm, bars, bars + F::ST, abort_s};
    const WalkPipe back{sm + L::BACK, bars + 2 * F::ST, bars + 2 * F::ST + B::ST, abort_s};
    if (tid == 0) {
        *abort_s = 0;
        pipe_init(fwd, F::ST, 4);
        pipe_init(back, B::ST, 4);
        fence_mbar_init();
    }
    grid_dependents();
    grid_wait();  // the images, and the table and order, of the launches before
    WalkUnit u;
    if (!walk_unit<F::kCols>(p, co, order, chunk_slots, u)) return;
    __syncthreads();
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (lane == 0 && warp == 8) forward_copies<F>(u, fwd, p, &tm_q, &tm_k, &tm_v, images);
        if (lane == 0 && warp == 9) back_copies<B>(u, back, p, &tm_q, &tm_k, &tm_do, images);
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 248;");
        walk_back<B, NT>(u, back, p, gr, records, warp - 4, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        walk_forward<F, NT>(u, fwd, p, records, warp, lane);
    }
    __syncthreads();
    if (tid == 0 && *abort_s && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
}

// ============================================================== the rest ==
// A CTA of 8 warps for every SM, each going over its share of the (chunk, q/k head) units and over the value
// heads of each.  What the next value head needs is copied as soon as its place is free: S and dO once S and X
// have been read (S goes where X was), U and W behind the 64 x 64 products, X once dO is in registers.
// 8192 tokens x 16/32 heads: 377 us, 420 with a CTA for every unit, whose first copies nothing hides.  What bounds it
// is mma.sync at two warps an SM quarter (255 registers a thread): the tensor pipe is busy 47% of the time.
// SPLIT: the CTAs of a cluster take a value head each of one unit and add up dq and dk in one another's shared memory.
// Warp (mr, nh): tokens 16 mr, channels 64 nh of dq and dk.
// Of the 64 x 64 products the warps nh = 0 form dP and Q K^T, the others dA and K K^T; the two warps of an
// SM quarter have row blocks mr and 3 - mr, so that the quarters' triangles are even.
constexpr int kRestThreads = 256;
struct RestSmem {
    static constexpr uint32_t SX = 0, kSX = 65536;   // S and X of a record, in turn in either place
    static constexpr uint32_t U = 131072, W = 163840;
    static constexpr uint32_t K = 196608, Q = 212992;
    static constexpr uint32_t G = 229376;            // the image's vectors
    static constexpr uint32_t BARS = G + 1328;       // u64: K and Q, S and dO, X, U and W
    static constexpr uint32_t TOTAL = BARS + 32;
    static constexpr uint32_t ALLOC = TOTAL + 1024;
    // over S once it and X have been read; behind them the next dO
    static constexpr uint32_t M = 0, E = 8192;       // bf16 [64][64], 128B-swizzled
    static constexpr uint32_t P = 16384;             // f32: parts of the sums, below
    static constexpr uint32_t DO = 32768;            // [2][64][128 B], 128B-swizzled
};
static_assert(RestSmem::ALLOC <= 232448 && RestSmem::BARS % 8 == 0, "shared memory");
// parts (floats): a per nh [2][64], w per nh [2][64], the pairs' sums per warp [8][64], db [64],
// <X, S> per warp [8]
constexpr int kPtA = 0, kPtW = 128, kPtC = 256, kPtB = 768, kPtI = 832;

template <bool SPLIT>
__global__ void __launch_bounds__(kRestThreads, 1)
    kda_gdn_grad_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_do, const GdnArgs p, const GdnBackwardArgs gr,
                        const int32_t* __restrict__ co, const uint8_t* __restrict__ images, int64_t chunk_slots,
                        const uint8_t* __restrict__ records) {
    using L = RestSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.num_seqs, Hv = p.Hv, group = Hv / p.Hk;
    grid_wait();  // the walks' records
    if (!table_ok(p, co)) return;
    const int units = table_at(p, co, N) * p.Hk;
    // The first token and the number of tokens of a unit's chunk; units come in rising order.
    int seq = 0, tok0, Lc, next_tok0 = 0, next_Lc = 0;
    auto locate = [&](int unit, int& tok, int& len) {
        if (unit >= units) return false;
        const int j = unit / p.Hk;
        while (seq + 1 < N && table_at(p, co, seq + 1) <= j) ++seq;
        const int64_t t0 = static_cast<int64_t>(p.cu_seqlens[seq]) + static_cast<int64_t>(j - table_at(p, co, seq)) * C;
        const int64_t rem = p.cu_seqlens[seq + 1] - t0;
        tok = static_cast<int>(t0);
        len = static_cast<int>(rem < C ? rem : C);
        return KDA_BOUNDS(seq >= 0 && seq < N && j < chunk_slots && t0 >= 0 && len >= 1 && t0 + len <= p.total_tokens,
                          p.device_status);
    };
    const int rank = SPLIT ? static_cast<int>(blockIdx.x) % group : 0;  // in the cluster: the value head it takes
    int unit = SPLIT ? static_cast<int>(blockIdx.x) / group : static_cast<int>(blockIdx.x);
    if (!locate(unit, tok0, Lc)) return;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
    float* const gs = reinterpret_cast<float*>(sm + L::G);
    // the copies of value head hh of a unit, whose chunk starts at token tok: record and image (j Hv + h)
    auto record = [&](int u, int hh) {
        return records + (static_cast<size_t>(u / p.Hk) * Hv + static_cast<size_t>(u % p.Hk) * group + hh) * kRecStride;
    };
    auto issue_kq = [&](int u, int tok) {
        mbar_arrive_expect_tx(&bars[0], 32768);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
            tma_load_3d(sm + L::K + kh * 8192, &tm_k, &bars[0], 64 * kh, u % p.Hk, tok);
            tma_load_3d(sm + L::Q + kh * 8192, &tm_q, &bars[0], 64 * kh, u % p.Hk, tok);
        }
    };
    auto issue_s = [&](int u, int hh, int tok, uint32_t s_at, uint32_t x_at) {  // dO through X's place
        mbar_arrive_expect_tx(&bars[1], 65536 + 16384);
        bulk_g2s(sm + s_at, record(u, hh) + kRecS, 65536, &bars[1]);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
            tma_load_3d(sm + x_at + L::DO + kh * 8192, &tm_do, &bars[1], 64 * kh, u % p.Hk * group + hh, tok);
    };
    auto issue_x = [&](int u, int hh, uint32_t x_at) {
        mbar_arrive_expect_tx(&bars[2], 65536);
        bulk_g2s(sm + x_at, record(u, hh) + kRecX, 65536, &bars[2]);
    };
    auto issue_uw = [&](int u, int hh) {
        mbar_arrive_expect_tx(&bars[3], 65536);
        bulk_g2s(sm + L::U, record(u, hh) + kRecU, 65536, &bars[3]);  // W follows U
    };
    auto image_vec = [&](int u, int hh) {
        return reinterpret_cast<const float*>(
            images + (static_cast<size_t>(u / p.Hk) * Hv + static_cast<size_t>(u % p.Hk) * group + hh) * kImgStrideBwd + kImgG);
    };
    constexpr int kVec = 5 * C + 4;
    static_assert(kRecW == kRecU + 32768 && L::W == L::U + 32768 && kVec <= 2 * kRestThreads, "layouts");
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&bars[i], 1);
        fence_mbar_init();
        issue_s(unit, rank, tok0, L::SX, L::SX + L::kSX);
        issue_uw(unit, rank);
        issue_kq(unit, tok0);
    }
    for (int e = tid; e < kVec; e += kRestThreads) gs[e] = image_vec(unit, rank)[e];
    __syncthreads();
    bool ok = true;
    const int g = lane >> 2, t = lane & 3;
    const int nh = warp >> 2, mr = nh ? 7 - warp : warp;
    const int lr = lane & 15, lc = lane >> 4;                                      // row-major A operand
    const uint32_t la = ((lane >> 3) & 1) * 2048 + (lane >> 4) * 128 + (lane & 7) * 16;  // the same, of a record
    const uint32_t lb = (lane >> 4) * 2048 + ((lane >> 3) & 1) * 128 + (lane & 7) * 16;  // B from its [n][k] rows
    const int br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;          // B operand from [n][k] rows
    const int kr = (lane & 7) + (((lane >> 3) & 1) << 3), kc = lane >> 4;          // B operand from [k][n] rows
    const uint32_t base = smem_u32(sm);
    float dq[8][4], dk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[n][e] = dk[n][e] = 0.f;

    uint32_t kq_par = 0;
    for (int it = 0, hh = rank;; ++it) {  // value head hh of a unit
        const uint32_t par = it & 1, s_at = L::SX + L::kSX * par, x_at = L::SX + L::kSX * (par ^ 1);
        float* const parts = reinterpret_cast<float*>(sm + s_at + L::P);
        const bool first = SPLIT || hh == 0;  // of the unit
        if (first && Lc < C) {  // rows behind the sequence's end
            ok = mbar_wait_pipe(&bars[0], kq_par) && ok;
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            for (int e = tid; e < (C - Lc) * 16; e += kRestThreads) {
                const uint32_t off = (e & 1) * 8192 + sw128_chunk(Lc + (e >> 4), (e >> 1) & 7);
                *reinterpret_cast<uint4*>(sm + L::K + off) = z;
                *reinterpret_cast<uint4*>(sm + L::Q + off) = z;
            }
        }
        uint32_t dof[8][4];  // dO rows 16 mr as A operand
        ok = mbar_wait_pipe(&bars[1], par) && ok;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ldsm4(dof[k], base + x_at + L::DO + (k >> 2) * 8192 + sw128_chunk(16 * mr + lr, 2 * (k & 3) + lc));
            const bool r0 = 16 * mr + g < Lc, r1 = 16 * mr + g + 8 < Lc;
            if (!r0) dof[k][0] = dof[k][2] = 0u;
            if (!r1) dof[k][1] = dof[k][3] = 0u;
        }
        __syncthreads();  // the vectors (and the cleared rows) are there, dO's tile has been read
        if (tid == 0) issue_x(unit, hh, x_at);
        float eg[2], eo[2], be[2], gh[2], gl[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            gh[e] = gs[kVecGh + 16 * mr + g + 8 * e];
            gl[e] = gs[kVecGl + 16 * mr + g + 8 * e];
            eg[e] = gs[kVecEg + 16 * mr + g + 8 * e];
            eo[e] = gs[kVecEo + 16 * mr + g + 8 * e];
            be[e] = gs[kVecB + 16 * mr + g + 8 * e];
        }
        // an accumulator's rows against the same rows of q or k, over this warp's channels
        auto row_dots = [&](const float (&acc)[8][4], uint32_t tile, float (&d)[2]) {
            d[0] = d[1] = 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 x = unpack_bf16(*reinterpret_cast<const uint32_t*>(
                        sm + tile + nh * 8192 + sw128_chunk(16 * mr + g + 8 * e, n) + 4 * t));
                    d[e] = fmaf(acc[n][2 * e], x.x, fmaf(acc[n][2 * e + 1], x.y, d[e]));
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                d[e] += __shfl_xor_sync(0xffffffffu, d[e], 1);
                d[e] += __shfl_xor_sync(0xffffffffu, d[e], 2);
            }
        };
        float row_a[2], row_w[2];
        ok = mbar_wait_pipe(&bars[3], par) && ok;
        {  // dO S^T and W S^T
            float a1[8][4], a2[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) a1[n][e] = a2[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t wh[4], wl[4];
                const uint32_t wa = base + L::W + la + mr * 4096 + k * 256;
                ldsm4(wh, wa);
                ldsm4(wl, wa + 16384);
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t sh[4], sl[4];
                    const uint32_t sa = base + s_at + lb + (4 * nh + np) * 4096 + k * 256;
                    ldsm4(sh, sa);
                    ldsm4(sl, sa + 32768);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma16(a1[2 * np + n], dof[k], sh[2 * n], sh[2 * n + 1]);
                        mma16(a2[2 * np + n], wh, sh[2 * n], sh[2 * n + 1]);
                        mma16(a1[2 * np + n], dof[k], sl[2 * n], sl[2 * n + 1]);
                        mma16(a2[2 * np + n], wh, sl[2 * n], sl[2 * n + 1]);
                        mma16(a2[2 * np + n], wl, sh[2 * n], sh[2 * n + 1]);
                    }
                }
            }
            float d1[2], d2[2];
            if (first) ok = mbar_wait_pipe(&bars[0], kq_par) && ok;
            row_dots(a1, L::Q, d1);
            row_dots(a2, L::K, d2);
#pragma unroll
            for (int e = 0; e < 2; ++e) row_a[e] = eg[e] * (d1[e] - be[e] * d2[e]);
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dq[n][e] = fmaf(eg[e >> 1], a1[n][e], dq[n][e]);
                    dk[n][e] = fmaf(-eg[e >> 1] * be[e >> 1], a2[n][e], dk[n][e]);
                }
        }
        ok = mbar_wait_pipe(&bars[2], par) && ok;
        {  // U X^T
            float a1[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) a1[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t uh[4], ul[4];
                const uint32_t ua = base + L::U + la + mr * 4096 + k * 256;
                ldsm4(uh, ua);
                ldsm4(ul, ua + 16384);
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t xh[4], xl[4];
                    const uint32_t xa = base + x_at + lb + (4 * nh + np) * 4096 + k * 256;
                    ldsm4(xh, xa);
                    ldsm4(xl, xa + 32768);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma16(a1[2 * np + n], uh, xh[2 * n], xh[2 * n + 1]);
                        mma16(a1[2 * np + n], uh, xl[2 * n], xl[2 * n + 1]);
                        mma16(a1[2 * np + n], ul, xh[2 * n], xh[2 * n + 1]);
                    }
                }
            }
            row_dots(a1, L::K, row_w);
#pragma unroll
            for (int e = 0; e < 2; ++e) row_w[e] *= eo[e];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) dk[n][e] = fmaf(eo[e >> 1], a1[n][e], dk[n][e]);
        }
        float inner = 0.f;  // <X, S>
        for (int e = tid; e < 2048; e += kRestThreads) {
            const uint4 sh = *reinterpret_cast<const uint4*>(sm + s_at + 16 * e);
            const uint4 sl = *reinterpret_cast<const uint4*>(sm + s_at + 32768 + 16 * e);
            const uint4 xh = *reinterpret_cast<const uint4*>(sm + x_at + 16 * e);
            const uint4 xl = *reinterpret_cast<const uint4*>(sm + x_at + 32768 + 16 * e);
            const uint32_t* a = &sh.x;
            const uint32_t* b = &sl.x;
            const uint32_t* c = &xh.x;
            const uint32_t* d = &xl.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 s1 = unpack_bf16(a[i]), s2 = unpack_bf16(b[i]), x1 = unpack_bf16(c[i]), x2 = unpack_bf16(d[i]);
                inner = fmaf(s1.x + s2.x, x1.x + x2.x, inner);
                inner = fmaf(s1.y + s2.y, x1.y + x2.y, inner);
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, off);
        const bool last = SPLIT || hh + 1 == group;  // of the unit; the next item is another's first head then
        const int next_unit = last ? unit + static_cast<int>(gridDim.x) : unit, next_hh = last ? 0 : hh + 1;
        const bool more = !SPLIT && (!last || locate(next_unit, next_tok0, next_Lc));
        __syncthreads();  // S and X have been read: M, E and the parts take S's place, the next S X's
        if (tid == 0 && more) issue_s(next_unit, next_hh, last ? next_tok0 : tok0, x_at, s_at);
        if (t == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                parts[kPtA + 64 * nh + 16 * mr + g + 8 * e] = row_a[e];
                parts[kPtW + 64 * nh + 16 * mr + g + 8 * e] = row_w[e];
            }
        }
        if (lane == 0) parts[kPtI + warp] = inner;
        // The 64 x 64 products, 32 columns (two blocks) at a time: dP = dO U^T with Q K^T, or W U^T with K K^T.
        float left[2] = {0.f, 0.f};  // of rows g and g + 8: the sums of the columns so far
#pragma unroll 1
        for (int ph = 0; ph < 2; ++ph) {
            if (2 * ph > mr) {  // above the diagonal
                if (g == 0) {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        *reinterpret_cast<float2*>(parts + kPtC + 64 * warp + 32 * ph + 8 * n + 2 * t) = make_float2(0.f, 0.f);
                }
                continue;
            }
            float a1[4][4], kk[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) a1[n][e] = kk[n][e] = 0.f;
            if (nh) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t wh[4], wl[4], ga[4];
                    const uint32_t aoff = (k >> 2) * 8192 + sw128_chunk(16 * mr + lr, 2 * (k & 3) + lc);
                    ldsm4(wh, base + L::W + la + mr * 4096 + k * 256);
                    ldsm4(wl, base + L::W + 16384 + la + mr * 4096 + k * 256);
                    ldsm4(ga, base + L::K + aoff);
#pragma unroll
                    for (int np = 0; np < 2; ++np) {
                        uint32_t uh[4], ul[4], kf[4];
                        const uint32_t off = (k >> 2) * 8192 + sw128_chunk(32 * ph + 16 * np + br, 2 * (k & 3) + bc);
                        ldsm4(uh, base + L::U + lb + (2 * ph + np) * 4096 + k * 256);
                        ldsm4(ul, base + L::U + 16384 + lb + (2 * ph + np) * 4096 + k * 256);
                        ldsm4(kf, base + L::K + off);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma16(kk[2 * np + n], ga, kf[2 * n], kf[2 * n + 1]);
                            mma16(a1[2 * np + n], wh, uh[2 * n], uh[2 * n + 1]);
                            mma16(a1[2 * np + n], wh, ul[2 * n], ul[2 * n + 1]);
                            mma16(a1[2 * np + n], wl, uh[2 * n], uh[2 * n + 1]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t ga[4];
                    ldsm4(ga, base + L::Q + (k >> 2) * 8192 + sw128_chunk(16 * mr + lr, 2 * (k & 3) + lc));
#pragma unroll
                    for (int np = 0; np < 2; ++np) {
                        uint32_t uh[4], ul[4], kf[4];
                        const uint32_t off = (k >> 2) * 8192 + sw128_chunk(32 * ph + 16 * np + br, 2 * (k & 3) + bc);
                        ldsm4(uh, base + L::U + lb + (2 * ph + np) * 4096 + k * 256);
                        ldsm4(ul, base + L::U + 16384 + lb + (2 * ph + np) * 4096 + k * 256);
                        ldsm4(kf, base + L::K + off);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma16(kk[2 * np + n], ga, kf[2 * n], kf[2 * n + 1]);
                            mma16(a1[2 * np + n], dof[k], uh[2 * n], uh[2 * n + 1]);
                            mma16(a1[2 * np + n], dof[k], ul[2 * n], ul[2 * n + 1]);
                        }
                    }
                }
            }
            // M or E, and the pairs' sums: over rows i >= t of the sums over columns j < t
            const float sgn = nh ? -1.f : 1.f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float cs[2] = {0.f, 0.f};
                const int jj = 32 * ph + 8 * n + 2 * t;
                const float2 ch = *reinterpret_cast<const float2*>(gs + kVecGh + jj);
                const float2 cl = *reinterpret_cast<const float2*>(gs + kVecGl + jj);
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int i = 16 * mr + g + 8 * e2;
                    const int last = i < Lc ? i - nh : -1;  // columns up to this one count
                    const float f = nh ? be[e2] : 1.f;
                    float m[2], d[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = (gh[e2] - (e ? ch.y : ch.x)) + (gl[e2] - (e ? cl.y : cl.x));
                        const bool in = jj + e <= last;
                        const float gam = f * exp2_sfu(in ? x : 0.f);
                        const float v = sgn * a1[n][2 * e2 + e];
                        if (nh && jj + e == i) parts[kPtB + i] = a1[n][2 * e2 + e] / be[e2];
                        d[e] = in ? v * (gam * kk[n][2 * e2 + e]) : 0.f;
                        m[e] = in ? gam * v : 0.f;
                    }
                    float sum = d[0] + d[1];  // of the lanes up to this one in the row
                    float y = __shfl_up_sync(0xffffffffu, sum, 1, 4);
                    if (t >= 1) sum += y;
                    y = __shfl_up_sync(0xffffffffu, sum, 2, 4);
                    if (t >= 2) sum += y;
                    y = __shfl_up_sync(0xffffffffu, sum, 1, 4);
                    const float before = left[e2] + (t >= 1 ? y : 0.f);
                    left[e2] += __shfl_sync(0xffffffffu, sum, 3, 4);
                    if (jj <= i) cs[0] += before;
                    if (jj + 1 <= i) cs[1] += before + d[0];
                    *reinterpret_cast<uint32_t*>(sm + s_at + (nh ? L::E : L::M) + sw128_chunk(i, 4 * ph + n) + 4 * t) =
                        pack_bf16(m[0], m[1]);
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    cs[0] += __shfl_xor_sync(0xffffffffu, cs[0], off);
                    cs[1] += __shfl_xor_sync(0xffffffffu, cs[1], off);
                }
                if (g == 0) *reinterpret_cast<float2*>(parts + kPtC + 64 * warp + jj) = make_float2(cs[0], cs[1]);
            }
        }
        __syncthreads();
        float vec[2] = {0.f, 0.f};  // of the next item
        if (more) {
            if (tid == 0) issue_uw(next_unit, next_hh);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (tid + kRestThreads * e < kVec) vec[e] = image_vec(next_unit, next_hh)[tid + kRestThreads * e];
        }
        // dq += M K, dk += E K (columns up to the own rows), dk += E^T K + M^T Q (rows from the own columns on)
#pragma unroll 1
        for (int k = 0; k <= mr; ++k) {
            uint32_t am[4], ae[4];
            ldsm4(am, base + s_at + L::M + sw128_chunk(16 * mr + lr, 2 * k + lc));
            ldsm4(ae, base + s_at + L::E + sw128_chunk(16 * mr + lr, 2 * k + lc));
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t kf[4];
                ldsm4t(kf, base + L::K + nh * 8192 + sw128_chunk(16 * k + kr, 2 * np + kc));
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma16(dq[2 * np + n], am, kf[2 * n], kf[2 * n + 1]);
                    mma16(dk[2 * np + n], ae, kf[2 * n], kf[2 * n + 1]);
                }
            }
        }
#pragma unroll 1
        for (int k = mr; k < 4; ++k) {
            uint32_t tm[4], te[4];
            ldsm4t(tm, base + s_at + L::M + sw128_chunk(16 * k + br, 2 * mr + bc));
            ldsm4t(te, base + s_at + L::E + sw128_chunk(16 * k + br, 2 * mr + bc));
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t kf[4], qf[4];
                const uint32_t off = nh * 8192 + sw128_chunk(16 * k + kr, 2 * np + kc);
                ldsm4t(kf, base + L::K + off);
                ldsm4t(qf, base + L::Q + off);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma16(dk[2 * np + n], te, kf[2 * n], kf[2 * n + 1]);
                    mma16(dk[2 * np + n], tm, qf[2 * n], qf[2 * n + 1]);
                }
            }
        }
        const int hk = unit % p.Hk, h = hk * group + hh;
        if (warp == 0) {  // the decays' and b's gradients, two tokens a lane
            float ra[2], rw[2], pairs[2], in = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * lane + e;
                ra[e] = parts[kPtA + r] + parts[kPtA + 64 + r];
                rw[e] = parts[kPtW + r] + parts[kPtW + 64 + r];
                pairs[e] = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) pairs[e] += parts[kPtC + 64 * w + r];
            }
            if (lane < 8) in = parts[kPtI + lane];
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) in += __shfl_xor_sync(0xffffffffu, in, off);
            in = __shfl_sync(0xffffffffu, in, 0) * gs[kVecEc];
            float sa = ra[0] + ra[1], sw = rw[0] + rw[1];  // from this lane's tokens on; up to them
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float ya = __shfl_down_sync(0xffffffffu, sa, off), yw = __shfl_up_sync(0xffffffffu, sw, off);
                if (lane + off < 32) sa += ya;
                if (lane >= off) sw += yw;
            }
            float after = __shfl_down_sync(0xffffffffu, sa, 1), before = __shfl_up_sync(0xffffffffu, sw, 1);
            if (lane == 31) after = 0.f;
            if (lane == 0) before = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * lane + e;
                const float a_on = after + (e ? ra[1] : ra[0] + ra[1]), w_before = e ? before + rw[0] : before;
                if (r < Lc) {
                    gr.grad_log_decay[static_cast<int64_t>(tok0 + r) * Hv + h] = (pairs[e] + a_on) + (w_before + in);
                    gr.grad_beta[static_cast<int64_t>(tok0 + r) * Hv + h] = parts[kPtB + r];
                }
            }
        }
        fence_async_smem();  // M, E, the parts and the cleared rows, before the next copies
        if (__syncthreads_or(!ok) && !SPLIT) {  // a bounded wait expired: no copy is left in flight
            if (more) {
                (void)mbar_wait(&bars[1], par ^ 1, kDrainLimit);
                (void)mbar_wait(&bars[3], par ^ 1, kDrainLimit);
            }
            break;
        }
        if constexpr (SPLIT) {  // the heads' sums, in order; each CTA of the cluster takes 64 / group of a thread's values
            float* const mine = reinterpret_cast<float*>(sm + L::SX);  // [64][threads]
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mine[(4 * n + e) * kRestThreads + tid] = dq[n][e];
                    mine[(32 + 4 * n + e) * kRestThreads + tid] = dk[n][e];
                }
            cluster_sync();
            const uint32_t at = smem_u32(mine + tid);
            for (int i = rank * (64 / group); i < (rank + 1) * (64 / group); i += 2) {
                float x = 0.f, y = 0.f;
                for (int k = 0; k < group; ++k) {
                    const uint32_t there = cluster_address(at + i * kRestThreads * 4, k);
                    x += cluster_load(there);
                    y += cluster_load(there + kRestThreads * 4);
                }
                const int row = 16 * mr + g + 8 * ((i >> 1) & 1);
                if (row < Lc) {
                    const int64_t off =
                        (static_cast<int64_t>(tok0 + row) * p.Hk + hk) * D + 64 * nh + 2 * t + 8 * ((i & 31) >> 2);
                    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(i < 32 ? gr.grad_q : gr.grad_k) + off) =
                        pack_bf16(x, y);
                }
            }
            cluster_sync();  // the others have read this CTA's
            break;
        } else {
            if (last) {
                if (tid == 0 && more) issue_kq(next_unit, next_tok0);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * mr + g + 8 * e;
                    if (row >= Lc) continue;
                    const int64_t off = (static_cast<int64_t>(tok0 + row) * p.Hk + hk) * D + 64 * nh + 2 * t;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(gr.grad_q) + off + 8 * n) =
                            pack_bf16(dq[n][2 * e], dq[n][2 * e + 1]);
                        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(gr.grad_k) + off + 8 * n) =
                            pack_bf16(dk[n][2 * e], dk[n][2 * e + 1]);
                    }
                }
                if (!more) break;
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dq[n][e] = dk[n][e] = 0.f;
                unit = next_unit;
                tok0 = next_tok0;
                Lc = next_Lc;
                kq_par ^= 1;
            }
            hh = next_hh;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (tid + kRestThreads * e < kVec) gs[tid + kRestThreads * e] = vec[e];
        }
    }
    if (!ok && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
}

template <int NT>
cudaError_t launch_walks(const GdnArgs& a, const GdnBackwardArgs& b, const GdnWorkspace& w, const CUtensorMap& tm_q,
                         const CUtensorMap& tm_k, cudaStream_t stream) {
    using L = WalksCfg<NT>;
    using F = typename L::F;
    static int configured[64];
    const cudaError_t err = set_smem(kda_gdn_walks_kernel<NT>, L::ALLOC, configured);
    if (err != cudaSuccess) return err;
    CUtensorMap tm_v, tm_do;
    const CUtensorMapSwizzle sw = F::kVRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!make_tensor_map(&tm_v, a.v, a.Hv, a.total_tokens, F::kCols, C, sw) ||
        !make_tensor_map(&tm_do, b.grad_o, a.Hv, a.total_tokens, F::kCols, C, sw))
        return cudaErrorInvalidValue;
    const int64_t blocks = static_cast<int64_t>(a.num_seqs) * a.Hv * (D / F::kCols);
    return launch_dependent(kda_gdn_walks_kernel<NT>, blocks, L::kThreads, L::ALLOC, stream, tm_q, tm_k, tm_v, tm_do, a, b,
                            w.table, w.order, w.images, w.chunks, w.records);
}

}  // namespace

cudaError_t launch_gdn_backward(const GdnArgs& a, const GdnBackwardArgs& b, const GdnWorkspace& w, const CUtensorMap& tm_q,
                                const CUtensorMap& tm_k, cudaStream_t stream) {
    // columns a CTA as in the prefill's scan
    cudaError_t err = gdn_narrow(a.num_seqs, a.Hv) ? launch_walks<1>(a, b, w, tm_q, tm_k, stream)
                                                   : launch_walks<2>(a, b, w, tm_q, tm_k, stream);
    CUtensorMap tm_do;
    if (!make_tensor_map(&tm_do, b.grad_o, a.Hv, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    static int configured[64];
    if (err == cudaSuccess) err = set_smem(kda_gdn_grad_kernel<false>, RestSmem::ALLOC, configured);
    if (err != cudaSuccess) return err;
    // Where the value heads of all units find an SM each, a group's share a unit as a cluster (333 tokens in three
    // sequences x 4/8 heads, the whole call: 58 us, one head after the other 64).
    const int group = a.Hv / a.Hk;
    if ((group == 2 || group == 4 || group == 8) && w.chunks * a.Hv <= device_sm_count()) {
        static int configured_split[64];
        err = set_smem(kda_gdn_grad_kernel<true>, RestSmem::ALLOC, configured_split);
        if (err != cudaSuccess) return err;
        return launch_dependent_clusters(group, kda_gdn_grad_kernel<true>, w.chunks * a.Hv, kRestThreads, RestSmem::ALLOC,
                                         stream, tm_q, tm_k, tm_do, a, b, w.table, w.images, w.chunks, w.records);
    }
    const int64_t blocks = std::min<int64_t>(w.chunks * a.Hk, device_sm_count());
    return launch_dependent(kda_gdn_grad_kernel<false>, blocks, kRestThreads, RestSmem::ALLOC, stream, tm_q, tm_k, tm_do, a,
                            b, w.table, w.images, w.chunks, w.records);
}

}  // namespace kda
