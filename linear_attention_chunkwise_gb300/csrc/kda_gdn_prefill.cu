// kda_gdn_prefill.cu -- the gated delta rule, chunkwise, for bf16 inputs.
//
// With g the inclusive cumulative log decay of a 64-token chunk, S0 the state at its start, and
// G_ij = exp(g_i - g_j) (i >= j):
//   A_ij = b_i G_ij (k_i . k_j)  (i > j),   T = (I + A)^-1,   P_ij = G_ij (q_i . k_j)  (i >= j)
//   U = T Diag(b) (V - Diag(e^g) K S0),   O = Diag(e^g) Q S0 + P U,   S1 = e^gC S0 + K^T Diag(e^(gC - g)) U
// (the chunk form of "Understanding Kimi Delta Attention" (pyshine), "The Chunkwise DPLR Algorithm",
// with its scalar gate).  Unlike the channel-wise gate, the scalar one multiplies the Gram matrices
// afterwards, so every product has the raw bf16 k or q as one operand, and the decays enter as
// exponentials of differences: no lower limit on log_decay.  What else a state's products take (the state itself, the
// right-hand side, T, U) is two bf16 terms, x = hi + lo with |x - hi - lo| <= 2^-17 |x|, accumulated in fp32: S_final is good
// to about 4e-6 of itself, where fp32 products give up to 4e-7.  The outputs' products take one term of S, P
// and U, since o is rounded to bf16 anyway: 3.3e-3 of itself, where the rounding alone is 1.7e-3.  (Second terms there
// would be 52 more products a chunk beside the 200 of the mma.sync scan's warps; the tcgen05 scan has neither the TMEM columns
// for U's nor the shared memory for P's.)
//
// pass 0  chunk table (launch_chunk_table)
// pass 1  one CTA per (chunk, q/k head, up to four of its value heads): Gram matrices, T, P, decays -> images in the workspace
// pass 2  scan: the walk of kda_gdn_walk.cuh over the chunks of every (sequence, value head).
#include <algorithm>

#include "kda_gdn_walk.cuh"

namespace kda {
namespace {

using namespace gdn;

// =============================================================== pass 1 ==
// One CTA of four warps for a (chunk, q/k head) and `hp` of its value heads, which share the Gram
// matrices: K K^T's and Q K^T's ten 16 x 16 blocks on and below the diagonal stay in the warps' registers, at
// most three of each to a warp.  Per value head: the decays and
// b make A and P of them; the 16 x 16 diagonal blocks of I + A are inverted by forward substitution
// in fp32 (stable for any A; a column for each of 64 threads); then warp j forms block column j of the
// inverse, T_ij = -D_i sum_{j <= k < i} A_ik T_kj, by mma.sync on two-term operands, its blocks staying in
// its registers.  (The block products in fp32 on the CUDA cores and one value head a CTA, 256 threads:
// 109 us for 8192 tokens x 32 heads, 16.1 K warp instructions a (chunk, head); a warp for every row of blocks
// and the decays of one value head after the other: 70 us; now 63.  The issue slots are 38% busy, HBM 34%: the
// rest is the latency of a CTA's steps, five CTAs an SM: 61.6 us, four of them 66.  The 96 registers that leaves spill 27
// words of the plain images' kernel and 35 of the tiles'.)
constexpr int kPrepThreads = 128;
constexpr int kPrepHeads = 4;  // most value heads of a CTA: a warp for each one's decays

struct PrepSmem {
    static constexpr uint32_t K = 0, Q = 16384;  // 2 x [64][128 B] each, 128B-swizzled
    static constexpr uint32_t AH = 0;            // two terms of A's blocks, the diagonal ones inverted (over K and
    static constexpr uint32_t AL = kTriBytes;    // Q once the Gram matrices are out)
    static constexpr uint32_t DG = 16384;        // f32 [4][16][17]: diagonal blocks of A
    static constexpr uint32_t G = 32768;         // f32 [heads][3][64]: g (two terms, base 2), beta
    static constexpr uint32_t BAR = G + kPrepHeads * 3 * C * 4;
    static constexpr uint32_t TOTAL = BAR + 16;
    static constexpr uint32_t ALLOC = TOTAL + 1024;
};

// log decays below this (a decay of 0 in fp32, as -inf) are taken as this, so that differences of the
// cumulative sums stay numbers.
constexpr float kDecayFloor = -1e4f;
// In the gradient's images a smaller b, 0 too, is taken as this: U / b is then still what the rows of U
// hold before b multiplies them, and b's own part in every sum is below fp32's rounding.
constexpr float kBetaFloor = 8.271806e-25f;  // 2^-80

template <bool TILE>
__global__ void __launch_bounds__(kPrepThreads, 5)
    kda_gdn_prep_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const GdnArgs p, const int32_t* __restrict__ co, uint8_t* images, int64_t chunk_slots,
                        int32_t hp, bool bwd) {
    using L = PrepSmem;
    constexpr bool tile = TILE;
    const size_t stride = tile ? kImgStrideTile : bwd ? kImgStrideBwd : kImgStride;
    // T's terms and P are three matrices of this many bytes; the vectors follow
    constexpr uint32_t mat = tile ? kTileBytes : kTriBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.num_seqs, Hv = p.Hv, groups = Hv / hp;
    const int j = blockIdx.x / groups, h0 = (blockIdx.x - j * groups) * hp;
    grid_dependents();
    if (!table_ok(p, co)) {
        if (!co && blockIdx.x == 0 && threadIdx.x == 0 && p.device_status) atomicOr(p.device_status, KDA_DEV_BAD_CU_SEQLENS);
        return;
    }
    if (j >= table_at(p, co, N)) return;  // no such chunk
    int seq = 0;
    if (co) {  // the largest n with co[n] <= j
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (co[mid] <= j) lo = mid;
            else hi = mid - 1;
        }
        seq = lo;
    }
    const int64_t t0 = static_cast<int64_t>(p.cu_seqlens[seq]) + static_cast<int64_t>(j - table_at(p, co, seq)) * C;
    const int64_t rem = p.cu_seqlens[seq + 1] - t0;
    const int Lc = static_cast<int>(rem < C ? rem : C);
    if (!KDA_BOUNDS(seq >= 0 && seq < N && j < chunk_slots && t0 >= 0 && Lc >= 1 && t0 + Lc <= p.total_tokens,
                    p.device_status))
        return;

    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar, 32768);
        const int hk = h0 / (Hv / p.Hk);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
            tma_load_3d(sm + L::K + kh * 8192, &tm_k, bar, 64 * kh, hk, static_cast<int32_t>(t0));
            tma_load_3d(sm + L::Q + kh * 8192, &tm_q, bar, 64 * kh, hk, static_cast<int32_t>(t0));
        }
    }
    // A value head's cumulative log decay (base 2, two tokens a lane, in fp64; kept as two fp32 terms), beta, and
    // the image's vectors.
    const int dw = (warp + 3) & 3;  // warp 0, whose first thread is held by the copies it issues, comes last
    if (dw < hp) {
        const int h = h0 + dw;
        float* const g_hi = reinterpret_cast<float*>(sm + L::G) + dw * 3 * C;
        float* const g_lo = g_hi + C;
        float* const beta_s = g_lo + C;
        double x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            float ld = 0.f, b = 0.f;
            if (r < Lc) {
                ld = p.log_decay[(t0 + r) * Hv + h];
                b = p.beta[(t0 + r) * Hv + h];
            }
            x[e] = static_cast<double>(ld < kDecayFloor ? kDecayFloor : ld) * 1.4426950408889634;
            if (bwd && fabsf(b) < kBetaFloor) b = kBetaFloor;
            beta_s[r] = b;
        }
        double s = x[0] + x[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        const double last = __shfl_sync(0xffffffffu, s, 31);
        float* gv = reinterpret_cast<float*>(images + (static_cast<size_t>(j) * Hv + h) * stride + 3 * mat);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            const double g = e ? s : s - x[1];
            const float hi = static_cast<float>(g);
            const float lo = static_cast<float>(g - hi);
            g_hi[r] = hi;
            g_lo[r] = lo;
            gv[kVecEg + r] = exp2f(static_cast<float>(g));
            gv[kVecEo + r] = exp2f(static_cast<float>(last - g));
            gv[kVecB + r] = beta_s[r];
            if (bwd) {
                gv[kVecGh + r] = hi;
                gv[kVecGl + r] = lo;
            }
        }
        if (lane == 0) gv[kVecEc] = exp2f(static_cast<float>(last));
    }
    bool ok = true;
    if (tid == 0) ok = mbar_wait_pipe(bar, 0);
    if (!ok && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
    __syncthreads();

    // The blocks of warp w (which turns with the CTA, so that no quarter of the SM has the long lists of every
    // one): 0: (0, 0); 1: (1, 0), (1, 1), (3, 3); 2: (2, 0..2); 3: (3, 0..2).
    const int g = lane >> 2, t = lane & 3;
    const int w = (warp + blockIdx.x) & 3;
    const int row2 = w == 1 ? 3 : w, col2 = w == 1 ? 3 : 2;  // of the third one
    float kk[3][2][4], qk[3][2][4];
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) kk[s][n][e] = qk[s][n][e] = 0.f;
    {
        const uint32_t kb = smem_u32(sm + L::K), qb = smem_u32(sm + L::Q);
        const int ar = lane & 15, br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt) {
            const uint32_t off = (kt >> 2) * 8192;
            uint32_t ak[4], aq[4], b[4];
            ldsm4(ak, kb + off + sw128_chunk(16 * w + ar, 2 * (kt & 3) + (lane >> 4)));
            ldsm4(aq, qb + off + sw128_chunk(16 * w + ar, 2 * (kt & 3) + (lane >> 4)));
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                if (s > 0 && w == 0) break;
                if (s == 2 && w == 1) {
                    ldsm4(ak, kb + off + sw128_chunk(48 + ar, 2 * (kt & 3) + (lane >> 4)));
                    ldsm4(aq, qb + off + sw128_chunk(48 + ar, 2 * (kt & 3) + (lane >> 4)));
                }
                ldsm4(b, kb + off + sw128_chunk(16 * (s == 2 ? col2 : s) + br, 2 * (kt & 3) + bc));
                mma16(kk[s][0], ak, b[0], b[1]);
                mma16(kk[s][1], ak, b[2], b[3]);
                mma16(qk[s][0], aq, b[0], b[1]);
                mma16(qk[s][1], aq, b[2], b[3]);
            }
        }
    }
    const uint32_t ah_base = smem_u32(sm + L::AH) + 16 * lane, al_base = smem_u32(sm + L::AL) + 16 * lane;
    float* const dg = reinterpret_cast<float*>(sm + L::DG);
    for (int hh = 0; hh < hp; ++hh) {
        const int h = h0 + hh;
        uint8_t* const img = images + (static_cast<size_t>(j) * Hv + h) * stride;
        const float* const g_hi = reinterpret_cast<const float*>(sm + L::G) + hh * 3 * C;
        const float* const g_lo = g_hi + C;
        const float* const beta_s = g_lo + C;
        __syncthreads();  // K and Q, or the previous head's A, have been read
        // A (two terms; its diagonal blocks in fp32) and P
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            if (s > 0 && w == 0) break;
            const int bi = s == 2 ? row2 : w, bj = s == 2 ? col2 : s;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int jj = 16 * bj + 8 * n + 2 * t;
                const float2 ch = *reinterpret_cast<const float2*>(g_hi + jj);
                const float2 cl = *reinterpret_cast<const float2*>(g_lo + jj);
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {  // rows g and g + 8 of the block
                    const int i = 16 * bi + g + 8 * e2;
                    const float gi = g_hi[i], gl = g_lo[i], b = beta_s[i];
                    const int last = i < Lc ? i : -1;  // columns up to this one count
                    const float d0 = exp2_sfu((gi - ch.x) + (gl - cl.x)), d1 = exp2_sfu((gi - ch.y) + (gl - cl.y));
                    const uint32_t pair = blk_pair(g, e2, n, t);
                    const float p0 = jj <= last ? d0 * qk[s][n][2 * e2] : 0.f;
                    const float p1 = jj + 1 <= last ? d1 * qk[s][n][2 * e2 + 1] : 0.f;
                    uint32_t ph, pl;
                    split2(p0, p1, ph, pl);
                    uint8_t* const pp = img + (tile ? sw128_chunk(i, 2 * bj + n) + 4 * t : tri_blk(bi, bj) + pair);
                    *reinterpret_cast<uint32_t*>(pp + 2 * mat) = ph;
                    if (bwd) {
                        *reinterpret_cast<uint32_t*>(pp + kImgPl) = pl;
                        *reinterpret_cast<uint32_t*>(pp + kImgPl2) = third2(p0, p1, ph, pl);
                    }
                    const float a0 = jj < last ? b * d0 * kk[s][n][2 * e2] : 0.f;
                    const float a1 = jj + 1 < last ? b * d1 * kk[s][n][2 * e2 + 1] : 0.f;
                    if (bi == bj) {
                        float* d = dg + bi * 272 + (g + 8 * e2) * 17 + 8 * n + 2 * t;
                        d[0] = a0;
                        d[1] = a1;
                    } else {
                        uint32_t hi, lo;
                        split2(a0, a1, hi, lo);
                        uint8_t* const ap = sm + tri_blk(bi, bj) + pair;
                        *reinterpret_cast<uint32_t*>(ap + L::AH) = hi;
                        *reinterpret_cast<uint32_t*>(ap + L::AL) = lo;
                    }
                }
            }
        }
        __syncthreads();
        if (tid < 64) {  // D_b = (I + A_bb)^-1, column c of block b
            const int b = tid >> 4, c = tid & 15;
            const float* A = dg + b * 272;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s0 = i == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < i; ++k) {
                    if (k & 1) s1 = fmaf(-A[i * 17 + k], x[k], s1);
                    else s0 = fmaf(-A[i * 17 + k], x[k], s0);
                }
                x[i] = s0 + s1;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t off = tri_blk(b, b) + blk_pair(i & 7, i >> 3, c >> 3, 0) + 2 * (c & 7);
                const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
                *reinterpret_cast<__nv_bfloat16*>(sm + L::AH + off) = hi;
                *reinterpret_cast<__nv_bfloat16*>(sm + L::AL + off) = __float2bfloat16_rn(x[i] - __bfloat162float(hi));
            }
        }
        __syncthreads();
        // Block column w of the inverse by warp w.  T_ww = D_w from shared memory, the others from the products.
        {
            BTerms T[4][2];  // blocks (k, w) as B operands, two 8-column halves
            {
                uint32_t bh[4], bl[4];
                ldsm4t(bh, ah_base + tri_blk(w, w));
                ldsm4t(bl, al_base + tri_blk(w, w));
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < 2; ++n)  // every slot below the diagonal is overwritten before its use
                        T[k][n] = BTerms{bh[2 * n], bh[2 * n + 1], bl[2 * n], bl[2 * n + 1]};
            }
            auto store = [&](int i, const float (&x)[2][4]) {  // block (i, w)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        uint32_t hi, lo;
                        split2(x[n][2 * e2], x[n][2 * e2 + 1], hi, lo);
                        uint8_t* const tp = img + (tile ? sw128_chunk(16 * i + g + 8 * e2, 2 * w + n) + 4 * t
                                                        : tri_blk(i, w) + blk_pair(g, e2, n, t));
                        *reinterpret_cast<uint32_t*>(tp) = hi;
                        *reinterpret_cast<uint32_t*>(tp + mat) = lo;
                    }
            };
            {  // the diagonal block itself, as accumulators hold it
                float x[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        const uint32_t off = tri_blk(w, w) + blk_pair(g, e2, n, t);
                        const float2 hi = unpack_bf16(*reinterpret_cast<const uint32_t*>(sm + L::AH + off));
                        const float2 lo = unpack_bf16(*reinterpret_cast<const uint32_t*>(sm + L::AL + off));
                        x[n][2 * e2] = hi.x + lo.x;
                        x[n][2 * e2 + 1] = hi.y + lo.y;
                    }
                store(w, x);
            }
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                if (i <= w) continue;
                float x[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
                uint32_t ah[4], al[4];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    if (k < w || k >= i) continue;
                    ldsm4(ah, ah_base + tri_blk(i, k));
                    ldsm4(al, al_base + tri_blk(i, k));
#pragma unroll
                    for (int n = 0; n < 2; ++n) mma16(x[n], ah, T[k][n].h0, T[k][n].h1);
#pragma unroll
                    for (int n = 0; n < 2; ++n) mma16(x[n], ah, T[k][n].l0, T[k][n].l1);
#pragma unroll
                    for (int n = 0; n < 2; ++n) mma16(x[n], al, T[k][n].h0, T[k][n].h1);
                }
                BTerms X[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = -x[n][e];
                    X[n] = b_terms(x[n]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
                }
                ldsm4(ah, ah_base + tri_blk(i, i));
                ldsm4(al, al_base + tri_blk(i, i));
#pragma unroll
                for (int n = 0; n < 2; ++n) mma16(x[n], ah, X[n].h0, X[n].h1);
#pragma unroll
                for (int n = 0; n < 2; ++n) mma16(x[n], ah, X[n].l0, X[n].l1);
#pragma unroll
                for (int n = 0; n < 2; ++n) mma16(x[n], al, X[n].h0, X[n].h1);
#pragma unroll
                for (int n = 0; n < 2; ++n) T[i][n] = b_terms(x[n]);
                store(i, x);
            }
        }
    }
}

// =============================================================== pass 2 ==
// Four warps of 8 columns: the narrow scan (kda_gdn_wide.cu has the one for many pairs).  8192 tokens x 32 heads: 205 us,
// 1.54 us a chunk, the chain of a warp's products; the tensor pipe is 52% busy.  One long sequence in pieces, prep of the
// next one beside a piece's scan, gains nothing: 270 us with 64 chunks a piece, 277 with 42, 290 with 32, against 272
// (the prep beside it slows the chain by what it saves).
struct ScanCfg : ForwardCfg<1, 4, 3, false> {
    using L = ForwardCfg<1, 4, 3, false>;
    static constexpr int kThreads = 160;  // four walking warps and the one that copies
    static constexpr uint32_t BARS = ST * L::STAGE;  // full[ST], empty[ST]
    static constexpr uint32_t ABORT = BARS + 16 * ST;
    static constexpr uint32_t ALLOC = ABORT + 16 + 1024;
    static_assert(ALLOC <= 232448, "shared memory");
};

__global__ void __launch_bounds__(ScanCfg::kThreads, 1)
    kda_gdn_scan_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const GdnArgs p, const int32_t* __restrict__ co,
                        const int32_t* __restrict__ order, const uint8_t* __restrict__ images, int64_t chunk_slots) {
    using L = ScanCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WalkPipe pipe{sm, reinterpret_cast<uint64_t*>(sm + L::BARS), reinterpret_cast<uint64_t*>(sm + L::BARS) + L::ST,
                        reinterpret_cast<volatile int*>(sm + L::ABORT)};
    if (tid == 0) {
        *pipe.abort_s = 0;
        pipe_init(pipe, L::ST, 4);
        fence_mbar_init();
    }
    grid_wait();  // the images, and the table and order, of the launches before
    WalkUnit u;
    if (!walk_unit<L::kCols>(p, co, order, chunk_slots, u)) return;
    __syncthreads();
    if (warp == 4) {
        if (lane == 0) forward_copies<typename L::L>(u, pipe, p, &tm_q, &tm_k, &tm_v, images);
    } else {
        walk_forward<typename L::L, 1>(u, pipe, p, nullptr, warp, lane);
    }
    __syncthreads();
    if (tid == 0 && *pipe.abort_s && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
}

cudaError_t launch_scan(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                        cudaStream_t stream) {
    using L = ScanCfg;
    static int configured[64];
    cudaError_t err = set_smem(kda_gdn_scan_kernel, L::ALLOC, configured);
    if (err != cudaSuccess) return err;
    CUtensorMap tm_v;
    if (!make_tensor_map(&tm_v, a.v, a.Hv, a.total_tokens, L::kCols, C, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    const int64_t blocks = static_cast<int64_t>(a.num_seqs) * a.Hv * (D / L::kCols);
    return launch_dependent(kda_gdn_scan_kernel, blocks, L::kThreads, L::ALLOC, stream, tm_q, tm_k, tm_v, a,
                            w.table, w.order, w.images, w.chunks);
}

}  // namespace

cudaError_t launch_gdn_tables(const GdnArgs& a, const GdnWorkspace& w, cudaStream_t stream) {
    cudaError_t err = cudaSuccess;
    if (w.table)
        err = launch_chunk_table(a.cu_seqlens, a.num_seqs, a.total_tokens, w.table, a.device_status, nullptr, nullptr, 0,
                                 stream);
    if (err == cudaSuccess && w.order)
        err = launch_schedule(a.cu_seqlens, a.num_seqs, a.total_tokens, w.order, a.device_status, stream);
    return err;
}

namespace {

// The prefill's scan: tcgen05, a CTA for the 128 columns of a (sequence, value head) pair, or mma.sync, four CTAs
// of 32 columns.  A chunk takes the wide one 3.2 us, prep's larger images apart, the narrow one 1.54, so the narrow one is
// ahead up to two of its CTAs an SM (8192 tokens: 64 pairs 270 us against 279, 96 pairs 274 against 214).
bool scan_wide(const GdnArgs& a) { return static_cast<int64_t>(a.num_seqs) * a.Hv * 2 > device_sm_count(); }

template <bool TILE>
cudaError_t launch_prep(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                        cudaStream_t stream) {
    static int configured[64];
    const cudaError_t err = set_smem(kda_gdn_prep_kernel<TILE>, PrepSmem::ALLOC, configured);
    if (err != cudaSuccess) return err;
    // the value heads of a group (four, two or one of them) share a CTA's Gram matrices where that leaves a CTA
    // for every SM
    const int m = a.Hv / a.Hk;
    int hp = m % 4 == 0 ? 4 : m % 2 == 0 ? 2 : 1;
    while (hp > 1 && w.chunks * (a.Hv / hp) < device_sm_count()) hp /= 2;
    kda_gdn_prep_kernel<TILE><<<static_cast<unsigned>(w.chunks * (a.Hv / hp)), kPrepThreads, PrepSmem::ALLOC, stream>>>(
        tm_q, tm_k, a, w.table, w.images, w.chunks, hp, w.records != nullptr);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdn_prep(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                            cudaStream_t stream) {
    return !w.records && scan_wide(a) ? launch_prep<true>(a, w, tm_q, tm_k, stream) : launch_prep<false>(a, w, tm_q, tm_k, stream);
}

// 32 columns a CTA while that many CTAs find an SM each.  (The gradient's walks of 32 columns, 32 pairs: 447 us for
// 8192 tokens.)
bool gdn_narrow(int32_t num_seqs, int32_t Hv) { return static_cast<int64_t>(num_seqs) * Hv * 4 <= device_sm_count(); }

cudaError_t launch_gdn_scan(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                            cudaStream_t stream) {
    return scan_wide(a) ? launch_gdn_wide(a, w, tm_q, tm_k, stream) : launch_scan(a, w, tm_q, tm_k, stream);
}

size_t gdn_workspace(int32_t num_seqs, int64_t total_tokens, int32_t Hv, bool bwd, uint8_t* base, GdnWorkspace* w) {
    const int64_t chunks = (total_tokens + C - 1) / C + num_seqs;
    const size_t units = static_cast<size_t>(chunks) * Hv;
    const size_t table = round_up(static_cast<size_t>(num_seqs > 0 ? num_seqs : 1) * 4, kAlign);
    const size_t images = table + round_up((static_cast<size_t>(num_seqs) + 2) * 4, kAlign);
    const size_t records = images + units * (bwd ? kImgStrideBwd : std::max(kImgStride, kImgStrideTile));
    if (w) {
        // one sequence needs no table; and where every CTA has an SM of its own, their order does not matter
        w->order = num_seqs > 1 && !gdn_narrow(num_seqs, Hv) ? reinterpret_cast<int32_t*>(base) : nullptr;
        w->table = num_seqs > 1 ? reinterpret_cast<int32_t*>(base + table) : nullptr;
        w->images = base + images;
        w->records = bwd ? base + records : nullptr;
        w->chunks = chunks;
    }
    return records + (bwd ? units * kRecStride : 0);
}

}  // namespace kda
