// kda_gdn_prefill.cu -- the gated delta rule, chunkwise, for bf16 inputs.
//
// With g the inclusive cumulative log decay of a 64-token chunk, S0 the state at its start, and
// G_ij = exp(g_i - g_j) (i >= j):
//   A_ij = b_i G_ij (k_i . k_j)  (i > j),   T = (I + A)^-1,   P_ij = G_ij (q_i . k_j)  (i >= j)
//   U = T Diag(b) (V - Diag(e^g) K S0),   O = Diag(e^g) Q S0 + P U,   S1 = e^gC S0 + K^T Diag(e^(gC - g)) U
// (the chunk form of "Understanding Kimi Delta Attention" (pyshine), "The Chunkwise DPLR Algorithm",
// with its scalar gate).  Unlike the channel-wise gate, the scalar one multiplies the Gram matrices
// afterwards, so every product has the raw bf16 k or q as one operand, and the decays enter as
// exponentials of differences: no lower limit on log_decay, and fp32 accuracy when the other operand
// (state, right-hand side, U) is split into two bf16 terms, x = hi + lo with |x - hi - lo| <= 2^-17 |x|.
//
// pass 0  chunk table (launch_chunk_table)
// pass 1  one CTA per (chunk, value head): Gram matrices, T, P, decays -> an image in the workspace
// pass 2  scan: one warp holds 8 NT columns of the state in mma.sync accumulators (fp32) and walks the
//         chunks of its sequence.  A column of the state needs no other one, so a warp's chain
//         S -> K S -> R -> U -> S stays in its registers: accumulators become the next product's B
//         operand by a pack and an 8 x 8 transpose (movmatrix), and there is no barrier between warps
//         beyond the arrival of the next chunk's tiles.  (tcgen05 would put a TMEM round trip and a
//         write to shared memory for each of the three chained products on the sequential path.)
#include "kda_gdn_common.cuh"

namespace kda {
namespace {

using namespace gdn;

// =============================================================== pass 1 ==
// One CTA of four warps for a (chunk, q/k head) and `hp` of its value heads, which share the Gram
// matrices: warp r holds rows 16 r of K K^T and Q K^T in registers.  Per value head: the decays and
// b make A and P of them; the 16 x 16 diagonal blocks of I + A are inverted by forward substitution
// in fp32 (stable for any A; a column for each of 64 threads); then warp j forms block column j of the
// inverse, T_ij = -D_i sum_{j <= k < i} A_ik T_kj, by mma.sync on two-term operands, its blocks staying in
// its registers.  (The block products in fp32 on the CUDA cores and one value head a CTA, 256 threads:
// 109 us for 8192 tokens x 32 heads, 16.1 K warp instructions a (chunk, head).)
constexpr int kPrepThreads = 128;

struct PrepSmem {
    static constexpr uint32_t K = 0, Q = 16384;  // 2 x [64][128 B] each, 128B-swizzled
    static constexpr uint32_t AH = 0;            // two terms of A's blocks, the diagonal ones inverted (over K and
    static constexpr uint32_t AL = kTriBytes;    // Q once the Gram matrices are out)
    static constexpr uint32_t DG = 16384;        // f32 [4][16][17]: diagonal blocks of A
    static constexpr uint32_t G = 32768;         // f32 [3][64]: g (two terms, base 2), beta
    static constexpr uint32_t BAR = G + 3 * C * 4;
    static constexpr uint32_t TOTAL = BAR + 16;
    static constexpr uint32_t ALLOC = TOTAL + 1024;
};

// log decays below this (a decay of 0 in fp32, as -inf) are taken as this, so that differences of the
// cumulative sums stay numbers.
constexpr float kDecayFloor = -1e4f;
// In the gradient's images a smaller b, 0 too, is taken as this: U / b is then still what the rows of U
// hold before b multiplies them, and b's own part in every sum is below fp32's rounding.
constexpr float kBetaFloor = 8.271806e-25f;  // 2^-80

__global__ void __launch_bounds__(kPrepThreads, 4)
    kda_gdn_prep_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const GdnArgs p, const int32_t* __restrict__ co, uint8_t* images, int64_t chunk_slots,
                        int32_t hp, bool bwd) {
    using L = PrepSmem;
    const size_t stride = bwd ? kImgStrideBwd : kImgStride;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.num_seqs, Hv = p.Hv, groups = Hv / hp;
    const int j = blockIdx.x / groups, h0 = (blockIdx.x - j * groups) * hp;
    if (co[N + 1] == 0 || j >= co[N]) return;  // malformed cu_seqlens, or no such chunk
    int seq;
    {  // the largest n with co[n] <= j
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (co[mid] <= j) lo = mid;
            else hi = mid - 1;
        }
        seq = lo;
    }
    const int64_t t0 = static_cast<int64_t>(p.cu_seqlens[seq]) + static_cast<int64_t>(j - co[seq]) * C;
    const int64_t rem = p.cu_seqlens[seq + 1] - t0;
    const int Lc = static_cast<int>(rem < C ? rem : C);
    if (!KDA_BOUNDS(seq >= 0 && seq < N && j < chunk_slots && t0 >= 0 && Lc >= 1 && t0 + Lc <= p.total_tokens,
                    p.device_status))
        return;

    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    float* const g_hi = reinterpret_cast<float*>(sm + L::G);
    float* const g_lo = g_hi + C;
    float* const beta_s = g_lo + C;
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
    // Value head h's cumulative log decay (base 2, two tokens a lane, in fp64; kept as two fp32 terms), beta,
    // and the image's decays.
    auto decays = [&](int h) {
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
        float* gv = reinterpret_cast<float*>(images + (static_cast<size_t>(j) * Hv + h) * stride + kImgG);
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
    };
    if (warp == 1) decays(h0);
    bool ok = true;
    if (tid == 0) ok = mbar_wait_pipe(bar, 0);
    if (!ok && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
    __syncthreads();

    // Gram rows up to the diagonal block.  The row block of a warp turns with the CTA, so that no quarter of
    // the SM has the long rows of every CTA.
    const int g = lane >> 2, t = lane & 3;
    const int mr = (warp + blockIdx.x) & 3;
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
    {
        const uint32_t kb = smem_u32(sm + L::K), qb = smem_u32(sm + L::Q);
        const int ar = 16 * mr + (lane & 15), br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt) {
            uint32_t ak[4], aq[4];
            const uint32_t off = (kt >> 2) * 8192;
            ldsm4(ak, kb + off + sw128_chunk(ar, 2 * (kt & 3) + (lane >> 4)));
            ldsm4(aq, qb + off + sw128_chunk(ar, 2 * (kt & 3) + (lane >> 4)));
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                if (np > mr) break;
                uint32_t b[4];
                ldsm4(b, kb + off + sw128_chunk(16 * np + br, 2 * (kt & 3) + bc));
                mma16(kk[2 * np], ak, b[0], b[1]);
                mma16(kk[2 * np + 1], ak, b[2], b[3]);
                mma16(qk[2 * np], aq, b[0], b[1]);
                mma16(qk[2 * np + 1], aq, b[2], b[3]);
            }
        }
    }
    const uint32_t ah_base = smem_u32(sm + L::AH) + 16 * lane, al_base = smem_u32(sm + L::AL) + 16 * lane;
    float* const dg = reinterpret_cast<float*>(sm + L::DG);
    for (int hh = 0; hh < hp; ++hh) {
        const int h = h0 + hh;
        uint8_t* const img = images + (static_cast<size_t>(j) * Hv + h) * stride;
        __syncthreads();  // K and Q, or the previous head's A and decays, have been read
        if (hh > 0) {
            if (warp == 1) decays(h);
            __syncthreads();
        }
        // A (two terms; its diagonal blocks in fp32) and P
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (n > 2 * mr + 1) break;
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {  // rows g and g + 8 of the tile
                const int i = 16 * mr + g + 8 * e2;
                const float2 ch = *reinterpret_cast<const float2*>(g_hi + 8 * n + 2 * t);
                const float2 cl = *reinterpret_cast<const float2*>(g_lo + 8 * n + 2 * t);
                const float gi = g_hi[i], gl = g_lo[i], b = beta_s[i];
                const int jj = 8 * n + 2 * t;
                const bool row = i < Lc;
                const float d0 = exp2_sfu((gi - ch.x) + (gl - cl.x)), d1 = exp2_sfu((gi - ch.y) + (gl - cl.y));
                const uint32_t pair = blk_pair(g, e2, n & 1, t);
                const float p0 = row && jj <= i ? d0 * qk[n][2 * e2] : 0.f;
                const float p1 = row && jj + 1 <= i ? d1 * qk[n][2 * e2 + 1] : 0.f;
                uint32_t ph, pl;
                split2(p0, p1, ph, pl);
                uint8_t* const pp = img + tri_blk(mr, n >> 1) + pair;
                *reinterpret_cast<uint32_t*>(pp + kImgP) = ph;
                if (bwd) {
                    *reinterpret_cast<uint32_t*>(pp + kImgPl) = pl;
                    *reinterpret_cast<uint32_t*>(pp + kImgPl2) = third2(p0, p1, ph, pl);
                }
                const float a0 = row && jj < i ? b * d0 * kk[n][2 * e2] : 0.f;
                const float a1 = row && jj + 1 < i ? b * d1 * kk[n][2 * e2 + 1] : 0.f;
                if ((n >> 1) == mr) {
                    float* d = dg + mr * 272 + (g + 8 * e2) * 17 + 8 * (n & 1) + 2 * t;
                    d[0] = a0;
                    d[1] = a1;
                } else {
                    uint32_t hi, lo;
                    split2(a0, a1, hi, lo);
                    uint8_t* const ap = sm + tri_blk(mr, n >> 1) + pair;
                    *reinterpret_cast<uint32_t*>(ap + L::AH) = hi;
                    *reinterpret_cast<uint32_t*>(ap + L::AL) = lo;
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
            const int w = mr;
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
                        uint8_t* const tp = img + tri_blk(i, w) + blk_pair(g, e2, n, t);
                        *reinterpret_cast<uint32_t*>(tp + kImgTh) = hi;
                        *reinterpret_cast<uint32_t*>(tp + kImgTl) = lo;
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
// NW warps of 8 NT state columns each and one that issues the copies; ST stages of tiles.
template <int NT, int NW, int ST>
struct ScanCfg {
    static constexpr int kCols = 8 * NT * NW;
    static constexpr int kThreads = 32 * (NW + 1);
    static constexpr uint32_t kVRow = kCols >= 64 ? 128 : kCols * 2;  // bytes of a v row in a block
    static constexpr int kVBlocks = kCols >= 64 ? kCols / 64 : 1;
    static constexpr uint32_t K = 0, Q = 16384, IMG = 32768, V = IMG + 16384;
    static constexpr uint32_t STAGE = V + C * kVRow * kVBlocks;
    static constexpr uint32_t BARS = ST * STAGE;  // full[ST], empty[ST]
    static constexpr uint32_t ABORT = BARS + 16 * ST;
    static constexpr uint32_t ALLOC = ABORT + 16 + 1024;
    static_assert(STAGE % 1024 == 0 && ALLOC <= 232448 && kImgScanBytes <= 16384, "stages");
};

// REC: the gradient's walk, which leaves every chunk's start state and U in two bf16 terms and no outputs.
template <int NT, int NW, int ST, bool REC>
__global__ void __launch_bounds__(ScanCfg<NT, NW, ST>::kThreads, 1)
    kda_gdn_scan_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const GdnArgs p, const int32_t* __restrict__ co,
                        const int32_t* __restrict__ order, const uint8_t* __restrict__ images, int64_t chunk_slots,
                        uint8_t* records) {
    using L = ScanCfg<NT, NW, ST>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.num_seqs, Hv = p.Hv;
    constexpr int NSL = D / L::kCols;
    const int slice = blockIdx.x % NSL;
    const int h = (blockIdx.x / NSL) % Hv;
    const int pos = blockIdx.x / (NSL * Hv);
    if (co[N + 1] == 0) return;
    const int seq = order ? order[pos] : pos;
    const int nch = co[seq + 1] - co[seq], jb = co[seq];
    const int64_t t_begin = p.cu_seqlens[seq], t_end = p.cu_seqlens[seq + 1];
    if (!KDA_BOUNDS(seq >= 0 && seq < N && h < Hv && t_begin >= 0 && t_end <= p.total_tokens && jb >= 0 &&
                        static_cast<int64_t>(jb) + nch <= chunk_slots &&
                        static_cast<int64_t>(nch) * C >= t_end - t_begin,
                    p.device_status))
        return;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint64_t* empty = full + ST;
    volatile int* abort_s = reinterpret_cast<volatile int*>(sm + L::ABORT);
    if (tid == 0) {
        *abort_s = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], NW);
        }
        fence_mbar_init();
    }
    __syncthreads();

    // A warp of its own issues the copies (a thread is held for about 0.1 us by each): chunk c's tiles go into
    // stage c mod ST once every reader is done with chunk c - ST.
    if (warp == NW) {
        if (lane == 0) {
            const int hk = h / (Hv / p.Hk);
            int c = 0;
            for (; c < nch && !*abort_s; ++c) {
                const int s = c % ST;
                if (c >= ST && !mbar_wait_pipe(&empty[s], ((c / ST) - 1) & 1)) {
                    *abort_s = 1;
                    break;
                }
                uint8_t* st = sm + s * L::STAGE;
                const int32_t tok = static_cast<int32_t>(t_begin + static_cast<int64_t>(c) * C);
                mbar_arrive_expect_tx(&full[s], (REC ? 16384 : 32768) + kImgScanBytes + C * L::kVRow * L::kVBlocks);
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) tma_load_3d(st + L::K + kh * 8192, &tm_k, &full[s], 64 * kh, hk, tok);
#pragma unroll
                for (int b = 0; b < L::kVBlocks; ++b)
                    tma_load_3d(st + L::V + b * C * L::kVRow, &tm_v, &full[s], slice * L::kCols + 64 * b, h, tok);
                bulk_g2s(st + L::IMG, images + (static_cast<size_t>(jb + c) * Hv + h) * (REC ? kImgStrideBwd : kImgStride),
                         kImgScanBytes, &full[s]);
#pragma unroll
                for (int kh = 0; kh < (REC ? 0 : 2); ++kh)
                    tma_load_3d(st + L::Q + kh * 8192, &tm_q, &full[s], 64 * kh, hk, tok);
            }
            for (int d = max(0, c - ST); d < c; ++d)  // no copy is left in flight
                (void)mbar_wait(&full[d % ST], (d / ST) & 1, kDrainLimit);
        }
    } else {
        const int g = lane >> 2, t = lane & 3;
        const int wc = 8 * NT * warp;                  // the warp's first column in the CTA's
        const int j0 = slice * L::kCols + wc + 2 * t;  // this thread's first state column
        const size_t sbase = (static_cast<size_t>(seq) * Hv + h) * D * D;
        float S[8][NT][4];  // rows 16 m + g (+ 8), columns j0 + 8 n (+ 1)
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const size_t off = sbase + static_cast<size_t>(16 * m + g + 8 * e) * D + j0 + 8 * n;
                    const float2 x = p.S0 ? *reinterpret_cast<const float2*>(p.S0 + off) : make_float2(0.f, 0.f);
                    S[m][n][2 * e] = x.x;
                    S[m][n][2 * e + 1] = x.y;
                }
        // ldmatrix addresses within a tile: rows of tokens (row-major operand) and their transposes
        const int lr = lane & 15, lc = lane >> 4;
        const int tr = (lane & 7) + ((lane >> 4) << 3), tc = (lane >> 3) & 1;
        for (int c = 0; c < nch; ++c) {
            const int s = c % ST;
            uint8_t* st = sm + s * L::STAGE;
            const bool landed = !*abort_s && mbar_wait_pipe(&full[s], (c / ST) & 1);
            if (!__all_sync(0xffffffffu, landed)) {  // a bounded wait expired, here or elsewhere
                *abort_s = 1;
                break;
            }
            const int64_t t0 = t_begin + static_cast<int64_t>(c) * C;
            const int Lc = static_cast<int>(t_end - t0 < C ? t_end - t0 : C);
            if (Lc < C) {  // k rows behind the sequence's end meet zeros of U: they must be numbers
                for (int e = lane; e < (C - Lc) * 16; e += 32)
                    *reinterpret_cast<uint4*>(st + L::K + (e & 1) * 8192 + sw128_chunk(Lc + (e >> 4), (e >> 1) & 7)) =
                        make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            }
            const uint32_t kb = smem_u32(st + L::K), qb = smem_u32(st + L::Q), ib = smem_u32(st + L::IMG) + 16 * lane;
            const float* gs = reinterpret_cast<const float*>(st + L::IMG + kImgG);
            uint8_t* const rec = REC ? records + (static_cast<size_t>(jb + c) * Hv + h) * kRecStride : nullptr;
            const int rcol = slice * L::kCols + wc + 2 * t;
            float ks[4][NT][4], qs[4][NT][4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) ks[m][n][e] = qs[m][n][e] = 0.f;
            // K S, the state in two terms; the first one is kept for Q S (the output is rounded to bf16 too)
            uint32_t sh[8][NT][2];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                BTerms b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (REC) {
                        put_record(S[k][n], rec + kRecS, 16384, 32768, 16 * k + g, rcol + 8 * n);
                        b[n] = b_terms(S[k][n]);
                    } else {
                        b[n] = b_terms(S[k][n]);
                    }
                    sh[k][n][0] = b[n].h0;
                    sh[k][n][1] = b[n].h1;
                }
                uint32_t a[4][4];
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    ldsm4(a[m], kb + (k >> 2) * 8192 + sw128_chunk(16 * m + lr, 2 * (k & 3) + lc));
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(ks[m][n], a[m], b[n].h0, b[n].h1);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(ks[m][n], a[m], b[n].l0, b[n].l1);
            }
            // R = b (V - e^g K S); Q S runs beside it, a quarter for each 16 rows of R
            float eg[4][2], be[2];
            BTerms r[4][NT];
            uint32_t r2[REC ? 4 : 1][NT][2];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    eg[k][e] = gs[kVecEg + 16 * k + g + 8 * e];
                    be[e] = gs[kVecB + 16 * k + g + 8 * e];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 16 * k + g + 8 * e;
                        const uint32_t piece = static_cast<uint32_t>((wc + 8 * n) >> 3);  // 16 bytes: 8 columns
                        uint32_t off;
                        if constexpr (L::kVRow == 128) off = (piece >> 3) * (C * 128) + sw128_chunk(row, piece & 7);
                        else off = row * 64 + (((piece ^ (row >> 1)) & 3) << 4);  // 64-byte rows
                        const uint32_t vv = *reinterpret_cast<const uint32_t*>(st + L::V + off + 4 * t);
                        x[2 * e] = be[e] * fmaf(-eg[k][e], ks[k][n][2 * e], __uint_as_float(vv << 16));
                        x[2 * e + 1] = be[e] * fmaf(-eg[k][e], ks[k][n][2 * e + 1], __uint_as_float(vv & 0xffff0000u));
                        if (row >= Lc) x[2 * e] = x[2 * e + 1] = 0.f;
                    }
                    if constexpr (REC) {
                        const BTerms3 x3 = b_terms3(x);
                        r[k][n] = x3.b;
                        r2[k][n][0] = x3.m0;
                        r2[k][n][1] = x3.m1;
                    } else {
                        r[k][n] = b_terms(x);
                    }
                }
#pragma unroll
                for (int kq = 2 * k; kq < (REC ? 0 : 2 * k + 2); ++kq) {
                    uint32_t a[4][4];
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        ldsm4(a[m], qb + (kq >> 2) * 8192 + sw128_chunk(16 * m + lr, 2 * (kq & 3) + lc));
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16(qs[m][n], a[m], sh[kq][n][0], sh[kq][n][1]);
                }
            }
            // U = T R, both in two terms
            float u[4][NT][4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[m][n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t ah[4][4], al[4][4];
#pragma unroll
                for (int m = k; m < 4; ++m) {
                    ldsm4(ah[m], ib + kImgTh + tri_blk(m, k));
                    ldsm4(al[m], ib + kImgTl + tri_blk(m, k));
                }
#pragma unroll
                for (int m = k; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], r[k][n].h0, r[k][n].h1);
                if constexpr (REC) {  // the gradient of b takes U . W: the right-hand side in three terms
#pragma unroll
                    for (int m = k; m < 4; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], r2[k][n][0], r2[k][n][1]);
                }
#pragma unroll
                for (int m = k; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], r[k][n].l0, r[k][n].l1);
#pragma unroll
                for (int m = k; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16(u[m][n], al[m], r[k][n].h0, r[k][n].h1);
            }
            // S <- e^gC S + K^T (e^(gC - g) U), U in two terms
            const float gc = gs[kVecEc];
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[m][n][e] *= gc;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float e0 = gs[kVecEo + 16 * k + g], e1 = gs[kVecEo + 16 * k + g + 8];
                BTerms b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float x[4] = {u[k][n][0] * e0, u[k][n][1] * e0, u[k][n][2] * e1, u[k][n][3] * e1};
                    b[n] = b_terms(x);
                }
#pragma unroll
                for (int mh = 0; mh < 2; ++mh) {
                    uint32_t a[4][4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) ldsm4t(a[m], kb + mh * 8192 + sw128_chunk(16 * k + tr, 2 * m + tc));
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16(S[4 * mh + m][n], a[m], b[n].h0, b[n].h1);
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16(S[4 * mh + m][n], a[m], b[n].l0, b[n].l1);
                }
            }
            if constexpr (REC) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n) put_record(u[k][n], rec + kRecU, 8192, 16384, 16 * k + g, rcol + 8 * n);
            } else {
                // O = e^g Q S + P U
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) qs[m][n][e] *= eg[m][e >> 1];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t b0[NT], b1[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        b0[n] = transpose8(pack_bf16(u[k][n][0], u[k][n][1]));
                        b1[n] = transpose8(pack_bf16(u[k][n][2], u[k][n][3]));
                    }
#pragma unroll
                    for (int m = k; m < 4; ++m) {
                        uint32_t a[4];
                        ldsm4(a, ib + kImgP + tri_blk(m, k));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16(qs[m][n], a, b0[n], b1[n]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);  // the warp has read all it takes of this stage
            if constexpr (!REC) {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + (t0 * Hv + h) * D + j0;
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 16 * m + g + 8 * e;
                        if (row < Lc) {
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                *reinterpret_cast<uint32_t*>(o + static_cast<int64_t>(row) * Hv * D + 8 * n) =
                                    pack_bf16(qs[m][n][2 * e], qs[m][n][2 * e + 1]);
                        }
                    }
            }
        }
        if (p.S_final && !*abort_s) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2*>(p.S_final + sbase + static_cast<size_t>(16 * m + g + 8 * e) * D + j0 +
                                                   8 * n) = make_float2(S[m][n][2 * e], S[m][n][2 * e + 1]);
        }
    }
    __syncthreads();
    if (tid == 0 && *abort_s && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
}

template <int NT, int NW, int ST, bool REC>
cudaError_t launch_scan(const GdnArgs& a, const GdnWorkspace& w, cudaStream_t stream) {
    using L = ScanCfg<NT, NW, ST>;
    static int configured[64];
    cudaError_t err = set_smem(kda_gdn_scan_kernel<NT, NW, ST, REC>, L::ALLOC, configured);
    if (err != cudaSuccess) return err;
    CUtensorMap tm_q, tm_k, tm_v;
    if (!make_tensor_map(&tm_q, a.q, a.Hk, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&tm_k, a.k, a.Hk, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&tm_v, a.v, a.Hv, a.total_tokens, L::kVRow / 2, C,
                         L::kVRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * a.Hv * (D / L::kCols));
    kda_gdn_scan_kernel<NT, NW, ST, REC><<<blocks, L::kThreads, L::ALLOC, stream>>>(
        tm_q, tm_k, tm_v, a, w.table, w.order, w.images, w.chunks, w.records);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdn_tables(const GdnArgs& a, const GdnWorkspace& w, cudaStream_t stream) {
    cudaError_t err = launch_chunk_table(a.cu_seqlens, a.num_seqs, a.total_tokens, w.table, a.device_status, nullptr, nullptr,
                                         0, stream);
    if (err == cudaSuccess && w.order)
        err = launch_schedule(a.cu_seqlens, a.num_seqs, a.total_tokens, w.order, a.device_status, stream);
    return err;
}

cudaError_t launch_gdn_prep(const GdnArgs& a, const GdnWorkspace& w, cudaStream_t stream) {
    CUtensorMap tm_q, tm_k;
    if (!make_tensor_map(&tm_q, a.q, a.Hk, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&tm_k, a.k, a.Hk, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    static int configured[64];
    const cudaError_t err = set_smem(kda_gdn_prep_kernel, PrepSmem::ALLOC, configured);
    if (err != cudaSuccess) return err;
    // the value heads of a group share a CTA's Gram matrices where that leaves a CTA for every SM
    const int m = a.Hv / a.Hk;
    const int hp = w.chunks * a.Hk >= device_sm_count() ? m : 1;
    kda_gdn_prep_kernel<<<static_cast<unsigned>(w.chunks * (a.Hv / hp)), kPrepThreads, PrepSmem::ALLOC, stream>>>(
        tm_q, tm_k, a, w.table, w.images, w.chunks, hp, w.records != nullptr);
    return cudaGetLastError();
}

// 32 columns a CTA while that many CTAs find an SM each (the shortest chain: 1.54 us a chunk), else 64
// (packed 24.6 k tokens x 32 heads: 663 us against 701 us).
cudaError_t launch_gdn_scan(const GdnArgs& a, const GdnWorkspace& w, cudaStream_t stream) {
    if (static_cast<int64_t>(a.num_seqs) * a.Hv * 4 <= device_sm_count())
        return w.records ? launch_scan<1, 4, 3, true>(a, w, stream) : launch_scan<1, 4, 3, false>(a, w, stream);
    return w.records ? launch_scan<2, 4, 3, true>(a, w, stream) : launch_scan<2, 4, 3, false>(a, w, stream);
}

size_t gdn_workspace(int32_t num_seqs, int64_t total_tokens, int32_t Hv, bool bwd, uint8_t* base, GdnWorkspace* w) {
    const int64_t chunks = (total_tokens + C - 1) / C + num_seqs;
    const size_t units = static_cast<size_t>(chunks) * Hv;
    const size_t table = round_up(static_cast<size_t>(num_seqs > 0 ? num_seqs : 1) * 4, kAlign);
    const size_t images = table + round_up((static_cast<size_t>(num_seqs) + 2) * 4, kAlign);
    const size_t records = images + units * (bwd ? kImgStrideBwd : kImgStride);
    if (w) {
        w->order = num_seqs > 1 ? reinterpret_cast<int32_t*>(base) : nullptr;
        w->table = reinterpret_cast<int32_t*>(base + table);
        w->images = base + images;
        w->records = bwd ? base + records : nullptr;
        w->chunks = chunks;
    }
    return records + (bwd ? units * kRecStride : 0);
}

}  // namespace kda
