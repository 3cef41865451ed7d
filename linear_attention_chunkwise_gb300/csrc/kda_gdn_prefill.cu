// kda_gdn_prefill.cu -- the gated delta rule, chunkwise, for bf16 inputs.
//
// With g the inclusive cumulative log decay of a 64-token chunk, S0 the state at its start, and
// G_ij = exp(g_i - g_j) (i >= j):
//   A_ij = b_i G_ij (k_i . k_j)  (i > j),   T = (I + A)^-1 Diag(b),   P_ij = G_ij (q_i . k_j)  (i >= j)
//   U = T (V - Diag(e^g) K S0),   O = Diag(e^g) Q S0 + P U,   S1 = e^gC S0 + K^T Diag(e^(gC - g)) U
// (the chunk form of "Understanding Kimi Delta Attention" (pyshine), "The Chunkwise DPLR Algorithm",
// with its scalar gate).  Unlike the channel-wise gate, the scalar one multiplies the Gram matrices
// afterwards, so every product has the raw bf16 k or q as one operand, and the decays enter as
// exponentials of differences: no lower limit on log_decay, and fp32 accuracy when the other operand
// (state, right-hand side, U) is split into two bf16 terms, x = hi + lo with |x - hi - lo| <= 2^-18 |x|.
//
// pass 0  chunk table (launch_chunk_table)
// pass 1  one CTA per (chunk, value head): Gram matrices, T, P, decays -> an image in the workspace
// pass 2  scan: one warp holds 8 NT columns of the state in mma.sync accumulators (fp32) and walks the
//         chunks of its sequence.  A column of the state needs no other one, so a warp's chain
//         S -> K S -> R -> U -> S stays in its registers: accumulators become the next product's B
//         operand by a pack and an 8 x 8 transpose (movmatrix), and there is no barrier between warps
//         beyond the arrival of the next chunk's tiles.  (tcgen05 would put a TMEM round trip and a
//         write to shared memory for each of the three chained products on the sequential path.)
#include <cuda_bf16.h>

#include "kda_args.h"
#include "kda_internal.h"
#include "kda_ptx.cuh"

namespace kda {
namespace {

constexpr int C = kChunk;    // 64
constexpr int D = kHeadDim;  // 128

// Image of a (chunk, value head): T's two terms and P as 128B-swizzled [64][64] bf16 tiles (16 x 16
// blocks above the diagonal are neither written nor read), then e^g [64], e^(gC - g) [64], e^gC.
constexpr uint32_t kImgTh = 0, kImgTl = 8192, kImgP = 16384, kImgG = 24576;
constexpr uint32_t kImgBytes = kImgG + 528;
constexpr size_t kImgStride = 25344;
static_assert(kImgStride % kAlign == 0 && kImgStride >= kImgBytes && kImgBytes % 16 == 0, "image layout");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// d += a b for one 16 x 8 tile (m16n8k16).  With g = lane / 4, t = lane % 4: a = A(g, 2t..), A(g + 8, 2t..),
// A(g, 2t + 8..), A(g + 8, 2t + 8..); b = B(2t.., g), B(2t + 8.., g); d = D(g, 2t..), D(g + 8, 2t..).
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two bf16 terms of a pair of floats.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// An accumulator tile (16 rows of k, 8 columns) as the B operand of the next product, in two terms.
struct BTerms {
    uint32_t h0, h1, l0, l1;
};
__device__ __forceinline__ BTerms b_terms(const float (&c)[4]) {
    BTerms b;
    uint32_t h0, h1, l0, l1;
    split2(c[0], c[1], h0, l0);
    split2(c[2], c[3], h1, l1);
    b.h0 = transpose8(h0);
    b.h1 = transpose8(h1);
    b.l0 = transpose8(l0);
    b.l1 = transpose8(l1);
    return b;
}

// =============================================================== pass 1 ==
constexpr int kPrepThreads = 256;
constexpr int kLd = 68;  // floats in a row of the fp32 matrices: rows of 4 consecutive threads in other banks

struct PrepSmem {
    static constexpr uint32_t K = 0, Q = 16384;        // 2 x [64][128 B] each, 128B-swizzled
    static constexpr uint32_t T = 0;                   // f32 [64][kLd], over K and Q once the Gram matrices are out
    static constexpr uint32_t X = C * kLd * 4;         // f32 [32][kLd / 2 + ...]: product scratch, beside T
    static constexpr uint32_t A = 32768;               // f32 [64][kLd]
    static constexpr uint32_t G = A + C * kLd * 4;     // f32 [4][64]: g (two terms), beta, e^g
    static constexpr uint32_t BAR = G + 4 * C * 4;
    static constexpr uint32_t TOTAL = BAR + 16;
    static constexpr uint32_t ALLOC = TOTAL + 1024;
};
static_assert(PrepSmem::X + 32 * 36 * 4 <= PrepSmem::A, "the inverse's scratch fits beside T");

// log decays below this (a decay of 0 in fp32, as -inf) are taken as this, so that differences of the
// cumulative sums stay numbers.
constexpr float kDecayFloor = -1e4f;

__global__ void __launch_bounds__(kPrepThreads)
    kda_gdn_prep_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const GdnArgs p, const int32_t* __restrict__ co, uint8_t* images, int64_t chunk_slots) {
    using L = PrepSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int N = p.num_seqs, Hv = p.Hv;
    const int j = blockIdx.x / Hv, h = blockIdx.x - j * Hv;
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
    uint8_t* const img = images + (static_cast<size_t>(j) * Hv + h) * kImgStride;

    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
    float* const g_hi = reinterpret_cast<float*>(sm + L::G);
    float* const g_lo = g_hi + C;
    float* const beta_s = g_lo + C;
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(bar, 32768);
        const int hk = h / (Hv / p.Hk);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
            tma_load_3d(sm + L::K + kh * 8192, &tm_k, bar, 64 * kh, hk, static_cast<int32_t>(t0));
            tma_load_3d(sm + L::Q + kh * 8192, &tm_q, bar, 64 * kh, hk, static_cast<int32_t>(t0));
        }
    }
    if (warp == 1) {  // cumulative log decay, two tokens a lane, in fp64: kept as two fp32 terms
        double x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            float ld = 0.f, b = 0.f;
            if (r < Lc) {
                ld = p.log_decay[(t0 + r) * Hv + h];
                b = p.beta[(t0 + r) * Hv + h];
            }
            x[e] = ld < kDecayFloor ? kDecayFloor : ld;
            beta_s[r] = b;
        }
        double s = x[0] + x[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        const double last = __shfl_sync(0xffffffffu, s, 31);
        float* gv = reinterpret_cast<float*>(img + kImgG);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            const double g = e ? s : s - x[1];
            const float hi = static_cast<float>(g);
            g_hi[r] = hi;
            g_lo[r] = static_cast<float>(g - hi);
            gv[r] = expf(hi) * (1.f + static_cast<float>(g - hi));
            gv[C + r] = expf(static_cast<float>(last - g));
        }
        if (lane == 0) gv[2 * C] = expf(static_cast<float>(last));
    }
    bool ok = true;
    if (tid == 0) ok = mbar_wait_pipe(bar, 0);
    if (!ok && p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
    __syncthreads();

    // Gram rows: warp w < 4 takes rows 16 w of K K^T, warp 4 + w rows 16 (3 - w) of Q K^T (so that the two
    // warps of an SM quarter share its ten 16 x 16 blocks evenly), columns up to the diagonal block.
    const int g = lane >> 2, t = lane & 3;
    const bool is_q = warp >= 4;
    const int mr = is_q ? 7 - warp : warp;
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    {
        const uint32_t a_base = smem_u32(sm + (is_q ? L::Q : L::K)), b_base = smem_u32(sm + L::K);
        const int ar = 16 * mr + (lane & 15), br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
        for (int kt = 0; kt < 8; ++kt) {
            uint32_t a[4];
            ldsm4(a, a_base + (kt >> 2) * 8192 + sw128_chunk(ar, 2 * (kt & 3) + (lane >> 4)));
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                if (np > mr) continue;
                uint32_t b[4];
                ldsm4(b, b_base + (kt >> 2) * 8192 + sw128_chunk(16 * np + br, 2 * (kt & 3) + bc));
                mma16(acc[2 * np], a, b[0], b[1]);
                mma16(acc[2 * np + 1], a, b[2], b[3]);
            }
        }
    }
    __syncthreads();  // K and Q have been read: T may take their place
    float* const As = reinterpret_cast<float*>(sm + L::A);
    float* const Ts = reinterpret_cast<float*>(sm + L::T);
    float* const Xs = reinterpret_cast<float*>(sm + L::X);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        if (n > 2 * mr + 1) continue;
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {  // rows g and g + 8 of the tile
            const int i = 16 * mr + g + 8 * e2;
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int jj = 8 * n + 2 * t + e;
                const float d = (g_hi[i] - g_hi[jj]) + (g_lo[i] - g_lo[jj]);
                const bool in = i < Lc && (is_q ? jj <= i : jj < i);
                v[e] = in ? expf(d) * acc[n][2 * e2 + e] : 0.f;
            }
            if (is_q) {
                *reinterpret_cast<uint32_t*>(img + kImgP + sw128_chunk(i, n) + 4 * t) = pack_bf16(v[0], v[1]);
            } else {
                const float b = beta_s[i];
                *reinterpret_cast<float2*>(As + i * kLd + 8 * n + 2 * t) =
                    make_float2(v[0] * b, v[1] * b);
            }
        }
    }
    __syncthreads();
    // T = (I + A)^-1 by blocks.  Diagonal 16 x 16 blocks: a column for each of 64 threads, by forward
    // substitution (stable for any A).
    if (tid < 64) {
        const int b0 = tid & ~15, c = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 0; k < i; ++k) {
                const float av = As[(b0 + i) * kLd + b0 + k];
                if (k & 1) s1 = fmaf(-av, x[k], s1);
                else s0 = fmaf(-av, x[k], s0);
            }
            x[i] = s0 + s1;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) Ts[(b0 + i) * kLd + b0 + c] = x[i];
    }
    __syncthreads();
    // Blocks (1,0) and (3,2): X = A_lo T_diag, then T = -T_diag X; two outputs a thread.
    {
        const int pr = tid >> 7, e = tid & 127, r = e >> 3, c = 2 * (e & 7), b0 = 32 * pr;
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float av = As[(b0 + 16 + r) * kLd + b0 + k];
            const float2 tv = *reinterpret_cast<const float2*>(Ts + (b0 + k) * kLd + b0 + c);
            x0 = fmaf(av, tv.x, x0);
            x1 = fmaf(av, tv.y, x1);
        }
        *reinterpret_cast<float2*>(Xs + (16 * pr + r) * 36 + c) = make_float2(x0, x1);
        __syncthreads();
        x0 = x1 = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float tv = Ts[(b0 + 16 + r) * kLd + b0 + 16 + k];
            const float2 xv = *reinterpret_cast<const float2*>(Xs + (16 * pr + k) * 36 + c);
            x0 = fmaf(-tv, xv.x, x0);
            x1 = fmaf(-tv, xv.y, x1);
        }
        *reinterpret_cast<float2*>(Ts + (b0 + 16 + r) * kLd + b0 + c) = make_float2(x0, x1);
        *reinterpret_cast<float2*>(Ts + (b0 + r) * kLd + b0 + 16 + c) = make_float2(0.f, 0.f);
    }
    __syncthreads();
    // The lower left 32 x 32 block: X = A_hl T_ll, T_hl = -T_hh X; four columns of a row a thread.
    {
        const int r = tid >> 3, c = 4 * (tid & 7);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float av = As[(32 + r) * kLd + k];
            const float4 tv = *reinterpret_cast<const float4*>(Ts + k * kLd + c);
            x.x = fmaf(av, tv.x, x.x); x.y = fmaf(av, tv.y, x.y);
            x.z = fmaf(av, tv.z, x.z); x.w = fmaf(av, tv.w, x.w);
        }
        __syncthreads();  // the first products' scratch has been read
        *reinterpret_cast<float4*>(Xs + r * 36 + c) = x;
        __syncthreads();
        x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float tv = Ts[(32 + r) * kLd + 32 + k];
            const float4 xv = *reinterpret_cast<const float4*>(Xs + k * 36 + c);
            x.x = fmaf(-tv, xv.x, x.x); x.y = fmaf(-tv, xv.y, x.y);
            x.z = fmaf(-tv, xv.z, x.z); x.w = fmaf(-tv, xv.w, x.w);
        }
        *reinterpret_cast<float4*>(Ts + (32 + r) * kLd + c) = x;
    }
    __syncthreads();
    // T Diag(b) in two bf16 terms, 8 columns of a row at a time
    for (int e = tid; e < C * 8; e += kPrepThreads) {
        const int r = e >> 3, ch = e & 7;
        if ((ch >> 1) > (r >> 4)) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Ts[r * kLd + 8 * ch + i] * beta_s[8 * ch + i];
        uint4 hi, lo;
        split2(v[0], v[1], hi.x, lo.x);
        split2(v[2], v[3], hi.y, lo.y);
        split2(v[4], v[5], hi.z, lo.z);
        split2(v[6], v[7], hi.w, lo.w);
        *reinterpret_cast<uint4*>(img + kImgTh + sw128_chunk(r, ch)) = hi;
        *reinterpret_cast<uint4*>(img + kImgTl + sw128_chunk(r, ch)) = lo;
    }
}

// =============================================================== pass 2 ==
// NW warps of 8 NT state columns each; ST stages of tiles, filled by copies that thread 0 issues.
template <int NT, int NW, int ST>
struct ScanCfg {
    static constexpr int kCols = 8 * NT * NW;
    static constexpr int kThreads = 32 * NW;
    static constexpr uint32_t kVRow = kCols >= 64 ? 128 : kCols * 2;  // bytes of a v row in a block
    static constexpr int kVBlocks = kCols >= 64 ? kCols / 64 : 1;
    static constexpr uint32_t K = 0, Q = 16384, IMG = 32768, V = IMG + 25600;
    static constexpr uint32_t STAGE = V + C * kVRow * kVBlocks;
    static constexpr uint32_t BARS = ST * STAGE;  // full[ST], empty[ST]
    static constexpr uint32_t ABORT = BARS + 16 * ST;
    static constexpr uint32_t ALLOC = ABORT + 16 + 1024;
    static_assert(STAGE % 1024 == 0 && ALLOC <= 232448, "stages");
};

template <int NT, int NW, int ST>
__global__ void __launch_bounds__(ScanCfg<NT, NW, ST>::kThreads, 1)
    kda_gdn_scan_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const GdnArgs p, const int32_t* __restrict__ co,
                        const int32_t* __restrict__ order, const uint8_t* __restrict__ images, int64_t chunk_slots) {
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

    // Chunk c's tiles into stage c mod ST.
    auto issue = [&](int c) {
        const int s = c % ST;
        uint8_t* st = sm + s * L::STAGE;
        const int32_t tok = static_cast<int32_t>(t_begin + static_cast<int64_t>(c) * C);
        const int hk = h / (Hv / p.Hk);
        mbar_arrive_expect_tx(&full[s], 32768 + kImgBytes + C * L::kVRow * L::kVBlocks);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
            tma_load_3d(st + L::K + kh * 8192, &tm_k, &full[s], 64 * kh, hk, tok);
            tma_load_3d(st + L::Q + kh * 8192, &tm_q, &full[s], 64 * kh, hk, tok);
        }
        bulk_g2s(st + L::IMG, images + (static_cast<size_t>(jb + c) * Hv + h) * kImgStride, kImgBytes, &full[s]);
#pragma unroll
        for (int b = 0; b < L::kVBlocks; ++b)
            tma_load_3d(st + L::V + b * C * L::kVRow, &tm_v, &full[s], slice * L::kCols + 64 * b, h, tok);
    };
    int issued = min(ST, nch);  // chunks whose copies thread 0 has issued
    if (tid == 0)
        for (int c = 0; c < issued; ++c) issue(c);
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
        const uint32_t kb = smem_u32(st + L::K), qb = smem_u32(st + L::Q), ib = smem_u32(st + L::IMG);
        const float* gs = reinterpret_cast<const float*>(st + L::IMG + kImgG);
        float ks[4][NT][4], qs[4][NT][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) ks[m][n][e] = qs[m][n][e] = 0.f;
        // K S (state in two terms) and Q S (the output takes one term: it is rounded to bf16 too)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            BTerms b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = b_terms(S[k][n]);
            const uint32_t off = (k >> 2) * 8192;
            uint32_t a[4][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) ldsm4(a[m], kb + off + sw128_chunk(16 * m + lr, 2 * (k & 3) + lc));
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(ks[m][n], a[m], b[n].h0, b[n].h1);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(ks[m][n], a[m], b[n].l0, b[n].l1);
#pragma unroll
            for (int m = 0; m < 4; ++m) ldsm4(a[m], qb + off + sw128_chunk(16 * m + lr, 2 * (k & 3) + lc));
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(qs[m][n], a[m], b[n].h0, b[n].h1);
        }
        // The previous chunk's stage is refilled once every warp is done with it.
        if (warp == 0 && c > 0 && issued < nch) {
            bool done = true;
            if (lane == 0) {
                done = mbar_wait_pipe(&empty[(c - 1) % ST], ((c - 1) / ST) & 1);
                if (done) issue(issued);
                else *abort_s = 1;
            }
            if (__all_sync(0xffffffffu, done)) ++issued;
        }
        // R = V - e^g K S, then U = T R with both in two terms
        float u[4][NT][4];
        float eg[4][2];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) u[m][n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            BTerms b[NT];
#pragma unroll
            for (int e = 0; e < 2; ++e) eg[k][e] = gs[16 * k + g + 8 * e];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float r[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * k + g + 8 * e, col = wc + 8 * n;  // the 16-byte piece of 8 columns
                    const uint32_t piece = static_cast<uint32_t>(col >> 3);
                    uint32_t off;
                    if constexpr (L::kVRow == 128)
                        off = (piece >> 3) * (C * 128) + sw128_chunk(row, piece & 7);
                    else  // 64-byte rows: the swizzle takes bits 1 and 2 of the row
                        off = row * 64 + (((piece ^ (row >> 1)) & 3) << 4);
                    const uint32_t vv = *reinterpret_cast<const uint32_t*>(st + L::V + off + 4 * t);
                    r[2 * e] = fmaf(-eg[k][e], ks[k][n][2 * e], __uint_as_float(vv << 16));
                    r[2 * e + 1] = fmaf(-eg[k][e], ks[k][n][2 * e + 1], __uint_as_float(vv & 0xffff0000u));
                    if (row >= Lc) r[2 * e] = r[2 * e + 1] = 0.f;
                }
                b[n] = b_terms(r);
            }
            uint32_t ah[4][4];
#pragma unroll
            for (int m = k; m < 4; ++m) ldsm4(ah[m], ib + kImgTh + sw128_chunk(16 * m + lr, 2 * k + lc));
#pragma unroll
            for (int m = k; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], b[n].h0, b[n].h1);
#pragma unroll
            for (int m = k; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], b[n].l0, b[n].l1);
#pragma unroll
            for (int m = k; m < 4; ++m) ldsm4(ah[m], ib + kImgTl + sw128_chunk(16 * m + lr, 2 * k + lc));
#pragma unroll
            for (int m = k; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(u[m][n], ah[m], b[n].h0, b[n].h1);
        }
        // S <- e^gC S + K^T (e^(gC - g) U), U in two terms
        const float gc = gs[2 * C];
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][n][e] *= gc;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float e0 = gs[C + 16 * k + g], e1 = gs[C + 16 * k + g + 8];
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
                ldsm4(a, ib + kImgP + sw128_chunk(16 * m + lr, 2 * k + lc));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16(qs[m][n], a, b0[n], b1[n]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);  // the warp has read all it takes of this stage
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
    __syncthreads();
    if (tid == 0 && *abort_s) {
        for (int c = max(0, issued - ST); c < issued; ++c)  // no copy is left in flight
            (void)mbar_wait(&full[c % ST], (c / ST) & 1, kDrainLimit);
        if (p.device_status) atomicOr(p.device_status, KDA_DEV_TIMEOUT);
    }
}

template <typename K>
cudaError_t set_smem(K kernel, uint32_t bytes, int* configured) {  // on first use per device
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || (dev >= 0 && dev < 64 && configured[dev])) return err;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (err == cudaSuccess && dev >= 0 && dev < 64) configured[dev] = 1;
    return err;
}

template <int NT, int NW, int ST>
cudaError_t launch_scan(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const GdnArgs& a, const int32_t* table,
                        const int32_t* order, const uint8_t* images, int64_t slots, cudaStream_t stream) {
    using L = ScanCfg<NT, NW, ST>;
    static int configured[64];
    cudaError_t err = set_smem(kda_gdn_scan_kernel<NT, NW, ST>, L::ALLOC, configured);
    if (err != cudaSuccess) return err;
    CUtensorMap tm_v;
    if (!make_tensor_map(&tm_v, a.v, a.Hv, a.total_tokens, L::kVRow / 2, C,
                         L::kVRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * a.Hv * (D / L::kCols));
    kda_gdn_scan_kernel<NT, NW, ST><<<blocks, L::kThreads, L::ALLOC, stream>>>(tm_q, tm_k, tm_v, a, table, order, images,
                                                                               slots);
    return cudaGetLastError();
}

}  // namespace

GdnLayout gdn_layout(int32_t num_seqs, int64_t total_tokens, int32_t Hv) {
    GdnLayout l;
    l.chunks = (total_tokens + C - 1) / C + num_seqs;
    l.table = round_up(static_cast<size_t>(num_seqs > 0 ? num_seqs : 1) * 4, kAlign);
    l.images = l.table + round_up((static_cast<size_t>(num_seqs) + 2) * 4, kAlign);
    l.total = l.images + static_cast<size_t>(l.chunks) * Hv * kImgStride;
    return l;
}

cudaError_t launch_gdn_chunked(const GdnArgs& a, const GdnLayout& lay, uint8_t* workspace, cudaStream_t stream) {
    if (a.num_seqs == 0) return cudaSuccess;
    int32_t* order = reinterpret_cast<int32_t*>(workspace + lay.order);
    int32_t* table = reinterpret_cast<int32_t*>(workspace + lay.table);
    uint8_t* images = workspace + lay.images;
    CUtensorMap tm_q, tm_k;
    if (!make_tensor_map(&tm_q, a.q, a.Hk, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&tm_k, a.k, a.Hk, a.total_tokens, 64, C, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    cudaError_t err = launch_chunk_table(a.cu_seqlens, a.num_seqs, a.total_tokens, table, a.device_status, nullptr, nullptr,
                                         0, stream);
    if (err == cudaSuccess && a.num_seqs > 1)
        err = launch_schedule(a.cu_seqlens, a.num_seqs, a.total_tokens, order, a.device_status, stream);
    static int configured[64];
    if (err == cudaSuccess) err = set_smem(kda_gdn_prep_kernel, PrepSmem::ALLOC, configured);
    if (err != cudaSuccess) return err;
    const unsigned units = static_cast<unsigned>(lay.chunks * a.Hv);
    kda_gdn_prep_kernel<<<units, kPrepThreads, PrepSmem::ALLOC, stream>>>(tm_q, tm_k, a, table, images, lay.chunks);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int32_t* ord = a.num_seqs > 1 ? order : nullptr;
    if (static_cast<int64_t>(a.num_seqs) * a.Hv * 4 <= device_sm_count())
        return launch_scan<1, 4, 3>(tm_q, tm_k, a, table, ord, images, lay.chunks, stream);
    return launch_scan<2, 8, 2>(tm_q, tm_k, a, table, ord, images, lay.chunks, stream);
}

}  // namespace kda
