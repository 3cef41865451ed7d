// kda_gdn_walk.cuh -- the walk of the gated delta rule over the chunks of a sequence, for the prefill's scan and
// the gradient's two walks.
//
// A warp holds 8 NT columns of the state (or of its adjoint) in mma.sync accumulators (fp32) and walks the
// chunks of its sequence.  A column needs no other one, so a warp's chain S -> K S -> R -> U -> S stays in its
// registers: accumulators become the next product's B operand by a pack and an 8 x 8 transpose
// (movmatrix), and there is no barrier between warps beyond the arrival of the next chunk's tiles, which a
// warp of its own copies (a thread is held for about 0.1 us by each copy it issues: by one of the four
// walking warps the scan of 8192 tokens x 32 heads takes 265 us, not 198).  tcgen05 would put a TMEM round trip
// and a write to shared memory for each of the chained products on the sequential path, and at the 32
// columns a CTA has here its products, held by the reads of A, take as long.
#pragma once

#include "kda_gdn_common.cuh"

namespace kda {
namespace gdn {

// What a CTA walks over: (sequence, value head, columns from col0).
struct WalkUnit {
    int64_t t_begin, t_end;
    int seq, h, hk, col0, nch, jb;
};

// The chunk table: written by launch_chunk_table, or (NULL, one sequence) what follows from cu_seqlens.
__device__ __forceinline__ bool table_ok(const GdnArgs& p, const int32_t* co) {
    return co ? co[p.num_seqs + 1] != 0 : p.cu_seqlens[0] == 0 && p.cu_seqlens[1] == p.total_tokens;
}
__device__ __forceinline__ int table_at(const GdnArgs& p, const int32_t* co, int n) {
    return co ? co[n] : n ? static_cast<int>((p.total_tokens + C - 1) / C) : 0;
}

// blockIdx.x's unit; false when cu_seqlens is malformed (nothing is to be written).
template <int COLS>
__device__ __forceinline__ bool walk_unit(const GdnArgs& p, const int32_t* co, const int32_t* order, int64_t chunk_slots,
                                          WalkUnit& u) {
    constexpr int NSL = D / COLS;
    if (!table_ok(p, co)) return false;
    const int pos = blockIdx.x / (NSL * p.Hv);
    u.col0 = (blockIdx.x % NSL) * COLS;
    u.h = (blockIdx.x / NSL) % p.Hv;
    u.hk = u.h / (p.Hv / p.Hk);
    u.seq = order ? order[pos] : pos;
    u.jb = table_at(p, co, u.seq);
    u.nch = table_at(p, co, u.seq + 1) - u.jb;
    u.t_begin = p.cu_seqlens[u.seq];
    u.t_end = p.cu_seqlens[u.seq + 1];
    return KDA_BOUNDS(u.seq >= 0 && u.seq < p.num_seqs && u.h < p.Hv && u.t_begin >= 0 && u.t_end <= p.total_tokens &&
                          u.jb >= 0 && static_cast<int64_t>(u.jb) + u.nch <= chunk_slots &&
                          static_cast<int64_t>(u.nch) * C >= u.t_end - u.t_begin,
                      p.device_status);
}

// ST stages of tiles: full when their copies have landed, empty when the readers' warps are done with them.
struct WalkPipe {
    uint8_t* sm;
    uint64_t *full, *empty;
    volatile int* abort_s;  // a bounded wait expired somewhere in the CTA
};
__device__ __forceinline__ void pipe_init(const WalkPipe& p, int stages, int readers) {  // one thread
    for (int i = 0; i < stages; ++i) {
        mbar_init(&p.full[i], 1);
        mbar_init(&p.empty[i], readers);
    }
}
// One thread: step i's copies (`issue`) into stage i mod ST once its readers are done with step i - ST.
template <int ST, typename F>
__device__ __forceinline__ void pipe_copies(const WalkPipe& p, int steps, F issue) {
    int i = 0;
    for (; i < steps && !*p.abort_s; ++i) {
        const int s = i % ST;
        if (i >= ST && !mbar_wait_or_stop(&p.empty[s], ((i / ST) - 1) & 1)) {
            *p.abort_s = 1;
            break;
        }
        issue(i, s);
    }
    for (int d = max(0, i - ST); d < i; ++d)  // no copy is left in flight
        (void)mbar_wait(&p.full[d % ST], (d / ST) & 1, kDrainLimit);
}

// ------------------------------------------------------------- forward ----
// NW warps of 8 NT columns.  REC: the gradient's walk, which leaves every chunk's start state and U in two
// bf16 terms and no outputs.
template <int NT, int NW, int ST_, bool REC_>
struct ForwardCfg {
    static constexpr bool REC = REC_;
    static constexpr int ST = ST_;
    static constexpr int kCols = 8 * NT * NW;
    static constexpr uint32_t kVRow = 2 * kCols;  // bytes of a v row
    static constexpr uint32_t K = 0, IMG = 16384, V = IMG + 16384, Q = V + C * kVRow;
    static constexpr uint32_t STAGE = Q + (REC ? 0 : 16384);
    static_assert(kVRow == 64 || kVRow == 128, "swizzled rows");
    static_assert(STAGE % 1024 == 0 && kImgScanBytes <= 16384, "stages");
};

template <typename L>
__device__ __forceinline__ void forward_copies(const WalkUnit& u, const WalkPipe& pipe, const GdnArgs& p,
                                               const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                               const uint8_t* images) {
    pipe_copies<L::ST>(pipe, u.nch, [&](int c, int s) {
        uint8_t* st = pipe.sm + s * L::STAGE;
        uint64_t* bar = &pipe.full[s];
        const int32_t tok = static_cast<int32_t>(u.t_begin + static_cast<int64_t>(c) * C);
        mbar_arrive_expect_tx(bar, (L::REC ? 16384 : 32768) + kImgScanBytes + C * L::kVRow);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) tma_load_3d(st + L::K + kh * 8192, tm_k, bar, 64 * kh, u.hk, tok);
        tma_load_3d(st + L::V, tm_v, bar, u.col0, u.h, tok);
        bulk_g2s(st + L::IMG,
                 images + (static_cast<size_t>(u.jb + c) * p.Hv + u.h) * (L::REC ? kImgStrideBwd : kImgStride), kImgScanBytes,
                 bar);
#pragma unroll
        for (int kh = 0; kh < (L::REC ? 0 : 2); ++kh) tma_load_3d(st + L::Q + kh * 8192, tm_q, bar, 64 * kh, u.hk, tok);
    });
}

template <typename L, int NT>
__device__ __forceinline__ void walk_forward(const WalkUnit& wu, const WalkPipe& pipe, const GdnArgs& p, uint8_t* records,
                                             int warp, int lane) {
    constexpr bool REC = L::REC;
    constexpr int ST = L::ST;
    const int Hv = p.Hv;
    const int g = lane >> 2, t = lane & 3;
    const int wc = 8 * NT * warp;                  // the warp's first column in the CTA's
    const int j0 = wu.col0 + wc + 2 * t;  // this thread's first state column
    const size_t sbase = (static_cast<size_t>(wu.seq) * Hv + wu.h) * D * D;
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
    for (int c = 0; c < wu.nch; ++c) {
        const int s = c % ST;
        uint8_t* st = pipe.sm + s * L::STAGE;
        const bool landed = !*pipe.abort_s && mbar_wait_pipe(&pipe.full[s], (c / ST) & 1);
        if (!__all_sync(0xffffffffu, landed)) {  // a bounded wait expired, here or elsewhere
            *pipe.abort_s = 1;
            break;
        }
        const int64_t t0 = wu.t_begin + static_cast<int64_t>(c) * C;
        const int Lc = static_cast<int>(wu.t_end - t0 < C ? wu.t_end - t0 : C);
        if (Lc < C) {  // k rows behind the sequence's end meet zeros of U: they must be numbers
            for (int e = lane; e < (C - Lc) * 16; e += 32)
                *reinterpret_cast<uint4*>(st + L::K + (e & 1) * 8192 + sw128_chunk(Lc + (e >> 4), (e >> 1) & 7)) =
                    make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
        }
        const uint32_t kb = smem_u32(st + L::K), qb = smem_u32(st + L::Q), ib = smem_u32(st + L::IMG) + 16 * lane;
        const float* gs = reinterpret_cast<const float*>(st + L::IMG + kImgG);
        uint8_t* const rec = REC ? records + (static_cast<size_t>(wu.jb + c) * Hv + wu.h) * kRecStride : nullptr;
        const int rcol = (wu.col0 + wc) >> 3;  // matrices of 8 columns
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
                if constexpr (REC) put_record(S[k][n], rec + kRecS, 32768, 2 * k, rcol + n, lane);
                b[n] = b_terms(S[k][n]);
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
                    if constexpr (L::kVRow == 128) off = sw128_chunk(row, piece);
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
                for (int n = 0; n < NT; ++n) put_record(u[k][n], rec + kRecU, 16384, 2 * k, rcol + n, lane);
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
        if (lane == 0) mbar_arrive(&pipe.empty[s]);  // the warp has read all it takes of this stage
        if constexpr (!REC) {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + (t0 * Hv + wu.h) * D + j0;
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
    if (p.S_final && !*pipe.abort_s) {
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

}  // namespace gdn
}  // namespace kda
