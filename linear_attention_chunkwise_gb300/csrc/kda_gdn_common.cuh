// kda_gdn_common.cuh -- what the gated delta rule's chunkwise kernels share: the layout of a
// (chunk, value head)'s image and the warp-level pieces (ldmatrix, mma.sync, two-term operands).
#pragma once

#include <cuda_bf16.h>

#include "kda_gdn_internal.h"
#include "kda_gdn_ptx.cuh"

namespace kda {
namespace gdn {

constexpr int C = kChunk;    // 64
constexpr int D = kHeadDim;  // 128

// Image of a (chunk, value head): T's two terms and P's first, the ten 16 x 16 blocks on and below the
// diagonal of each; fp32 vectors; and, for the gradient, P's second and third term.  A block is its four
// 8 x 8 matrices (rows 0..7 and 8..15 of columns 0..7, then of columns 8..15), so that ldmatrix reads it
// with lane l's address at 16 l and a warp's fragment stores fill whole 128-byte lines.
constexpr uint32_t kBlkBytes = 512, kTriBytes = 10 * kBlkBytes;
constexpr uint32_t kImgTh = 0, kImgTl = kTriBytes, kImgP = 2 * kTriBytes, kImgG = 3 * kTriBytes;
constexpr uint32_t kImgPl = kImgG + 1536, kImgPl2 = kImgPl + kTriBytes;
// the vectors: e^g [64], e^(gC - g) [64], b [64], e^gC (and 3 floats unused), then g in base 2 as two terms
constexpr int kVecEg = 0, kVecEo = C, kVecB = 2 * C, kVecEc = 3 * C, kVecGh = 3 * C + 4, kVecGl = 4 * C + 4;
constexpr uint32_t kImgScanBytes = kImgG + (3 * C + 4) * 4;  // what the forward scan takes
constexpr size_t kImgStride = kImgPl, kImgStrideBwd = kImgPl2 + kTriBytes;
static_assert((5 * C + 4) * 4 <= 1536 && kImgStride % kAlign == 0 && kImgStrideBwd % kAlign == 0 &&
                  kImgScanBytes % 16 == 0,
              "image layout");
// The wide scan's images: T's two terms and P's first as whole 128B-swizzled [64][64] tiles, whose blocks above
// the diagonal are never written nor used, then the vectors.
constexpr uint32_t kTileBytes = 8192;
constexpr size_t kImgStrideTile = 3 * kTileBytes + 1536;
// Block (i, j), j <= i, and within it the pair of columns 2 t, 2 t + 1 of its half n in row g (+ 8 e).
__device__ __forceinline__ constexpr uint32_t tri_blk(int i, int j) { return (i * (i + 1) / 2 + j) * kBlkBytes; }
__device__ __forceinline__ uint32_t blk_pair(int g, int e, int n, int t) { return (2 * n + e) * 128 + 16 * g + 4 * t; }

// The gradient's record of a (chunk, value head): the state at the chunk's start, the adjoint of the state
// at its end ([128 channels][128 columns]), U and W ([64 tokens][128 columns]), each as two bf16 terms, in
// 8 x 8 matrices of 128 bytes, 16 of them to a row of matrices: a warp stores an accumulator's half as one
// line (as 128B-swizzled tiles, 16 bytes in each of 8 lines: the two walks 512 us for 8192 tokens x 32 heads),
// and ldmatrix reads it without conflicts.
constexpr uint32_t kRecS = 0, kRecX = 65536, kRecU = 131072, kRecW = 163840;
constexpr size_t kRecStride = 196608;

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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two bf16 terms of a pair of floats.  The first is off by at most 2^(e-8) for 2^e <= |x| <
// 2^(e+1); the second, rounding that, leaves at most 2^(e-17): 2^-17 of |x|.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(x, y);
    lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// 2^x by the special function unit (2 ulp); x is a difference of decays in base 2.
__device__ __forceinline__ float exp2_sfu(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t third2(float x, float y, uint32_t hi, uint32_t lo) {  // what two terms leave
    return pack_bf16((x - __uint_as_float(hi << 16)) - __uint_as_float(lo << 16),
                     (y - __uint_as_float(hi & 0xffff0000u)) - __uint_as_float(lo & 0xffff0000u));
}
// An accumulator tile's two terms into a record: matrices (rm, cm) and (rm + 1, cm), the second term `lo`
// bytes after the first.
__device__ __forceinline__ void put_record(const float (&c)[4], uint8_t* rec, uint32_t lo, int rm, int cm, int lane) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t h, l;
        split2(c[2 * e], c[2 * e + 1], h, l);
        uint8_t* p = rec + ((rm + e) * 16 + cm) * 128 + 4 * lane;
        *reinterpret_cast<uint32_t*>(p) = h;
        *reinterpret_cast<uint32_t*>(p + lo) = l;
    }
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

// The same with a third term, the rest to 2^-25.
struct BTerms3 {
    BTerms b;
    uint32_t m0, m1;
};
__device__ __forceinline__ BTerms3 b_terms3(const float (&c)[4]) {
    BTerms3 r;
    uint32_t h0, h1, l0, l1;
    split2(c[0], c[1], h0, l0);
    split2(c[2], c[3], h1, l1);
    r.m0 = transpose8(third2(c[0], c[1], h0, l0));
    r.m1 = transpose8(third2(c[2], c[3], h1, l1));
    r.b.h0 = transpose8(h0);
    r.b.h1 = transpose8(h1);
    r.b.l0 = transpose8(l0);
    r.b.l1 = transpose8(l1);
    return r;
}

}  // namespace gdn
}  // namespace kda
