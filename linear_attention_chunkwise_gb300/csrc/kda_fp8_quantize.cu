// kda_fp8_quantize.cu -- bf16 or fp32 to e4m3 with an fp32 scale for 128 elements of a row, 128 of a column, or a block of
// 128 x 128: the operands of kda_fp8_matmul that kda_rms_norm does not make.
//
//   scale = max(max |x| / 448, 2^-126),   code = x / scale rounded to nearest even
//
// Bound by HBM: x is read once, held in registers between the maximum and the rounding, and a byte an element is written.  The
// maximum is taken over the bits of |x|, whose order is that of the values with infinity and NaN on top, so either reaches the scale.
// The quotients are those of a division rounded once: with r = 1 / scale so rounded, q = x r and q + (x - q scale) r in fma (P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), three operations in place of a
// division's, which bound the kernel before (8192 x 4096 bf16 by rows: 59 us).  That needs a remainder that fp32 holds: its last bit stands 46
// places below the product of q's and scale's leading ones, and q counts down to 2^-11 (half of the smallest code rounds at 2^-10), so
// from scales of 2^-92 on it is 2^-149 or more.  Smaller scales divide.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_fp8_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

// N consecutive elements as they are in memory, bf16 two a word.
template <typename T, int N>
struct Held {
    static constexpr int kWords = N * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};
// Those behind `left` are zeros; VEC: all or none are there, and they are 16-byte aligned.
template <typename T, bool VEC, int N>
__device__ __forceinline__ void load(Held<T, N>& v, const T* p, int64_t left) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < Held<T, N>::kWords; i += 4) {
            const uint4 u = left >= N ? __ldcs(reinterpret_cast<const uint4*>(p) + i / 4) : make_uint4(0, 0, 0, 0);
            v.w[i] = u.x, v.w[i + 1] = u.y, v.w[i + 2] = u.z, v.w[i + 3] = u.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) v.w[i] = i < left ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : 0;
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < N; i += 2)
            v.w[i / 2] = (i < left ? __ldg(h + i) : 0) | static_cast<uint32_t>(i + 1 < left ? __ldg(h + i + 1) : 0) << 16;
    }
}
// The largest magnitudes word by word, as bits: of fp32, or of two bf16.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t most, uint32_t word) {
    if constexpr (sizeof(T) == 4) return max(most, word & 0x7fffffffu);
    else return __vmaxu2(most, word & 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t largest(uint32_t most) {  // of a word's, as bits of fp32
    if constexpr (sizeof(T) == 4) return most;
    else return max(most & 0xffff0000u, most << 16);
}
__device__ __forceinline__ float scale_of(uint32_t amax) {
    const float s = __fdiv_rn(__uint_as_float(amax), 448.0f);
    return s < 0x1p-126f ? 0x1p-126f : s;  // NaN stays
}
struct Scale {
    float s, r;  // and its reciprocal; r = 0 where quotients are divisions: s small or not finite
};
__device__ __forceinline__ Scale with_reciprocal(float s) {
    return {s, s >= 0x1p-92f && s < __int_as_float(0x7f800000) ? __frcp_rn(s) : 0.f};
}
// Codes of four quotients, the first in the lowest byte.
__device__ __forceinline__ uint32_t codes_of(const float (&q)[4]) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
// The same of WORDS times four values by one scale: value(i, j) is the j-th of word i.
template <int WORDS, typename F>
__device__ __forceinline__ void codes_by(const Scale& by, uint32_t (&c)[WORDS], const F& value) {
    if (by.r != 0.f) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            float q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = value(i, j), near = x * by.r;
                q[j] = fmaf(fmaf(-near, by.s, x), by.r, near);
            }
            c[i] = codes_of(q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            float q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = __fdiv_rn(value(i, j), by.s);
            c[i] = codes_of(q);
        }
    }
}
// N codes of a row; VEC as in load.
template <bool VEC, int N>
__device__ __forceinline__ void store(uint8_t* p, const uint32_t* c, int64_t left) {
    if constexpr (VEC) {
        if (left < N) return;
        if constexpr (N == 8) *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
        else *reinterpret_cast<uint32_t*>(p) = c[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = static_cast<uint8_t>(c[i / 4] >> 8 * (i % 4));
    }
}

// 128 of a row by 8 lanes, which have 16 each in vectors of 16 bytes that are 8 lanes apart; kAhead times a warp's four groups at once.
constexpr int kAhead = 2, kLanes = 8, kGroups = 32 / kLanes;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) kda_fp8_quantize_rows_kernel(const Fp8QuantizeArgs a) {
    constexpr int N = 16 / sizeof(T), kVectors = kFp8Block / kLanes / N;
    const int lane = threadIdx.x & 31;
    const int64_t per_row = (a.cols + kFp8Block - 1) / kFp8Block, groups = a.rows * per_row;
    const T* x = static_cast<const T*>(a.x);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kAhead * kGroups + lane / kLanes;
    Held<T, N> v[kAhead][kVectors];
    int64_t at[kAhead], row = first / per_row, group = first - row * per_row;
    int32_t left[kAhead];  // of a group's columns, behind the lane's first
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int64_t col = group * kFp8Block + lane % kLanes * N;
        at[i] = row * a.cols + col;
        left[i] = first + i * kGroups < groups ? static_cast<int32_t>(min(a.cols - col, static_cast<int64_t>(kFp8Block))) : 0;
#pragma unroll
        for (int j = 0; j < kVectors; ++j) load<T, VEC, N>(v[i][j], x + at[i] + j * kLanes * N, left[i] - j * kLanes * N);
        for (group += kGroups; group >= per_row; group -= per_row) ++row;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kVectors; ++j)
#pragma unroll
            for (int k = 0; k < Held<T, N>::kWords; ++k) m = larger<T>(m, v[i][j].w[k]);
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) m = larger<T>(m, __shfl_xor_sync(~0u, m, d));
        const Scale s = with_reciprocal(scale_of(largest<T>(m)));
        uint32_t c[4];
        codes_by(s, c, [&](int w, int j) { return v[i][w * 4 / N][w * 4 % N + j]; });
#pragma unroll
        for (int j = 0; j < kVectors; ++j)
            store<VEC, N>(static_cast<uint8_t*>(a.codes) + at[i] + j * kLanes * N, c + j * N / 4, left[i] - j * kLanes * N);
        if (lane % kLanes == 0 && first + i * kGroups < groups) a.scales[first + i * kGroups] = s.s;
    }
}

// 128 rows x 64 columns whose codes are turned over (COLUMNS), or a block of 128 x 128.  A thread has 4 rows beside each other of 8
// columns: their codes are a word of the turned rows.
template <bool COLUMNS>
constexpr int kTileCols = COLUMNS ? 64 : kFp8Block;
template <typename T, bool COLUMNS, bool VEC>
__global__ void __launch_bounds__(4 * kTileCols<COLUMNS>) kda_fp8_quantize_tile_kernel(const Fp8QuantizeArgs a) {
    constexpr int kCols = kTileCols<COLUMNS>, kAcross = kCols / 8, kWarps = kCols / 8;
    __shared__ uint32_t most[kWarps][COLUMNS ? kCols : 1];
    __shared__ Scale scale[COLUMNS ? kCols : 1];
    __shared__ __align__(16) uint32_t turned[COLUMNS ? kCols * 32 : 1];  // rows of 128 codes, 16-byte chunks swizzled
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = threadIdx.x % kAcross, rg = threadIdx.x / kAcross;
    const int64_t across = (a.cols + kCols - 1) / kCols, down = (a.rows + kFp8Block - 1) / kFp8Block;
    const int64_t tile_c = blockIdx.x % across, tile_r = blockIdx.x / across;
    const int64_t row0 = tile_r * kFp8Block + rg * 4, col0 = tile_c * kCols + ch * 8;
    const T* x = static_cast<const T*>(a.x);
    uint8_t* codes = static_cast<uint8_t*>(a.codes);
    using Row = Held<T, 8>;
    Row v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) load<T, VEC, 8>(v[i], x + (row0 + i) * a.cols + col0, row0 + i < a.rows ? a.cols - col0 : 0);
    uint32_t m[Row::kWords] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < Row::kWords; ++j) m[j] = larger<T>(m[j], v[i].w[j]);
    if constexpr (COLUMNS) {  // a warp: 4 groups of rows beside each other
#pragma unroll
        for (int j = 0; j < Row::kWords; ++j) {
            m[j] = larger<T>(m[j], __shfl_xor_sync(~0u, m[j], 8));
            m[j] = larger<T>(m[j], __shfl_xor_sync(~0u, m[j], 16));
            if (lane < 8) {
                if constexpr (sizeof(T) == 4) {
                    most[warp][lane * 8 + j] = m[j];
                } else {
                    most[warp][lane * 8 + 2 * j] = m[j] << 16;
                    most[warp][lane * 8 + 2 * j + 1] = m[j] & 0xffff0000u;
                }
            }
        }
    } else {
        uint32_t all = 0;
#pragma unroll
        for (int j = 0; j < Row::kWords; ++j) all = larger<T>(all, m[j]);
        const uint32_t of_warp = __reduce_max_sync(~0u, largest<T>(all));
        if (lane == 0) most[warp][0] = of_warp;
    }
    __syncthreads();
    if (threadIdx.x < (COLUMNS ? kCols : 1)) {
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all = max(all, most[w][threadIdx.x]);
        const Scale s = with_reciprocal(scale_of(all));
        scale[threadIdx.x] = s;
        const int64_t c = tile_c * kCols + threadIdx.x;
        if (!COLUMNS) a.scales[blockIdx.x] = s.s;
        else if (c < a.cols) a.scales[c * down + tile_r] = s.s;
    }
    __syncthreads();
    if constexpr (!COLUMNS) {
        const Scale s = scale[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c[2];
            codes_by(s, c, [&](int w, int j) { return v[i][w * 4 + j]; });
            store<VEC, 8>(codes + (row0 + i) * a.cols + col0, c, row0 + i < a.rows ? a.cols - col0 : 0);
        }
    } else {
        const auto word = [&](int c, int chunk) { return turned + c * 32 + ((chunk ^ c / 8) & 7) * 4; };
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t c[1];
            codes_by(scale[ch * 8 + j], c, [&](int, int i) { return v[i][j]; });
            word(ch * 8 + j, rg / 4)[rg % 4] = c[0];
        }
        __syncthreads();
        // rows of the result, where they are whole vectors apart 8 lanes each, 16 codes a lane
        if (a.rows % 16 == 0) {
            const int64_t first = tile_r * kFp8Block + lane % 8 * 16;
            for (int c = warp * 4 + lane / 8; c < kCols; c += kWarps * 4) {
                const int64_t out = tile_c * kCols + c;
                if (out >= a.cols) break;
                if (first < a.rows) *reinterpret_cast<uint4*>(codes + out * a.rows + first) = *reinterpret_cast<const uint4*>(word(c, lane % 8));
            }
        } else {  // else a warp each, consecutive bytes at once (8191 x 4096 bf16: 37 us, 16 bytes of a lane one by one 104)
            const int64_t first = tile_r * kFp8Block, left = a.rows - first;
            for (int c = warp; c < kCols; c += kWarps) {
                const int64_t out = tile_c * kCols + c;
                if (out >= a.cols) break;
                uint8_t* to = codes + out * a.rows + first;
#pragma unroll
                for (int i = 0; i < kFp8Block; i += 32)
                    if (i + lane < left) to[i + lane] = reinterpret_cast<const uint8_t*>(word(c, (i + lane) / 16))[lane % 16];
            }
        }
    }
}

template <typename T, bool VEC>
cudaError_t quantize(int32_t form, const Fp8QuantizeArgs& a, cudaStream_t stream) {
    const int64_t down = (a.rows + kFp8Block - 1) / kFp8Block;
    const auto across = [&](int cols) { return (a.cols + cols - 1) / cols; };
    if (form == KDA_FP8_ROWS) {
        const int64_t per_block = kThreads / 32 * kAhead * kGroups, groups = a.rows * across(kFp8Block);
        kda_fp8_quantize_rows_kernel<T, VEC><<<static_cast<unsigned>((groups + per_block - 1) / per_block), kThreads, 0, stream>>>(a);
    } else if (form == KDA_FP8_COLUMNS) {
        constexpr int kCols = kTileCols<true>;
        kda_fp8_quantize_tile_kernel<T, true, VEC><<<static_cast<unsigned>(across(kCols) * down), 4 * kCols, 0, stream>>>(a);
    } else {
        constexpr int kCols = kTileCols<false>;
        kda_fp8_quantize_tile_kernel<T, false, VEC><<<static_cast<unsigned>(across(kCols) * down), 4 * kCols, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(bool x_f32, int32_t form, const Fp8QuantizeArgs& a, cudaStream_t stream) {
    if (a.rows == 0 || a.cols == 0) return cudaSuccess;
    const bool vec = a.cols % 8 == 0;  // rows of whole vectors
    if (x_f32) return vec ? quantize<float, true>(form, a, stream) : quantize<float, false>(form, a, stream);
    return vec ? quantize<__nv_bfloat16, true>(form, a, stream) : quantize<__nv_bfloat16, false>(form, a, stream);
}

}  // namespace kda
