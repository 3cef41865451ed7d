// kda_rms_norm.cu -- root-mean-square norm with the residual's addition and an
// optional output in 8 bits with scales, and its gradient.
//
//   h = round(x + residual)            (stored, in the input type; h = x without one)
//   y = h * (mean_c h_c^2 + eps)^(-1/2) * w
//   8 bits: scale = max(max|y| / qmax, 2^-126) over the row or 128 columns of it,
//           code = round(y / scale)    (e4m3: qmax 448, int8: qmax 127)
//
// Both directions are bound by HBM: each row is read once, held in registers
// across its reduction(s), and written once.  A row of up to 128 vectors of
// 16 bytes belongs to one warp (no block barrier), a longer one to a block; a
// row too long for a block's registers is read again, from L2.  Every sum is
// fp32 in a fixed order, so results are bitwise repeatable.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kWarpRows = 8;        // rows of a block in the warp-per-row form
constexpr int kMaxThreads = 1024;

// V consecutive elements of a row as floats, and back.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};
__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
    const Vec<T, V> v = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = as_f32(v.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    Vec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f32(v.e[i], f[i]);
    *reinterpret_cast<Vec<T, V>*>(p) = v;
}
template <int V>
__device__ __forceinline__ void load_weight(const float* w, int c, float (&f)[V]) {
    if (w) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __ldg(w + c + i);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 1.f;
    }
}

// Sum (or the largest bit pattern) over the threads that hold a row: a warp, or the block.
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float x, float* part) {
    x = warp_sum(x);
    if (BLOCK) {
        const int lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
        if (lane == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        x = warp_sum(lane < nw ? part[lane] : 0.f);
    }
    return x;
}
// |y| of every sign is ordered as its bits are, infinity above the finite values and NaN above both.
__device__ __forceinline__ uint32_t abs_bits(float y) { return __float_as_uint(y) & 0x7fffffffu; }
template <bool BLOCK>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t* part) {
    x = __reduce_max_sync(0xffffffffu, x);
    if (BLOCK) {
        const int lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
        if (lane == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        x = __reduce_max_sync(0xffffffffu, lane < nw ? part[lane] : 0u);
    }
    return x;
}

// The output types: 0 = as the input, 1 = e4m3, 2 = int8.
template <int OUT>
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float s = __uint_as_float(amax_bits) * (OUT == 1 ? 1.f / 448.f : 1.f / 127.f);
    return s < 1.17549435e-38f ? 1.17549435e-38f : s;  // a row of zeros has a scale too; NaN stays
}
template <int OUT, int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&y)[V], float inv) {
    Vec<uint8_t, V> v;
    if constexpr (OUT == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) v.e[i] = __nv_cvt_float_to_fp8(y[i] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int q = __float2int_rn(y[i] * inv);  // NaN gives 0
            v.e[i] = static_cast<uint8_t>(static_cast<int8_t>(q > 127 ? 127 : q < -127 ? -127 : q));
        }
    }
    *reinterpret_cast<Vec<uint8_t, V>*>(p) = v;
}

// One row for each warp (BLOCK false, blockDim 32 x kWarpRows) or block.  NV vectors of V elements in
// each thread's registers: vector j of a thread starts at column V (t + j threads).
template <typename T, int OUT, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxThreads : 32 * kWarpRows) kda_rms_norm_kernel(const NormArgs a) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int nt = BLOCK ? blockDim.x : 32;
    const int t = BLOCK ? threadIdx.x : (threadIdx.x & 31);
    const int64_t row = BLOCK ? static_cast<int64_t>(blockIdx.x)
                              : static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5);
    if (!BLOCK && row >= a.rows) return;
    const int64_t base = row * a.dim;
    const T* x = static_cast<const T*>(a.x) + base;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + base : nullptr;
    T* hout = a.residual_out ? static_cast<T*>(a.residual_out) + base : nullptr;
    float h[NV][V];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = V * (t + j * nt);
        if (c < a.dim) {
            load_vec<T, V>(x + c, h[j]);
            if (res) {
                float r[V];
                load_vec<T, V>(res + c, r);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    T u;
                    from_f32(u, h[j][i] + r[i]);  // the norm is that of the stored row
                    h[j][i] = as_f32(u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] = 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = V * (t + j * nt);
        if (hout && c < a.dim) store_vec<T, V>(hout + c, h[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(h[j][i], h[j][i], ss);
    }
    const float r = rsqrtf(row_sum<BLOCK>(ss * (1.f / static_cast<float>(a.dim)), s_sum) + a.eps);
    uint32_t mx = 0u;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = V * (t + j * nt);
        if (c >= a.dim) continue;  // h there is 0 already
        float w[V];
        load_weight<V>(a.weight, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[j][i] = h[j][i] * r * w[i];
            if (OUT && a.group == 0) mx = max(mx, abs_bits(h[j][i]));
        }
    }
    if constexpr (OUT == 0) {
        T* y = static_cast<T*>(a.y) + base;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c < a.dim) store_vec<T, V>(y + c, h[j]);
        }
    } else {
        uint8_t* y = static_cast<uint8_t*>(a.y) + base;
        if (a.group == 0) {
            const float s = scale_of<OUT>(row_max<BLOCK>(mx, s_max)), inv = 1.f / s;
            if (t == 0) a.scales[row] = s;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = V * (t + j * nt);
                if (c < a.dim) store_codes<OUT, V>(y + c, h[j], inv);
            }
        } else if constexpr (V * sizeof(T) == 16) {  // 128 columns: 128 / V lanes of a warp (dim is a multiple)
            constexpr int LG = 128 / V;
            const int64_t g0 = row * (a.dim / 128);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = V * (t + j * nt);
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, abs_bits(h[j][i]));
#pragma unroll
                for (int off = LG / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
                if (c < a.dim) {
                    const float s = scale_of<OUT>(m), inv = 1.f / s;
                    if ((c & 127) == 0) a.scales[g0 + (c >> 7)] = s;
                    store_codes<OUT, V>(y + c, h[j], inv);
                }
            }
        }
    }
}

// A row too long for a block's registers: the block reads it once for the sum of squares, once more for
// the largest value (8 bits, one scale for the row) and once for the output, from L2 after the first.
template <typename T, int OUT, int V>
__global__ void __launch_bounds__(kMaxThreads) kda_rms_norm_long_kernel(const NormArgs a) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int nt = blockDim.x, t = threadIdx.x;
    const int64_t row = blockIdx.x, base = row * a.dim;
    // h of the columns from c; what this thread stores in residual_out (which may be x or the residual
    // itself) it reads back from there, each column staying with its thread
    const T* const hin = a.residual ? static_cast<const T*>(a.residual_out) : static_cast<const T*>(a.x);
    auto load_h = [&](int c, float(&f)[V]) {
        if (hin) {
            load_vec<T, V>(hin + base + c, f);
        } else {
            float r[V];
            load_vec<T, V>(static_cast<const T*>(a.x) + base + c, f);
            load_vec<T, V>(static_cast<const T*>(a.residual) + base + c, r);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                T u;
                from_f32(u, f[i] + r[i]);
                f[i] = as_f32(u);
            }
        }
    };
    float ss = 0.f;
    for (int c = V * t; c < a.dim; c += V * nt) {
        float f[V];
        load_vec<T, V>(static_cast<const T*>(a.x) + base + c, f);
        if (a.residual) {
            float r[V];
            load_vec<T, V>(static_cast<const T*>(a.residual) + base + c, r);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                T u;
                from_f32(u, f[i] + r[i]);
                f[i] = as_f32(u);
            }
        }
        if (a.residual_out) store_vec<T, V>(static_cast<T*>(a.residual_out) + base + c, f);
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(f[i], f[i], ss);
    }
    const float r = rsqrtf(row_sum<true>(ss * (1.f / static_cast<float>(a.dim)), s_sum) + a.eps);
    float inv = 0.f;
    if constexpr (OUT != 0) {
        if (a.group == 0) {
            uint32_t mx = 0u;
            for (int c = V * t; c < a.dim; c += V * nt) {
                float f[V], w[V];
                load_h(c, f);
                load_weight<V>(a.weight, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) mx = max(mx, abs_bits(f[i] * r * w[i]));
            }
            const float s = scale_of<OUT>(row_max<true>(mx, s_max));
            inv = 1.f / s;
            if (t == 0) a.scales[row] = s;
        }
    }
    for (int c0 = 0; c0 < a.dim; c0 += V * nt) {  // whole warps stay together for the groups' shuffles
        const int c = c0 + V * t;
        float f[V], w[V];
        const bool in = c < a.dim;
        if (in) {
            load_h(c, f);
            load_weight<V>(a.weight, c, w);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = in ? f[i] * r * w[i] : 0.f;
        if constexpr (OUT == 0) {
            if (in) store_vec<T, V>(static_cast<T*>(a.y) + base + c, f);
        } else {
            float gi = inv;
            if constexpr (V * sizeof(T) == 16) {
                if (a.group) {
                    constexpr int LG = 128 / V;
                    uint32_t m = 0u;
#pragma unroll
                    for (int i = 0; i < V; ++i) m = max(m, abs_bits(f[i]));
#pragma unroll
                    for (int off = LG / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
                    const float s = scale_of<OUT>(m);
                    gi = 1.f / s;
                    if (in && (c & 127) == 0) a.scales[row * (a.dim / 128) + (c >> 7)] = s;
                }
            }
            if (in) store_codes<OUT, V>(static_cast<uint8_t*>(a.y) + base + c, f, gi);
        }
    }
}

// ------------------------------------------------------------- gradient ----
//   grad_x = r w dy - h r^3 / dim * sum_c h w dy + grad_h,   grad_w = sum over rows of dy h r
// Both row sums (h^2 and h w dy) are taken in one reduction.  A block keeps its columns' share of
// grad_w in registers over its rows and writes it once; the blocks' shares are added in order by
// kda_rms_norm_weight_kernel.
template <bool BLOCK>
__device__ __forceinline__ float2 row_sum2(float x, float y, float2* part) {
    x = warp_sum(x);
    y = warp_sum(y);
    if (BLOCK) {
        const int lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
        __syncthreads();  // the previous row's sums have been read
        if (lane == 0) part[threadIdx.x >> 5] = make_float2(x, y);
        __syncthreads();
        const float2 p = lane < nw ? part[lane] : make_float2(0.f, 0.f);
        x = warp_sum(p.x);
        y = warp_sum(p.y);
    }
    return make_float2(x, y);
}

template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxThreads : 32 * kWarpRows)
    kda_rms_norm_backward_kernel(const NormBackwardArgs a) {
    __shared__ float2 s_sum[32];
    extern __shared__ float s_w[];  // warp-per-row form: the warps' shares of grad_w, [dim]
    const int nt = BLOCK ? blockDim.x : 32;
    const int t = BLOCK ? threadIdx.x : (threadIdx.x & 31);
    const int warp = threadIdx.x >> 5;
    const int64_t step = BLOCK ? gridDim.x : static_cast<int64_t>(gridDim.x) * kWarpRows;
    const T* gy = static_cast<const T*>(a.grad_y);
    const T* hh = static_cast<const T*>(a.h);
    const T* gh = static_cast<const T*>(a.grad_h);
    const float inv_dim = 1.f / static_cast<float>(a.dim);
    float w[NV][V], dw[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = V * (t + j * nt);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[j][i] = 0.f;
            dw[j][i] = 0.f;
        }
        if (c < a.dim) load_weight<V>(a.weight, c, w[j]);
    }
    for (int64_t row = BLOCK ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWarpRows + warp; row < a.rows;
         row += step) {
        const int64_t base = row * a.dim;
        float h[NV][V], dy[NV][V], g[NV][V];
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] = dy[j][i] = g[j][i] = 0.f;
            if (c < a.dim) {
                load_vec<T, V>(hh + base + c, h[j]);
                load_vec<T, V>(gy + base + c, dy[j]);
                if (gh) load_vec<T, V>(gh + base + c, g[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ss = fmaf(h[j][i], h[j][i], ss);
                sd = fmaf(h[j][i] * w[j][i], dy[j][i], sd);
            }
        const float2 s = row_sum2<BLOCK>(ss * inv_dim, sd * inv_dim, s_sum);
        const float r = rsqrtf(s.x + a.eps);
        const float m = s.y * r * r * r;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c >= a.dim) continue;
            float dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dx[i] = fmaf(r * w[j][i], dy[j][i], fmaf(-m, h[j][i], g[j][i]));
                dw[j][i] = fmaf(dy[j][i] * r, h[j][i], dw[j][i]);
            }
            store_vec<T, V>(static_cast<T*>(a.grad_x) + base + c, dx);
        }
    }
    if (!a.grad_weight) return;
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
    if (BLOCK) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c < a.dim) store_vec<float, V>(part + c, dw[j]);
        }
    } else {  // the block's warps in order
        for (int k = 0; k < kWarpRows; ++k) {
            if (warp == k) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = V * (t + j * nt);
                    if (c >= a.dim) continue;
#pragma unroll
                    for (int i = 0; i < V; ++i) s_w[c + i] = k ? s_w[c + i] + dw[j][i] : dw[j][i];
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.dim; c += blockDim.x) part[c] = s_w[c];
    }
}

// A row too long for a block's registers: each row is read twice, and grad_w's shares are added up in
// the block's own row of `partial`.
template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads) kda_rms_norm_backward_long_kernel(const NormBackwardArgs a) {
    __shared__ float2 s_sum[32];
    const int nt = blockDim.x, t = threadIdx.x;
    const T* gy = static_cast<const T*>(a.grad_y);
    const T* hh = static_cast<const T*>(a.h);
    const T* gh = static_cast<const T*>(a.grad_h);
    const float inv_dim = 1.f / static_cast<float>(a.dim);
    float* part = a.grad_weight ? a.partial + static_cast<int64_t>(blockIdx.x) * a.dim : nullptr;
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false) {
        const int64_t base = row * a.dim;
        float ss = 0.f, sd = 0.f;
        for (int c = V * t; c < a.dim; c += V * nt) {
            float h[V], dy[V], w[V];
            load_vec<T, V>(hh + base + c, h);
            load_vec<T, V>(gy + base + c, dy);
            load_weight<V>(a.weight, c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ss = fmaf(h[i], h[i], ss);
                sd = fmaf(h[i] * w[i], dy[i], sd);
            }
        }
        const float2 s = row_sum2<true>(ss * inv_dim, sd * inv_dim, s_sum);
        const float r = rsqrtf(s.x + a.eps);
        const float m = s.y * r * r * r;
        for (int c = V * t; c < a.dim; c += V * nt) {
            float h[V], dy[V], w[V], g[V], dw[V];
            load_vec<T, V>(hh + base + c, h);
            load_vec<T, V>(gy + base + c, dy);
            load_weight<V>(a.weight, c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = dw[i] = 0.f;
            if (gh) load_vec<T, V>(gh + base + c, g);
            if (part && !first) load_vec<float, V>(part + c, dw);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dw[i] = fmaf(dy[i] * r, h[i], dw[i]);
                g[i] = fmaf(r * w[i], dy[i], fmaf(-m, h[i], g[i]));
            }
            store_vec<T, V>(static_cast<T*>(a.grad_x) + base + c, g);
            if (part) store_vec<float, V>(part + c, dw);
        }
    }
}

// grad_w = the row blocks' shares in a fixed order: a block takes 32 columns, each of its 32 warps every
// 32nd share, and the warps' sums are added in order.
__global__ void __launch_bounds__(1024) kda_rms_norm_weight_kernel(const float* __restrict__ partial, int64_t parts,
                                                                   int32_t dim, float* __restrict__ grad_weight) {
    __shared__ float s_part[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < dim) {
#pragma unroll 8
        for (int64_t p = warp; p < parts; p += 32) s += partial[p * dim + c];
    }
    s_part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < dim) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += s_part[k][lane];
        grad_weight[c] = s;
    }
}

// Elements in a vector: 16 bytes when every row starts on 16 bytes, else 4 bytes, else one element.
template <typename T>
int vec_of(int32_t dim) {
    constexpr int full = 16 / sizeof(T), word = 4 / sizeof(T);
    return dim % full == 0 ? full : dim % word == 0 ? word : 1;
}

template <typename T, int OUT, int V>
cudaError_t norm_v(const NormArgs& a, cudaStream_t stream) {
    const int nvec = a.dim / V;
    if (nvec <= 128) {  // a warp's registers hold the row
        const unsigned blocks = static_cast<unsigned>((a.rows + kWarpRows - 1) / kWarpRows);
        if (nvec <= 32) kda_rms_norm_kernel<T, OUT, V, 1, false><<<blocks, 32 * kWarpRows, 0, stream>>>(a);
        else if (nvec <= 64) kda_rms_norm_kernel<T, OUT, V, 2, false><<<blocks, 32 * kWarpRows, 0, stream>>>(a);
        else kda_rms_norm_kernel<T, OUT, V, 4, false><<<blocks, 32 * kWarpRows, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const unsigned blocks = static_cast<unsigned>(a.rows);
    const int nv = nvec <= 2 * kMaxThreads ? 2 : 4;
    const int threads = std::min(kMaxThreads, ((nvec + nv - 1) / nv + 31) / 32 * 32);
    if (nvec <= 2 * kMaxThreads) kda_rms_norm_kernel<T, OUT, V, 2, true><<<blocks, threads, 0, stream>>>(a);
    else if (nvec <= 4 * kMaxThreads) kda_rms_norm_kernel<T, OUT, V, 4, true><<<blocks, threads, 0, stream>>>(a);
    else kda_rms_norm_long_kernel<T, OUT, V><<<blocks, kMaxThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int OUT>
cudaError_t norm_out(const NormArgs& a, cudaStream_t stream) {
    constexpr int full = 16 / sizeof(T), word = 4 / sizeof(T);
    const int v = vec_of<T>(a.dim);
    if (v == full) return norm_v<T, OUT, full>(a, stream);
    if (word > 1 && v == word) return norm_v<T, OUT, word>(a, stream);
    return norm_v<T, OUT, 1>(a, stream);
}

template <typename T>
cudaError_t norm_t(int32_t out_type, const NormArgs& a, cudaStream_t stream) {
    if (out_type == KDA_NORM_OUT_E4M3) return norm_out<T, 1>(a, stream);
    if (out_type == KDA_NORM_OUT_INT8) return norm_out<T, 2>(a, stream);
    return norm_out<T, 0>(a, stream);
}

template <typename T, int V>
cudaError_t norm_backward_v(const NormBackwardArgs& a, unsigned blocks, cudaStream_t stream) {
    const int nvec = a.dim / V;
    if (nvec <= 128) {
        const size_t smem = a.grad_weight ? static_cast<size_t>(a.dim) * 4 : 0;  // at most 4 KB
        if (nvec <= 32) kda_rms_norm_backward_kernel<T, V, 1, false><<<blocks, 32 * kWarpRows, smem, stream>>>(a);
        else if (nvec <= 64) kda_rms_norm_backward_kernel<T, V, 2, false><<<blocks, 32 * kWarpRows, smem, stream>>>(a);
        else kda_rms_norm_backward_kernel<T, V, 4, false><<<blocks, 32 * kWarpRows, smem, stream>>>(a);
        return cudaGetLastError();
    }
    const int nv = nvec <= kMaxThreads ? 1 : 2;
    const int threads = std::min(kMaxThreads, ((nvec + nv - 1) / nv + 31) / 32 * 32);
    if (nvec <= kMaxThreads) kda_rms_norm_backward_kernel<T, V, 1, true><<<blocks, threads, 0, stream>>>(a);
    else if (nvec <= 2 * kMaxThreads) kda_rms_norm_backward_kernel<T, V, 2, true><<<blocks, threads, 0, stream>>>(a);
    else kda_rms_norm_backward_long_kernel<T, V><<<blocks, kMaxThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_t(const NormBackwardArgs& a, unsigned blocks, cudaStream_t stream) {
    constexpr int full = 16 / sizeof(T), word = 4 / sizeof(T);
    const int v = vec_of<T>(a.dim);
    if (v == full) return norm_backward_v<T, full>(a, blocks, stream);
    if (word > 1 && v == word) return norm_backward_v<T, word>(a, blocks, stream);
    return norm_backward_v<T, 1>(a, blocks, stream);
}

}  // namespace

cudaError_t launch_rms_norm(bool f32_io, int32_t out_type, const NormArgs& a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    return f32_io ? norm_t<float>(out_type, a, stream) : norm_t<__nv_bfloat16>(out_type, a, stream);
}

// Four blocks an SM (of 152): enough rows in flight, few enough shares of grad_w.
int64_t rms_norm_backward_partials(int64_t rows) { return std::min<int64_t>(rows, 608); }

cudaError_t launch_rms_norm_backward(bool f32_io, const NormBackwardArgs& a, cudaStream_t stream) {
    const int64_t parts = rms_norm_backward_partials(a.rows);
    cudaError_t err = cudaSuccess;
    if (parts > 0) {
        const unsigned blocks = static_cast<unsigned>(parts);
        err = f32_io ? norm_backward_t<float>(a, blocks, stream) : norm_backward_t<__nv_bfloat16>(a, blocks, stream);
    }
    if (err != cudaSuccess || !a.grad_weight) return err;
    kda_rms_norm_weight_kernel<<<(a.dim + 31) / 32, 1024, 0, stream>>>(a.partial, parts, a.dim, a.grad_weight);
    return cudaGetLastError();
}

}  // namespace kda
