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
// fp32 in a fixed order, so results are bitwise repeatable.  8192 x 4096 bf16
// with a residual to e4m3 in groups of 128: 44 us, 5.4 TB/s of what it has to
// move; its gradient 47 us, 5.7 TB/s, 5 us of it the weight's second pass.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_gdn_internal.h"
#include "kda_gdn_ptx.cuh"

namespace kda {
namespace {

constexpr int kWarpRows = 8;        // rows of a block in the warp-per-row form
constexpr int kRowThreads = 512;    // most threads of a block that holds a row in registers (128 each)
constexpr int kMaxThreads = 1024;   // of one that reads it again

// V consecutive elements of a row, as they are in memory and as floats.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};
__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_raw(const T* p) {
    Vec<T, V> v;
    if constexpr (sizeof(v) == 16) {  // read once: not kept in L1
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        v = *reinterpret_cast<const Vec<T, V>*>(&u);
    } else {
        v = *reinterpret_cast<const Vec<T, V>*>(p);
    }
    return v;
}
// A row's vectors come through a thread's own slots of shared memory, S rows ahead (16-byte vectors; others
// are loaded when their row starts): enough bytes in flight without the registers for them.  The slots are
// the thread's alone, so there is no barrier; a slot is refilled after its row's sums, which need its values.
template <typename T, int V, int NV, int A, int S>
struct Ring {
    static constexpr bool ON = sizeof(Vec<T, V>) == 16;
    static constexpr uint32_t bytes(int threads) { return ON ? S * A * NV * 16u * threads : 0u; }
    uint32_t base;   // this thread's first slot
    uint32_t step;   // bytes between slots
    __device__ void start(const void* smem) {
        base = smem_u32(smem) + 16 * threadIdx.x;
        step = 16 * blockDim.x;
    }
    __device__ void fetch(int slot, int a, int j, const T* p, bool in) const {
        if (in)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + ((slot * A + a) * NV + j) * step),
                         "l"(reinterpret_cast<uint64_t>(p))
                         : "memory");
    }
    __device__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    __device__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory"); }
    __device__ Vec<T, V> get(int slot, int a, int j) const {
        uint4 u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(base + ((slot * A + a) * NV + j) * step)
                     : "memory");
        Vec<T, V> v;
        memcpy(&v, &u, 16);
        return v;
    }
};
// Rows ahead: blocks of 256 and 512 threads then leave several on an SM, with 100 to 200 KB in flight.
constexpr int ahead(int nv, bool block) { return block ? (nv <= 2 ? 4 : 3) : 5 - (nv < 3 ? nv : 3); }

template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& v, float (&f)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint32_t u;
            memcpy(&u, &v.e[i], 4);
            f[i] = __uint_as_float(u << 16);
            f[i + 1] = __uint_as_float(u & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = as_f32(v.e[i]);
    }
}
// x + y in their type, rounded once.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> add_vec(const Vec<T, V>& x, const Vec<T, V>& y) {
    Vec<T, V> z;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            __nv_bfloat162 a, b;
            memcpy(&a, &x.e[i], 4);
            memcpy(&b, &y.e[i], 4);
            a = __hadd2(a, b);
            memcpy(&z.e[i], &a, 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) from_f32(z.e[i], as_f32(x.e[i]) + as_f32(y.e[i]));
    }
    return z;
}
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
    widen<T, V>(load_raw<T, V>(p), f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    Vec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f32(v.e[i], f[i]);
    *reinterpret_cast<Vec<T, V>*>(p) = v;
}
// The weights of V columns from c (a multiple of V); ones without a weight.
template <int V>
__device__ __forceinline__ void load_weight(const float* w, int c, float (&f)[V]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = 1.f;
    } else if (V % 4 == 0 && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
#pragma unroll
        for (int i = 0; i + 4 <= V; i += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(w + c + i));
            f[i] = x.x; f[i + 1] = x.y; f[i + 2] = x.z; f[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __ldg(w + c + i);
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
// The larger of m and |y|, NaN if either is.
__device__ __forceinline__ float max_abs(float m, float y) {
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(y)));
    return m;
}
template <bool BLOCK>
__device__ __forceinline__ float row_max(float x, float* part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = max_abs(x, __shfl_xor_sync(0xffffffffu, x, off));
    if (BLOCK) {
        const int lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
        if (lane == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        x = lane < nw ? part[lane] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x = max_abs(x, __shfl_xor_sync(0xffffffffu, x, off));
    }
    return x;
}

// The output types: 0 = as the input, 1 = e4m3, 2 = int8.
template <int OUT>
__device__ __forceinline__ float scale_of(float amax) {
    const float s = amax * (OUT == 1 ? 1.f / 448.f : 1.f / 127.f);
    return s < 1.17549435e-38f ? 1.17549435e-38f : s;  // a row of zeros has a scale too; NaN stays
}
template <int OUT, int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&y)[V], float inv) {
    Vec<uint8_t, V> v;
    if constexpr (OUT == 1) {
        if constexpr (V % 2 == 0) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const __nv_fp8x2_storage_t q =
                    __nv_cvt_float2_to_fp8x2(make_float2(y[i] * inv, y[i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                v.e[i] = static_cast<uint8_t>(q & 0xff);
                v.e[i + 1] = static_cast<uint8_t>(q >> 8);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v.e[i] = __nv_cvt_float_to_fp8(y[i] * inv, __NV_SATFINITE, __NV_E4M3);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int q = __float2int_rn(y[i] * inv);  // NaN gives 0
            v.e[i] = static_cast<uint8_t>(static_cast<int8_t>(q > 127 ? 127 : q < -127 ? -127 : q));
        }
    }
    *reinterpret_cast<Vec<uint8_t, V>*>(p) = v;
}

// Rows of a warp (BLOCK false, blockDim 32 x kWarpRows) or of a block, one after the other.  NV vectors of V
// elements in each thread's registers: vector j of a thread starts at column V (t + j threads).
// (8192 x 4096 bf16 + residual into e4m3 with a scale for 128 columns: a block for every row, its loads at its
// start, 58 us; the next row's loads in registers, 64 us, for the blocks that those leave on an SM.)
template <typename T, int OUT, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kRowThreads : 32 * kWarpRows, BLOCK && NV > 2 ? 1 : 2)
    kda_rms_norm_kernel(const NormArgs a) {
    constexpr int S = ahead(NV, BLOCK);
    __shared__ float s_sum[2][32];
    __shared__ float s_max[2][32];
    extern __shared__ __align__(16) uint8_t s_ring[];
    const int nt = BLOCK ? blockDim.x : 32;
    const int t = BLOCK ? threadIdx.x : (threadIdx.x & 31);
    const int64_t step = BLOCK ? gridDim.x : static_cast<int64_t>(gridDim.x) * kWarpRows;
    int64_t row = BLOCK ? static_cast<int64_t>(blockIdx.x)
                        : static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5);
    const T* const xs = static_cast<const T*>(a.x);
    const T* const rs = static_cast<const T*>(a.residual);
    Ring<T, V, NV, 2, S> ring;
    ring.start(s_ring);
    auto fetch = [&](int64_t r, int slot) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            const bool in = r < a.rows && c < a.dim;
            ring.fetch(slot, 0, j, xs + r * a.dim + c, in);
            if (rs) ring.fetch(slot, 1, j, rs + r * a.dim + c, in);
        }
        ring.commit();
    };
    if constexpr (ring.ON) {
        for (int i = 0; i < S; ++i) fetch(row + i * step, i);
    }
    constexpr bool KEEP = NV <= 2;  // the weights stay in registers
    float w[KEEP ? NV : 1][V];
    if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (V * (t + j * nt) < a.dim) load_weight<V>(a.weight, V * (t + j * nt), w[j]);
    }
    const float inv_dim = 1.f / static_cast<float>(a.dim);
    int slot = 0;
    for (int par = 0; row < a.rows; row += step, par ^= 1, slot = slot + 1 == S ? 0 : slot + 1) {
        Vec<T, V> xr[NV], rr[NV];
        if constexpr (ring.ON) ring.wait();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c >= a.dim) continue;
            if constexpr (ring.ON) {
                xr[j] = ring.get(slot, 0, j);
                if (rs) rr[j] = ring.get(slot, 1, j);
            } else {
                xr[j] = load_raw<T, V>(xs + row * a.dim + c);
                if (rs) rr[j] = load_raw<T, V>(rs + row * a.dim + c);
            }
        }
        const int64_t base = row * a.dim;
        float h[NV][V];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c < a.dim) {
                if (rs) xr[j] = add_vec<T, V>(xr[j], rr[j]);
                if (a.residual_out) *reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.residual_out) + base + c) = xr[j];
                widen<T, V>(xr[j], h[j]);  // the norm is that of the stored row
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) h[j][i] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(h[j][i], h[j][i], ss);
        const float r = rsqrtf(row_sum<BLOCK>(ss * inv_dim, s_sum[par]) + a.eps);
        if constexpr (ring.ON) fetch(row + S * step, slot);
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c >= a.dim) continue;  // h there is 0 already
            if constexpr (!KEEP) load_weight<V>(a.weight, c, w[0]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h[j][i] = h[j][i] * r * w[KEEP ? j : 0][i];
                if (OUT && a.group == 0) mx = max_abs(mx, h[j][i]);
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
                const float s = scale_of<OUT>(row_max<BLOCK>(mx, s_max[par])), inv = __frcp_rn(s);
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
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) m = max_abs(m, h[j][i]);
#pragma unroll
                    for (int off = LG / 2; off > 0; off >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, off));
                    if (c < a.dim) {
                        const float s = scale_of<OUT>(m), inv = __frcp_rn(s);
                        if ((c & 127) == 0) a.scales[g0 + (c >> 7)] = s;
                        store_codes<OUT, V>(y + c, h[j], inv);
                    }
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
    __shared__ float s_max[32];
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
            float mx = 0.f;
            for (int c = V * t; c < a.dim; c += V * nt) {
                float f[V], w[V];
                load_h(c, f);
                load_weight<V>(a.weight, c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) mx = max_abs(mx, f[i] * r * w[i]);
            }
            const float s = scale_of<OUT>(row_max<true>(mx, s_max));
            inv = __frcp_rn(s);
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
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) m = max_abs(m, f[i]);
#pragma unroll
                    for (int off = LG / 2; off > 0; off >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, off));
                    const float s = scale_of<OUT>(m);
                    gi = __frcp_rn(s);
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
        if (lane == 0) part[threadIdx.x >> 5] = make_float2(x, y);
        __syncthreads();
        const float2 p = lane < nw ? part[lane] : make_float2(0.f, 0.f);
        x = warp_sum(p.x);
        y = warp_sum(p.y);
    }
    return make_float2(x, y);
}

template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kRowThreads : 32 * kWarpRows, BLOCK && NV > 1 ? 1 : 2)
    kda_rms_norm_backward_kernel(const NormBackwardArgs a) {
    constexpr int S = ahead(NV + 1, BLOCK);
    grid_dependents();  // the weight's kernel
    __shared__ float2 s_sum[2][32];
    extern __shared__ __align__(16) uint8_t s_ring[];  // and, after the last row, the warps' shares of grad_w [dim]
    float* const s_w = reinterpret_cast<float*>(s_ring);
    const int nt = BLOCK ? blockDim.x : 32;
    const int t = BLOCK ? threadIdx.x : (threadIdx.x & 31);
    const int warp = threadIdx.x >> 5;
    const int64_t step = BLOCK ? gridDim.x : static_cast<int64_t>(gridDim.x) * kWarpRows;
    const T* gy = static_cast<const T*>(a.grad_y);
    const T* hh = static_cast<const T*>(a.h);
    const T* gh = static_cast<const T*>(a.grad_h);
    const float inv_dim = 1.f / static_cast<float>(a.dim);
    int64_t row = BLOCK ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(blockIdx.x) * kWarpRows + warp;
    Ring<T, V, NV, 3, S> ring;
    ring.start(s_ring);
    auto fetch = [&](int64_t r, int slot) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            const bool in = r < a.rows && c < a.dim;
            ring.fetch(slot, 0, j, hh + r * a.dim + c, in);
            ring.fetch(slot, 1, j, gy + r * a.dim + c, in);
            if (gh) ring.fetch(slot, 2, j, gh + r * a.dim + c, in);
        }
        ring.commit();
    };
    if constexpr (ring.ON) {
        for (int i = 0; i < S; ++i) fetch(row + i * step, i);
    }
    constexpr bool KEEP = NV <= 2;  // the weights stay in registers
    float w[KEEP ? NV : 1][V], dw[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = 0.f;
        if (KEEP && V * (t + j * nt) < a.dim) load_weight<V>(a.weight, V * (t + j * nt), w[KEEP ? j : 0]);
    }
    int slot = 0;
    for (int par = 0; row < a.rows; row += step, par ^= 1, slot = slot + 1 == S ? 0 : slot + 1) {
        const int64_t base = row * a.dim;
        Vec<T, V> hv[NV], yv[NV], gv[NV];
        float ss = 0.f, sd = 0.f;
        if constexpr (ring.ON) ring.wait();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c >= a.dim) continue;
            if constexpr (ring.ON) {
                hv[j] = ring.get(slot, 0, j);
                yv[j] = ring.get(slot, 1, j);
                if (gh) gv[j] = ring.get(slot, 2, j);
            } else {
                hv[j] = load_raw<T, V>(hh + base + c);
                yv[j] = load_raw<T, V>(gy + base + c);
                if (gh) gv[j] = load_raw<T, V>(gh + base + c);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c >= a.dim) continue;
            float h[V], y[V];
            widen<T, V>(hv[j], h);
            widen<T, V>(yv[j], y);
            if constexpr (!KEEP) load_weight<V>(a.weight, c, w[0]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ss = fmaf(h[i], h[i], ss);
                sd = fmaf(h[i] * w[KEEP ? j : 0][i], y[i], sd);
            }
        }
        const float2 s = row_sum2<BLOCK>(ss * inv_dim, sd * inv_dim, s_sum[par]);
        const float r = rsqrtf(s.x + a.eps);
        const float m = s.y * r * r * r;
        if constexpr (ring.ON) fetch(row + S * step, slot);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = V * (t + j * nt);
            if (c >= a.dim) continue;
            float h[V], y[V], dx[V];
            widen<T, V>(hv[j], h);
            widen<T, V>(yv[j], y);
            if (gh) {
                widen<T, V>(gv[j], dx);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) dx[i] = 0.f;
            }
            if constexpr (!KEEP) load_weight<V>(a.weight, c, w[0]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] *= r;
                dx[i] = fmaf(w[KEEP ? j : 0][i], y[i], fmaf(-m, h[i], dx[i]));
                dw[j][i] = fmaf(y[i], h[i], dw[j][i]);
            }
            store_vec<T, V>(static_cast<T*>(a.grad_x) + base + c, dx);
        }
    }
    if (!a.grad_weight) return;
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
    if constexpr (ring.ON && !BLOCK) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // every warp is done with its slots
    }
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
    __shared__ float2 s_sum[2][32];
    const int nt = blockDim.x, t = threadIdx.x;
    const T* gy = static_cast<const T*>(a.grad_y);
    const T* hh = static_cast<const T*>(a.h);
    const T* gh = static_cast<const T*>(a.grad_h);
    const float inv_dim = 1.f / static_cast<float>(a.dim);
    float* part = a.grad_weight ? a.partial + static_cast<int64_t>(blockIdx.x) * a.dim : nullptr;
    bool first = true;
    int par = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false, par ^= 1) {
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
        const float2 s = row_sum2<true>(ss * inv_dim, sd * inv_dim, s_sum[par]);
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
    grid_wait();  // the shares
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

// Blocks walk over the rows: as many as are resident at once, at most one for every row (or kWarpRows rows).
template <typename T, int OUT, int V, int NV, bool BLOCK>
cudaError_t norm_launch(const NormArgs& a, int threads, cudaStream_t stream) {
    const uint32_t smem = Ring<T, V, NV, 2, ahead(NV, BLOCK)>::bytes(threads);
    static int configured[64];
    cudaError_t err = set_smem(kda_rms_norm_kernel<T, OUT, V, NV, BLOCK>,
                               Ring<T, V, NV, 2, ahead(NV, BLOCK)>::bytes(BLOCK ? kRowThreads : 32 * kWarpRows), configured);
    if (err != cudaSuccess) return err;
    static int per_sm[kRowThreads / 32 + 1];  // this kernel's resident blocks on an SM, by the warps of a block
    int& n = per_sm[threads / 32];
    if (n == 0) {
        int b = 0;
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kda_rms_norm_kernel<T, OUT, V, NV, BLOCK>, threads, smem);
        if (err != cudaSuccess) return err;
        n = std::max(1, b);
    }
    const int64_t need = BLOCK ? a.rows : (a.rows + kWarpRows - 1) / kWarpRows;
    const int64_t blocks = std::min<int64_t>(need, static_cast<int64_t>(std::max(1, device_sm_count())) * n);
    kda_rms_norm_kernel<T, OUT, V, NV, BLOCK><<<static_cast<unsigned>(blocks), threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int OUT, int V>
cudaError_t norm_v(const NormArgs& a, cudaStream_t stream) {
    const int nvec = a.dim / V;
    // a warp's registers hold the row, or a block's
    if (nvec <= 32) return norm_launch<T, OUT, V, 1, false>(a, 32 * kWarpRows, stream);
    if (nvec <= 64) return norm_launch<T, OUT, V, 2, false>(a, 32 * kWarpRows, stream);
    if (nvec <= 128) return norm_launch<T, OUT, V, 4, false>(a, 32 * kWarpRows, stream);
    if (nvec <= 2 * kRowThreads) return norm_launch<T, OUT, V, 2, true>(a, ((nvec + 1) / 2 + 31) / 32 * 32, stream);
    if (nvec <= 4 * kRowThreads) return norm_launch<T, OUT, V, 4, true>(a, ((nvec + 3) / 4 + 31) / 32 * 32, stream);
    kda_rms_norm_long_kernel<T, OUT, V><<<static_cast<unsigned>(a.rows), kMaxThreads, 0, stream>>>(a);
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

template <typename T, int V, int NV, bool BLOCK>
cudaError_t norm_backward_launch(const NormBackwardArgs& a, unsigned blocks, int threads, cudaStream_t stream) {
    using R = Ring<T, V, NV, 3, ahead(NV + 1, BLOCK)>;
    static int configured[64];
    const cudaError_t err =
        set_smem(kda_rms_norm_backward_kernel<T, V, NV, BLOCK>, R::bytes(BLOCK ? kRowThreads : 32 * kWarpRows), configured);
    if (err != cudaSuccess) return err;
    // the warps' shares of grad_w want at most 4 KB, which the slots have where there are any
    const uint32_t smem = R::ON || BLOCK || !a.grad_weight ? R::bytes(threads) : static_cast<uint32_t>(a.dim) * 4;
    kda_rms_norm_backward_kernel<T, V, NV, BLOCK><<<blocks, threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t norm_backward_v(const NormBackwardArgs& a, unsigned blocks, cudaStream_t stream) {
    const int nvec = a.dim / V;
    if (nvec <= 32) return norm_backward_launch<T, V, 1, false>(a, blocks, 32 * kWarpRows, stream);
    if (nvec <= 64) return norm_backward_launch<T, V, 2, false>(a, blocks, 32 * kWarpRows, stream);
    if (nvec <= 128) return norm_backward_launch<T, V, 4, false>(a, blocks, 32 * kWarpRows, stream);
    if (nvec <= kRowThreads) return norm_backward_launch<T, V, 1, true>(a, blocks, (nvec + 31) / 32 * 32, stream);
    if (nvec <= 2 * kRowThreads)
        return norm_backward_launch<T, V, 2, true>(a, blocks, ((nvec + 1) / 2 + 31) / 32 * 32, stream);
    kda_rms_norm_backward_long_kernel<T, V><<<blocks, kMaxThreads, 0, stream>>>(a);
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

// Two blocks an SM (of 152): what the registers of 512 threads leave, and few enough shares of grad_w.
int64_t rms_norm_backward_partials(int64_t rows) { return std::min<int64_t>(rows, 304); }

cudaError_t launch_rms_norm_backward(bool f32_io, const NormBackwardArgs& a, cudaStream_t stream) {
    const int64_t parts = rms_norm_backward_partials(a.rows);
    cudaError_t err = cudaSuccess;
    if (parts > 0) {
        const unsigned blocks = static_cast<unsigned>(parts);
        err = f32_io ? norm_backward_t<float>(a, blocks, stream) : norm_backward_t<__nv_bfloat16>(a, blocks, stream);
    }
    if (err != cudaSuccess || !a.grad_weight) return err;
    return launch_dependent(kda_rms_norm_weight_kernel, (a.dim + 31) / 32, 1024, 0, stream, a.partial, parts, a.dim,
                            a.grad_weight);
}

}  // namespace kda
