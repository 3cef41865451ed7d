// kda_gdn_recurrent.cu -- the gated delta rule token by token, in fp32: the decode
// step, the prefill of short sequences and of fp32 inputs, and the gradient of a
// few tokens.
//
// The gated delta rule is the recurrence of "Understanding Kimi Delta Attention"
// (pyshine), "The KDA Recurrence: Scalar Gate vs Channel-wise Gate", with its
// scalar gate: one decay a_t = exp(log_decay_t) per (token, value head),
//   S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   o_t = S_t^T q_t,
// evaluated in one pass over the state:
//   y = a S^T k,  p = a S^T q,  u = b (v - y),  S <- a S + k u^T,  o = p + (k . q) u.
// Value head h reads q/k head h / (Hv / Hk).
#include <cuda_bf16.h>

#include "kda_gdn_internal.h"
#include "kda_gdn_ptx.cuh"

namespace kda {
namespace {

constexpr int D = kHeadDim;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void st_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void st_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}

// ================================================================ decode ==
// One CTA per (sequence, value head); the 64 KB state passes once through the registers of 256
// threads: thread (warp w, lane l) holds rows 16w..16w+15 of columns 4l..4l+3, so that a warp reads
// and writes whole 512-byte rows.  Bound by HBM: 256 sequences x 32 heads 160 us, 6.7 TB/s.
constexpr int kDecThreads = 256;
constexpr int kDecRows = D / (kDecThreads / 32);  // rows of a warp

template <typename IoT>
__global__ void __launch_bounds__(kDecThreads, 2)
    kda_gdn_decode_kernel(const IoT* __restrict__ q, const IoT* __restrict__ k, const IoT* __restrict__ v,
                          const float* __restrict__ log_decay, const float* __restrict__ beta, float* S,
                          int32_t num_slots, const int32_t* __restrict__ state_indices, int32_t Hk, int32_t Hv,
                          IoT* __restrict__ o, int32_t* device_status) {
    const int n = blockIdx.x / Hv, h = blockIdx.x - n * Hv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t slot = state_indices ? state_indices[n] : n;
    if (slot < 0 || slot >= num_slots) {
        if (tid == 0 && device_status) atomicOr(device_status, KDA_DEV_BAD_SLOT);
        return;
    }
    __shared__ __align__(16) float k_s[D], q_s[D], u_s[D];
    __shared__ __align__(16) float red_y[kDecThreads / 32][D], red_p[kDecThreads / 32][D];
    __shared__ float kq_s;

    float* const Sg = S + (static_cast<size_t>(slot) * Hv + h) * D * D + static_cast<size_t>(warp) * kDecRows * D;
    float4 s[kDecRows];  // the whole state in flight before anything is waited for
#pragma unroll
    for (int i = 0; i < kDecRows; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(Sg + i * D) + lane);

    const size_t tok = static_cast<size_t>(n) * Hv + h;
    const size_t qk = (static_cast<size_t>(n) * Hk + h / (Hv / Hk)) * D;
    float vv = 0.f, b = 0.f;
    if (tid < D) {
        k_s[tid] = to_f32(k[qk + tid]);
        q_s[tid] = to_f32(q[qk + tid]);
        vv = to_f32(v[tok * D + tid]);
        b = beta[tok];
    }
    const float a = expf(log_decay[tok]);
    __syncthreads();
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f), p = y;
#pragma unroll
    for (int i = 0; i < kDecRows; ++i) {
        const float kr = k_s[warp * kDecRows + i], qr = q_s[warp * kDecRows + i];
        s[i].x *= a; s[i].y *= a; s[i].z *= a; s[i].w *= a;
        y.x = fmaf(kr, s[i].x, y.x); y.y = fmaf(kr, s[i].y, y.y);
        y.z = fmaf(kr, s[i].z, y.z); y.w = fmaf(kr, s[i].w, y.w);
        p.x = fmaf(qr, s[i].x, p.x); p.y = fmaf(qr, s[i].y, p.y);
        p.z = fmaf(qr, s[i].z, p.z); p.w = fmaf(qr, s[i].w, p.w);
    }
    reinterpret_cast<float4*>(red_y[warp])[lane] = y;
    reinterpret_cast<float4*>(red_p[warp])[lane] = p;
    if (warp == 0) {
        const float4 kk = reinterpret_cast<const float4*>(k_s)[lane], qq = reinterpret_cast<const float4*>(q_s)[lane];
        float d = fmaf(kk.x, qq.x, fmaf(kk.y, qq.y, fmaf(kk.z, qq.z, kk.w * qq.w)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        if (lane == 0) kq_s = d;
    }
    __syncthreads();
    if (tid < D) {
        float yy = 0.f, pp = 0.f;
#pragma unroll
        for (int w = 0; w < kDecThreads / 32; ++w) {
            yy += red_y[w][tid];
            pp += red_p[w][tid];
        }
        const float u = b * (vv - yy);
        u_s[tid] = u;
        st_f32(o + tok * D + tid, fmaf(kq_s, u, pp));
    }
    __syncthreads();
    const float4 uu = reinterpret_cast<const float4*>(u_s)[lane];
#pragma unroll
    for (int i = 0; i < kDecRows; ++i) {
        const float kr = k_s[warp * kDecRows + i];
        float4 t = s[i];
        t.x = fmaf(kr, uu.x, t.x); t.y = fmaf(kr, uu.y, t.y);
        t.z = fmaf(kr, uu.z, t.z); t.w = fmaf(kr, uu.w, t.w);
        __stcs(reinterpret_cast<float4*>(Sg + i * D) + lane, t);
    }
}

// =============================================================== prefill ==
// The state's columns never mix, so a CTA takes 16 of them for one (sequence, value head): 8 lanes
// hold a column, 16 rows each (rows 4 (8 i + part) .. + 3, i = 0..3, so that the 8 lanes of a column
// read 128 consecutive bytes of a k or q row, and the warp's other columns the same ones).  A token
// is a chain of multiply-adds, three shuffles and the update, with no barrier; the rows of kTB tokens
// are staged at a time, with their k . q, the next ones in flight meanwhile.  Bound by instructions
// issued, so the arithmetic is on pairs of floats (512 fp32 tokens x 32 heads: 158 us with single
// ones and k . q in every lane, 163 instructions a token and warp; 8192 x 32 heads now 2.57 ms, 0.31 us a token).
constexpr int kTB = 16;          // tokens staged at a time
constexpr int kRecThreads = 128;
constexpr int kRecCols = 16;     // state columns of a CTA

// Two floats in a 64-bit register.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float sum_pair(uint64_t p) {
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
    return x + y;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <typename IoT>
__global__ void __launch_bounds__(kRecThreads) kda_gdn_recurrent_kernel(const GdnArgs a) {
    __shared__ __align__(16) float k_s[2][kTB][D], q_s[2][kTB][D], v_s[2][kTB][kRecCols];
    __shared__ float4 g_s[2][kTB];  // decay, beta, k . q
    const int tid = threadIdx.x, part = tid & 7, col = tid >> 3;
    constexpr int NSL = D / kRecCols;
    const int slice = blockIdx.x % NSL;
    const int h = (blockIdx.x / NSL) % a.Hv;
    const int n = blockIdx.x / (NSL * a.Hv);
    const int hk = h / (a.Hv / a.Hk);
    const int j0 = slice * kRecCols;
    const int64_t t_begin = a.cu_seqlens[n], t_end = a.cu_seqlens[n + 1];
    const bool ends_ok = a.cu_seqlens[0] == 0 && a.cu_seqlens[a.num_seqs] == a.total_tokens;
    const bool ok = t_begin >= 0 && t_end >= t_begin && t_end <= a.total_tokens;
    if ((!ok || !ends_ok) && tid == 0 && a.device_status) atomicOr(a.device_status, KDA_DEV_BAD_CU_SEQLENS);
    if (!ok) return;
    const IoT* const q = static_cast<const IoT*>(a.q);
    const IoT* const k = static_cast<const IoT*>(a.k);
    const IoT* const v = static_cast<const IoT*>(a.v);

    uint64_t S[8];  // rows 4 (8 (i / 2) + part) + 2 (i % 2) and the next
    const size_t st = ((static_cast<size_t>(n) * a.Hv + h) * D) * D + j0 + col;
    auto row_of = [&](int i) { return static_cast<size_t>(4 * (8 * (i >> 1) + part) + 2 * (i & 1)); };
#pragma unroll
    for (int i = 0; i < 8; ++i)
        S[i] = a.S0 ? pair(a.S0[st + row_of(i) * D], a.S0[st + (row_of(i) + 1) * D]) : 0ull;

    // this thread's share of a batch of rows: four quads of k and of q, two values of v, one gate
    float4 kr[4], qr[4];
    float vr[2], ar = 0.f, br = 0.f;
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = (tid + e * kRecThreads) >> 5, c = 4 * (tid & 31);
            kr[e] = qr[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t0 + r < t_end) {
                const size_t off = (static_cast<size_t>(t0 + r) * a.Hk + hk) * D + c;
                kr[e] = ld4(k + off);
                qr[e] = ld4(q + off);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = (tid + e * kRecThreads) >> 4, c = tid & 15;
            vr[e] = t0 + r < t_end ? to_f32(v[(static_cast<size_t>(t0 + r) * a.Hv + h) * D + j0 + c]) : 0.f;
        }
        if (tid < kTB && t0 + tid < t_end) {
            ar = a.log_decay[(t0 + tid) * a.Hv + h];
            br = a.beta[(t0 + tid) * a.Hv + h];
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = (tid + e * kRecThreads) >> 5, c = 4 * (tid & 31);
            *reinterpret_cast<float4*>(&k_s[buf][r][c]) = kr[e];
            *reinterpret_cast<float4*>(&q_s[buf][r][c]) = qr[e];
            float kq = fmaf(kr[e].x, qr[e].x, fmaf(kr[e].y, qr[e].y, fmaf(kr[e].z, qr[e].z, kr[e].w * qr[e].w)));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, off);
            if (c == 0) g_s[buf][r].z = kq;  // a warp holds whole rows
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) v_s[buf][(tid + e * kRecThreads) >> 4][tid & 15] = vr[e];
        if (tid < kTB) {
            g_s[buf][tid].x = expf(ar);
            g_s[buf][tid].y = br;
        }
    };
    if (t_begin < t_end) fetch(t_begin);
    int buf = 0;
    for (int64_t t0 = t_begin; t0 < t_end; t0 += kTB, buf ^= 1) {
        stage(buf);
        __syncthreads();  // the other buffer's readers are past it too
        if (t0 + kTB < t_end) fetch(t0 + kTB);
        const int nt = static_cast<int>(t_end - t0 < kTB ? t_end - t0 : kTB);
#pragma unroll 2
        for (int t = 0; t < nt; ++t) {
            uint64_t kk[8], y[2] = {0ull, 0ull}, p[2] = {0ull, 0ull};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&k_s[buf][t][4 * (8 * i + part)]);
                const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(&q_s[buf][t][4 * (8 * i + part)]);
                kk[2 * i] = k2.x;
                kk[2 * i + 1] = k2.y;
                y[0] = fma2(k2.x, S[2 * i], y[0]);
                y[1] = fma2(k2.y, S[2 * i + 1], y[1]);
                p[0] = fma2(q2.x, S[2 * i], p[0]);
                p[1] = fma2(q2.y, S[2 * i + 1], p[1]);
            }
            const float4 gv = g_s[buf][t];
            const float vv = v_s[buf][t][col];
            const uint64_t al = pair(gv.x, gv.x);
            float ys = sum_pair(add2(y[0], y[1])), ps = sum_pair(add2(p[0], p[1]));
#pragma unroll
            for (int i = 0; i < 8; ++i) S[i] = mul2(al, S[i]);
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) {
                ys += __shfl_xor_sync(0xffffffffu, ys, off);
                ps += __shfl_xor_sync(0xffffffffu, ps, off);
            }
            const float u = gv.y * (vv - gv.x * ys);
            const uint64_t uu = pair(u, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) S[i] = fma2(kk[i], uu, S[i]);
            if (part == 0)
                st_f32(static_cast<IoT*>(a.o) + (static_cast<size_t>(t0 + t) * a.Hv + h) * D + j0 + col,
                       fmaf(gv.z, u, gv.x * ps));
        }
    }
    if (a.S_final) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x, y;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(S[i]));
            a.S_final[st + row_of(i) * D] = x;
            a.S_final[st + (row_of(i) + 1) * D] = y;
        }
    }
}

// ============================================================== gradient ==
// The gradient of short sequences, token by token in fp32: a CTA per (sequence, value head), and where groups share a
// q/k head a kernel that adds them up.  A walk forward leaves the state before every token in the workspace, the
// walk back takes them: with G the adjoint of the state after a token, S' = a S its decayed state, y = S'^T k, u = b (v - y), z = -b G^T k,
//   G += q dO^T;  dq = S' dO + k (u . dO);  dv = b G^T k;  db = (G^T k) . (v - y);  dk = G u + S' z;
//   G' = G + k z^T;  gradient of log_decay = <G', S'>;  the adjoint of the state before = a G'.
// A few tokens leave few numbers to average an error over, and a sum that cancels among them shows every
// rounding: with operands of two bf16 terms single gradients of log_decay and b were off by 1e-5 to 1e-4 of themselves.
// Thread (warp w, lane l) holds rows 16 w .. and columns 4 l .. + 3 of S' and of G.  Bound by the chain of a token's
// reductions, 3.5 us both ways.
constexpr int kGradThreads = 256;
constexpr int kGradRows = D / (kGradThreads / 32);  // rows of a warp: 16

// x[0 .. 15] of 32 lanes: lane l gets the sum over the lanes of x[l / 2].
__device__ __forceinline__ float sum_rows(float (&x)[kGradRows], int lane) {
#pragma unroll
    for (int n = 8, off = 16; n > 0; n >>= 1, off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? x[i + n] : x[i], give = up ? x[i] : x[i + n];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}
// The sum over the block of x (every thread's), for every thread; `part` is one of a kind until the block's next barrier.
__device__ __forceinline__ float block_sum(float x, float* part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < kGradThreads / 32; ++w) x += part[w];
    return x;
}

__global__ void __launch_bounds__(kGradThreads, 1)
    kda_gdn_recurrent_grad_kernel(const GdnArgs a, const GdnBackwardArgs gr, float* __restrict__ states,
                                  float* __restrict__ sums) {
    __shared__ __align__(16) float k_s[D], q_s[D], v_s[D], do_s[D], u_s[D], z_s[D];
    __shared__ __align__(16) float red[2][kGradThreads / 32][D];
    __shared__ float part[3][kGradThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv, group = a.Hv / a.Hk, hk = h / group;
    grid_dependents();  // the groups' sums
    const int64_t t_begin = a.cu_seqlens[n], t_end = a.cu_seqlens[n + 1];
    const bool ends_ok = a.cu_seqlens[0] == 0 && a.cu_seqlens[a.num_seqs] == a.total_tokens;
    const bool ok = t_begin >= 0 && t_end >= t_begin && t_end <= a.total_tokens;
    if ((!ok || !ends_ok) && tid == 0 && a.device_status) atomicOr(a.device_status, KDA_DEV_BAD_CU_SEQLENS);
    if (!ok) return;
    const auto bf16 = [](const void* p) { return static_cast<const __nv_bfloat16*>(p); };
    const int r0 = kGradRows * warp;
    const size_t state = (static_cast<size_t>(n) * a.Hv + h) * D * D + static_cast<size_t>(r0) * D;
    // this thread's places in the state before token t
    auto saved = [&](int64_t t) {
        return reinterpret_cast<float4*>(states + ((static_cast<size_t>(t) * a.Hv + h) * D + r0) * D) + lane;
    };
    float4 S[kGradRows], G[kGradRows];
#pragma unroll
    for (int i = 0; i < kGradRows; ++i)
        S[i] = a.S0 ? reinterpret_cast<const float4*>(a.S0 + state + i * D)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    // a token's rows into shared memory; the barrier also ends the reads of the one before
    auto stage = [&](int64_t t) {
        __syncthreads();
        const size_t qk = (static_cast<size_t>(t) * a.Hk + hk) * D, v = (static_cast<size_t>(t) * a.Hv + h) * D;
        if (tid < D) {
            k_s[tid] = to_f32(bf16(a.k)[qk + tid]);
            q_s[tid] = to_f32(bf16(a.q)[qk + tid]);
        } else {
            v_s[tid - D] = to_f32(bf16(a.v)[v + tid - D]);
            do_s[tid - D] = to_f32(bf16(gr.grad_o)[v + tid - D]);
        }
        __syncthreads();
    };
    auto column = [&](float (*r)[D], int c) {  // over the warps
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kGradThreads / 32; ++w) x += r[w][c];
        return x;
    };
    for (int64_t t = t_begin; t < t_end; ++t) {
        stage(t);
        const float al = expf(a.log_decay[t * a.Hv + h]), b = a.beta[t * a.Hv + h];
        float4* const to = saved(t);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            to[i * (D / 4)] = S[i];
            const float kr = k_s[r0 + i];
            S[i].x *= al; S[i].y *= al; S[i].z *= al; S[i].w *= al;
            y.x = fmaf(kr, S[i].x, y.x); y.y = fmaf(kr, S[i].y, y.y);
            y.z = fmaf(kr, S[i].z, y.z); y.w = fmaf(kr, S[i].w, y.w);
        }
        reinterpret_cast<float4*>(red[0][warp])[lane] = y;
        __syncthreads();
        if (tid < D) u_s[tid] = b * (v_s[tid] - column(red[0], tid));
        __syncthreads();
        const float4 u = reinterpret_cast<const float4*>(u_s)[lane];
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            const float kr = k_s[r0 + i];
            S[i].x = fmaf(kr, u.x, S[i].x); S[i].y = fmaf(kr, u.y, S[i].y);
            S[i].z = fmaf(kr, u.z, S[i].z); S[i].w = fmaf(kr, u.w, S[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < kGradRows; ++i)
        G[i] = gr.grad_S_final ? reinterpret_cast<const float4*>(gr.grad_S_final + state + i * D)[lane]
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t t = t_end - 1; t >= t_begin; --t) {
        const float4* const from = saved(t);
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) S[i] = from[i * (D / 4)];
        stage(t);
        const float al = expf(a.log_decay[t * a.Hv + h]), b = a.beta[t * a.Hv + h];
        const float4 dO = reinterpret_cast<const float4*>(do_s)[lane];
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f), gk = y;
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            const float kr = k_s[r0 + i], qr = q_s[r0 + i];
            S[i].x *= al; S[i].y *= al; S[i].z *= al; S[i].w *= al;
            G[i].x = fmaf(qr, dO.x, G[i].x); G[i].y = fmaf(qr, dO.y, G[i].y);
            G[i].z = fmaf(qr, dO.z, G[i].z); G[i].w = fmaf(qr, dO.w, G[i].w);
            y.x = fmaf(kr, S[i].x, y.x); y.y = fmaf(kr, S[i].y, y.y);
            y.z = fmaf(kr, S[i].z, y.z); y.w = fmaf(kr, S[i].w, y.w);
            gk.x = fmaf(kr, G[i].x, gk.x); gk.y = fmaf(kr, G[i].y, gk.y);
            gk.z = fmaf(kr, G[i].z, gk.z); gk.w = fmaf(kr, G[i].w, gk.w);
        }
        reinterpret_cast<float4*>(red[0][warp])[lane] = y;
        reinterpret_cast<float4*>(red[1][warp])[lane] = gk;
        __syncthreads();
        float db = 0.f, ud = 0.f;
        if (tid < D) {
            const float e = v_s[tid] - column(red[0], tid), g = column(red[1], tid), u = b * e;
            u_s[tid] = u;
            z_s[tid] = -b * g;
            db = g * e;
            ud = u * do_s[tid];
            static_cast<__nv_bfloat16*>(gr.grad_v)[(static_cast<size_t>(t) * a.Hv + h) * D + tid] =
                __float2bfloat16_rn(b * g);
        }
        db = block_sum(db, part[0]);
        ud = block_sum(ud, part[1]);
        const float4 u = reinterpret_cast<const float4*>(u_s)[lane], z = reinterpret_cast<const float4*>(z_s)[lane];
        float rq[kGradRows], rk[kGradRows], ld = 0.f;
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            rq[i] = fmaf(S[i].x, dO.x, fmaf(S[i].y, dO.y, fmaf(S[i].z, dO.z, S[i].w * dO.w)));
            rk[i] = fmaf(S[i].x, z.x, fmaf(S[i].y, z.y, fmaf(S[i].z, z.z, S[i].w * z.w)));
            rk[i] = fmaf(G[i].x, u.x, fmaf(G[i].y, u.y, fmaf(G[i].z, u.z, fmaf(G[i].w, u.w, rk[i]))));
            const float kr = k_s[r0 + i];
            G[i].x = fmaf(kr, z.x, G[i].x); G[i].y = fmaf(kr, z.y, G[i].y);
            G[i].z = fmaf(kr, z.z, G[i].z); G[i].w = fmaf(kr, z.w, G[i].w);
            ld = fmaf(G[i].x, S[i].x, fmaf(G[i].y, S[i].y, fmaf(G[i].z, S[i].z, fmaf(G[i].w, S[i].w, ld))));
            G[i].x *= al; G[i].y *= al; G[i].z *= al; G[i].w *= al;
        }
        const int row = r0 + (lane >> 1);
        const float dq = fmaf(k_s[row], ud, sum_rows(rq, lane)), dk = sum_rows(rk, lane);
        if (!(lane & 1)) {
            if (group == 1) {
                const size_t at = (static_cast<size_t>(t) * a.Hk + hk) * D + row;
                static_cast<__nv_bfloat16*>(gr.grad_q)[at] = __float2bfloat16_rn(dq);
                static_cast<__nv_bfloat16*>(gr.grad_k)[at] = __float2bfloat16_rn(dk);
            } else {
                float* const at = sums + (static_cast<size_t>(t) * a.Hv + h) * 2 * D + row;
                at[0] = dq;
                at[D] = dk;
            }
        }
        ld = block_sum(ld, part[2]);
        if (tid == 0) {
            gr.grad_log_decay[t * a.Hv + h] = ld;
            gr.grad_beta[t * a.Hv + h] = db;
        }
    }
    if (gr.grad_S0) {
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) reinterpret_cast<float4*>(gr.grad_S0 + state + i * D)[lane] = G[i];
    }
}

// dq and dk of a token's q/k head: its value heads' added up in order, rounded once.
__global__ void __launch_bounds__(2 * D)
    kda_gdn_group_sum_kernel(const float* __restrict__ sums, int32_t Hk, int32_t group, __nv_bfloat16* __restrict__ grad_q,
                             __nv_bfloat16* __restrict__ grad_k) {
    grid_wait();
    const float* from = sums + static_cast<size_t>(blockIdx.x) * group * 2 * D + threadIdx.x;
    float x = 0.f;
    for (int i = 0; i < group; ++i) x += from[static_cast<size_t>(i) * 2 * D];
    __nv_bfloat16* const to = threadIdx.x < D ? grad_q : grad_k;
    to[static_cast<size_t>(blockIdx.x) * D + threadIdx.x % D] = __float2bfloat16_rn(x);
}

}  // namespace

cudaError_t launch_gdn_decode(bool f32_io, const void* q, const void* k, const void* v, const float* log_decay,
                              const float* beta, float* S, int32_t num_slots, const int32_t* state_indices, int32_t N,
                              int32_t Hk, int32_t Hv, void* o, int32_t* device_status, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(N) * Hv;
    if (units == 0) return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>(units);
    if (f32_io)
        kda_gdn_decode_kernel<float><<<blocks, kDecThreads, 0, stream>>>(
            static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v), log_decay, beta, S,
            num_slots, state_indices, Hk, Hv, static_cast<float*>(o), device_status);
    else
        kda_gdn_decode_kernel<__nv_bfloat16><<<blocks, kDecThreads, 0, stream>>>(
            static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
            static_cast<const __nv_bfloat16*>(v), log_decay, beta, S, num_slots, state_indices, Hk, Hv,
            static_cast<__nv_bfloat16*>(o), device_status);
    return cudaGetLastError();
}

cudaError_t launch_gdn_recurrent(bool f32_io, const GdnArgs& a, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(a.num_seqs) * a.Hv * (D / kRecCols);
    if (units == 0) return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>(units);
    if (f32_io) kda_gdn_recurrent_kernel<float><<<blocks, kRecThreads, 0, stream>>>(a);
    else kda_gdn_recurrent_kernel<__nv_bfloat16><<<blocks, kRecThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

size_t gdn_recurrent_backward_workspace(int64_t total_tokens, int32_t Hk, int32_t Hv) {
    const size_t T = static_cast<size_t>(total_tokens);
    return round_up(T * Hv * D * D * 4, kAlign) + round_up(Hv > Hk ? 2 * T * Hv * D * 4 : 0, kAlign) + kAlign;
}

cudaError_t launch_gdn_recurrent_backward(const GdnArgs& a, const GdnBackwardArgs& b, void* workspace, cudaStream_t stream) {
    const int64_t blocks = static_cast<int64_t>(a.num_seqs) * a.Hv;
    if (blocks == 0) return cudaSuccess;
    float* const states = static_cast<float*>(workspace);
    float* const sums = states + round_up(static_cast<size_t>(a.total_tokens) * a.Hv * D * D * 4, kAlign) / 4;
    kda_gdn_recurrent_grad_kernel<<<static_cast<unsigned>(blocks), kGradThreads, 0, stream>>>(a, b, states, sums);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || a.Hv == a.Hk || a.total_tokens == 0) return err;
    return launch_dependent(kda_gdn_group_sum_kernel, a.total_tokens * a.Hk, 2 * D, 0, stream, sums, a.Hk, a.Hv / a.Hk,
                            static_cast<__nv_bfloat16*>(b.grad_q), static_cast<__nv_bfloat16*>(b.grad_k));
}

}  // namespace kda
