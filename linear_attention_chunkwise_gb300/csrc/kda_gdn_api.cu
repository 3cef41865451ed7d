// kda_gdn_api.cu -- the extern "C" entry points of the gated delta rule and of
// the RMS norm: argument validation, workspace carving and kernel launches.
#include <algorithm>
#include <climits>

#include "kda_gdn_internal.h"

using kda::aligned;
using kda::esize_of;
using kda::kAlign;
using kda::kHeadDim;
using kda::overlap;
using kda::Range;
using kda::range_of;
using kda::round_up;
using kda::sizes_ok;

namespace {

constexpr int64_t kStateBytes = static_cast<int64_t>(kHeadDim) * kHeadDim * 4;

// Shapes that every kda_gdn_ entry point takes; `rows` = tokens.
kda_status gdn_shape(kda_dtype t, int64_t rows, int32_t states, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv) {
    if (t != KDA_DTYPE_BF16 && t != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || states < 0 || Hk <= 0 || Hv <= 0 || rows > INT32_MAX - 64) return KDA_ERR_INVALID_ARG;
    if (dk != kHeadDim || dv != kHeadDim) return KDA_ERR_UNSUPPORTED;
    if (Hv % Hk != 0 || (states == 0 && rows > 0)) return KDA_ERR_INVALID_ARG;
    // a launch has one grid dimension: 8 blocks for every (sequence, value head), one for every chunk's
    if (!sizes_ok(rows, Hv, kHeadDim, 4) || !sizes_ok(states, Hv, kStateBytes, 1) ||
        static_cast<double>(states) * Hv * 8.0 > 2147483647.0 ||
        (static_cast<double>(rows) / kda::kChunk + 1.0 + states) * Hv > 2147483647.0)
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

bool qk_maps(const kda::GdnArgs& a, CUtensorMap* tm_q, CUtensorMap* tm_k) {
    return kda::make_tensor_map(tm_q, a.q, a.Hk, a.total_tokens, 64, kda::kChunk, CU_TENSOR_MAP_SWIZZLE_128B) &&
           kda::make_tensor_map(tm_k, a.k, a.Hk, a.total_tokens, 64, kda::kChunk, CU_TENSOR_MAP_SWIZZLE_128B);
}

// fp32 inputs and short sequences go token by token: one of up to 16 tokens (14 us against 17), several of up to 8 on
// average, and up to so many in all that a sequence that has them all to itself, 0.3 us each one after the other, takes no
// more than about two and a half times what chunks take: the host does not know the longest, and empty sequences count in
// num_seqs.  (us token by token and in chunks, tokens spread evenly, and all in one of the sequences:
//   64 sequences x 32 heads,  256 tokens:  134, 176;   155,   96       512:   176,  177;   247, 101 (in chunks)
//   256 x 32,                1024:         510, 614;   592,  306      2048:   677,  616;   988, 323 (in chunks)
//   64 x 4,                   256:          22,  37;    72,   37       512:    28,   36;   133,  49 (in chunks)
//   256 x 4,                  256:          57, 100;   107,   65       512:    62,  101;   186,  66 (in chunks)
// 3000 tokens beside 255 of one: 1493 and 650, in chunks.)
int64_t most_by_token(int64_t N, int32_t Hv) { return N == 1 ? 16 : std::min(8 * N, 240 + N * Hv / 8); }
bool chunked(kda_dtype t, int32_t num_seqs, int64_t total_tokens, int32_t Hv) {
    return t == KDA_DTYPE_BF16 && total_tokens > most_by_token(num_seqs, Hv);
}

// The gradient goes token by token up to two tokens a sequence and six more, and up to so many in all that a sequence that
// has them all to itself, 3.5 us each one after the other, takes no more than about four times what chunks take, since
// chunks take about five times as long where the tokens are spread evenly.  (us token by token and in chunks, even; in one:
//   64 sequences x 32 heads, 64 tokens: 119, 568;  322, 178       134: 179, 571;  642, 184
//   256 x 32,               256:        437, 2119; 1364, 542      518: 645, 2130; 2578, 561 (in chunks)
//   64 x 4,                  64:         25, 114;  221,  64       134:  26, 112;  463,  74 (in chunks)
//   256 x 8,                256:        120, 582;  1081, 187 (in chunks)
// 64 of one and one of 65: 32 heads 383 and 567, 4 heads 253 and 109, in chunks.)
int64_t most_by_token_backward(int64_t N, int32_t Hv) { return std::min(2 * N + 6, 64 + N * Hv / 20); }
bool chunked_backward(int32_t num_seqs, int64_t total_tokens, int32_t Hv) {
    return total_tokens > most_by_token_backward(num_seqs, Hv);
}

// What a call takes of its workspace.
size_t prefill_takes(kda_dtype t, int32_t num_seqs, int64_t total_tokens, int32_t Hv) {
    return chunked(t, num_seqs, total_tokens, Hv) ? kda::gdn_workspace(num_seqs, total_tokens, Hv, false, nullptr, nullptr) : kAlign;
}
size_t backward_takes(int32_t num_seqs, int64_t total_tokens, int32_t Hk, int32_t Hv) {
    return chunked_backward(num_seqs, total_tokens, Hv) ? kda::gdn_workspace(num_seqs, total_tokens, Hv, true, nullptr, nullptr)
                                                        : kda::gdn_recurrent_backward_workspace(total_tokens, Hk, Hv);
}
// The most sequences, up to num_seqs, with which so many tokens go in chunks (most(N) does not fall as N rises); 0 for
// none.  A workspace is to serve every smaller call too, and with fewer sequences the same tokens may go in chunks.
template <typename F>
int32_t most_in_chunks(int32_t num_seqs, int64_t total_tokens, F most) {
    int32_t lo = 0, hi = num_seqs;
    while (lo < hi) {
        const int32_t mid = hi - (hi - lo) / 2;
        if (total_tokens > most(mid)) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace

extern "C" {

size_t kda_gdn_prefill_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs, int64_t total_tokens, int32_t Hk,
                                       int32_t Hv, int32_t dk, int32_t dv) {
    if (gdn_shape(qkv_dtype, total_tokens, num_seqs, Hk, Hv, dk, dv) != KDA_OK) return 0;
    if (qkv_dtype != KDA_DTYPE_BF16) return kAlign;
    const int32_t n = most_in_chunks(num_seqs, total_tokens, [&](int64_t N) { return most_by_token(N, Hv); });
    return n ? prefill_takes(qkv_dtype, n, total_tokens, Hv) : kAlign;
}

kda_status kda_gdn_prefill(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const float* log_decay,
                           const float* beta, const float* S0, const int32_t* cu_seqlens, int32_t num_seqs,
                           int64_t total_tokens, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, void* o,
                           float* S_final, void* workspace, size_t workspace_bytes, int32_t* device_status,
                           kda_stream_t stream) {
    const kda_status shape = gdn_shape(qkv_dtype, total_tokens, num_seqs, Hk, Hv, dk, dv);
    if (shape != KDA_OK) return shape;
    if (!cu_seqlens || !workspace) return KDA_ERR_INVALID_ARG;
    const bool have_tokens = total_tokens > 0;
    if (have_tokens && (!q || !k || !v || !log_decay || !beta || !o)) return KDA_ERR_INVALID_ARG;
    if (have_tokens && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
                        !aligned(log_decay, 4) || !aligned(beta, 4)))
        return KDA_ERR_INVALID_ARG;
    if ((S0 && !aligned(S0, 16)) || (S_final && !aligned(S_final, 16)) || !aligned(workspace, kAlign) ||
        !aligned(cu_seqlens, 4) || (device_status && !aligned(device_status, 4)))
        return KDA_ERR_INVALID_ARG;
    const size_t need = prefill_takes(qkv_dtype, num_seqs, total_tokens, Hv);
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;

    // outputs (and the workspace) overlap nothing; S_final may be S0 exactly
    const size_t es = esize_of(qkv_dtype), T = static_cast<size_t>(total_tokens);
    const size_t nst = static_cast<size_t>(num_seqs) * Hv * kStateBytes;
    const Range outs[] = {range_of(o, T * Hv * kHeadDim * es), range_of(S_final, S_final ? nst : 0),
                          range_of(workspace, need), range_of(device_status, device_status ? 4 : 0)};
    const Range ins[] = {range_of(q, T * Hk * kHeadDim * es), range_of(k, T * Hk * kHeadDim * es),
                         range_of(v, T * Hv * kHeadDim * es), range_of(log_decay, T * Hv * 4),
                         range_of(beta, T * Hv * 4),          range_of(S0, S0 && S0 != S_final ? nst : 0),
                         range_of(cu_seqlens, (static_cast<size_t>(num_seqs) + 1) * 4)};
    for (int i = 0; i < 4; ++i) {
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
        for (const Range& in : ins)
            if (overlap(outs[i], in)) return KDA_ERR_INVALID_ARG;
    }
    const kda_status dev = kda::device_check();
    if (dev != KDA_OK) return dev;

    kda::GdnArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.beta = beta;
    a.S0 = S0;
    a.cu_seqlens = cu_seqlens;
    a.o = o;
    a.S_final = S_final;
    a.device_status = device_status;
    a.total_tokens = total_tokens;
    a.num_seqs = num_seqs;
    a.Hk = Hk;
    a.Hv = Hv;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (chunked(qkv_dtype, num_seqs, total_tokens, Hv)) {
        kda::GdnWorkspace w;
        kda::gdn_workspace(num_seqs, total_tokens, Hv, false, static_cast<uint8_t*>(workspace), &w);
        CUtensorMap tm_q, tm_k;
        if (!qk_maps(a, &tm_q, &tm_k)) return KDA_ERR_CUDA;
        err = kda::launch_gdn_tables(a, w, s);
        if (err == cudaSuccess) err = kda::launch_gdn_prep(a, w, tm_q, tm_k, s);
        if (err == cudaSuccess) err = kda::launch_gdn_scan(a, w, tm_q, tm_k, s);
    } else {
        err = kda::launch_gdn_recurrent(qkv_dtype == KDA_DTYPE_F32, a, s);
    }
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_gdn_prefill_backward_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs, int64_t total_tokens, int32_t Hk,
                                                int32_t Hv, int32_t dk, int32_t dv) {
    if (qkv_dtype != KDA_DTYPE_BF16 || gdn_shape(qkv_dtype, total_tokens, num_seqs, Hk, Hv, dk, dv) != KDA_OK) return 0;
    const int64_t few = std::min(total_tokens, most_by_token_backward(num_seqs, Hv));
    const int32_t n = most_in_chunks(num_seqs, total_tokens, [&](int64_t N) { return most_by_token_backward(N, Hv); });
    return std::max(backward_takes(num_seqs, few, Hk, Hv), n ? backward_takes(n, total_tokens, Hk, Hv) : 0);
}

kda_status kda_gdn_prefill_backward(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                                    const float* log_decay, const float* beta, const float* S0,
                                    const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t Hk,
                                    int32_t Hv, int32_t dk, int32_t dv, const void* grad_o,
                                    const float* grad_S_final, void* grad_q, void* grad_k, void* grad_v,
                                    float* grad_log_decay, float* grad_beta, float* grad_S0, void* workspace,
                                    size_t workspace_bytes, int32_t* device_status, kda_stream_t stream) {
    const kda_status shape = gdn_shape(qkv_dtype, total_tokens, num_seqs, Hk, Hv, dk, dv);
    if (shape != KDA_OK) return shape;
    if (qkv_dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens || !workspace) return KDA_ERR_INVALID_ARG;
    const bool have_tokens = total_tokens > 0;
    if (have_tokens && (!q || !k || !v || !log_decay || !beta || !grad_o || !grad_q || !grad_k || !grad_v ||
                        !grad_log_decay || !grad_beta))
        return KDA_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, grad_o, static_cast<const void*>(grad_q), static_cast<const void*>(grad_k),
                          static_cast<const void*>(grad_v), static_cast<const void*>(S0),
                          static_cast<const void*>(grad_S_final), static_cast<const void*>(grad_S0)})
        if (!aligned(x, 16)) return KDA_ERR_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(log_decay), static_cast<const void*>(beta),
                          static_cast<const void*>(grad_log_decay), static_cast<const void*>(grad_beta),
                          static_cast<const void*>(cu_seqlens), static_cast<const void*>(device_status)})
        if (!aligned(x, 4)) return KDA_ERR_INVALID_ARG;
    if (!aligned(workspace, kAlign)) return KDA_ERR_INVALID_ARG;
    const size_t need = backward_takes(num_seqs, total_tokens, Hk, Hv);
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;

    // the outputs (and the workspace) overlap nothing
    const size_t T = static_cast<size_t>(total_tokens), nqk = T * Hk * kHeadDim * 2, nv = T * Hv * kHeadDim * 2;
    const size_t nst = static_cast<size_t>(num_seqs) * Hv * kStateBytes;
    const Range outs[] = {range_of(grad_q, nqk),
                          range_of(grad_k, nqk),
                          range_of(grad_v, nv),
                          range_of(grad_log_decay, T * Hv * 4),
                          range_of(grad_beta, T * Hv * 4),
                          range_of(grad_S0, grad_S0 ? nst : 0),
                          range_of(workspace, need),
                          range_of(device_status, device_status ? 4 : 0)};
    const Range ins[] = {range_of(q, nqk), range_of(k, nqk), range_of(v, nv), range_of(grad_o, nv),
                         range_of(log_decay, T * Hv * 4), range_of(beta, T * Hv * 4), range_of(S0, S0 ? nst : 0),
                         range_of(grad_S_final, grad_S_final ? nst : 0),
                         range_of(cu_seqlens, (static_cast<size_t>(num_seqs) + 1) * 4)};
    constexpr int n_outs = sizeof(outs) / sizeof(outs[0]);
    for (int i = 0; i < n_outs; ++i) {
        for (int j = i + 1; j < n_outs; ++j)
            if (overlap(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
        for (const Range& in : ins)
            if (overlap(outs[i], in)) return KDA_ERR_INVALID_ARG;
    }
    const kda_status dev = kda::device_check();
    if (dev != KDA_OK) return dev;
    if (num_seqs == 0) return KDA_OK;

    kda::GdnArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.beta = beta;
    a.S0 = S0;
    a.cu_seqlens = cu_seqlens;
    a.device_status = device_status;
    a.total_tokens = total_tokens;
    a.num_seqs = num_seqs;
    a.Hk = Hk;
    a.Hv = Hv;
    kda::GdnBackwardArgs b;
    b.grad_o = grad_o;
    b.grad_S_final = grad_S_final;
    b.grad_q = grad_q;
    b.grad_k = grad_k;
    b.grad_v = grad_v;
    b.grad_log_decay = grad_log_decay;
    b.grad_beta = grad_beta;
    b.grad_S0 = grad_S0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!chunked_backward(num_seqs, total_tokens, Hv))
        return kda::launch_gdn_recurrent_backward(a, b, workspace, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    kda::GdnWorkspace w;
    kda::gdn_workspace(num_seqs, total_tokens, Hv, true, static_cast<uint8_t*>(workspace), &w);
    CUtensorMap tm_q, tm_k;
    if (!qk_maps(a, &tm_q, &tm_k)) return KDA_ERR_CUDA;
    cudaError_t err = kda::launch_gdn_tables(a, w, s);
    if (err == cudaSuccess) err = kda::launch_gdn_prep(a, w, tm_q, tm_k, s);
    if (err == cudaSuccess) err = kda::launch_gdn_backward(a, b, w, tm_q, tm_k, s);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_gdn_decode_step(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                               const float* log_decay, const float* beta, float* S, int32_t num_slots,
                               const int32_t* state_indices, int32_t N, int32_t Hk, int32_t Hv, int32_t dk,
                               int32_t dv, void* o, int32_t* device_status, kda_stream_t stream) {
    kda_status st = gdn_shape(qkv_dtype, N, num_slots, Hk, Hv, dk, dv);
    if (st != KDA_OK) return st;
    if (static_cast<double>(N) * Hv > 2147483647.0) return KDA_ERR_INVALID_ARG;
    if (!state_indices && N > num_slots) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!q || !k || !v || !log_decay || !beta || !S || !o)) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(S, 16) ||
                  !aligned(log_decay, 4) || !aligned(beta, 4)))
        return KDA_ERR_INVALID_ARG;
    if ((state_indices && !aligned(state_indices, 4)) || (device_status && !aligned(device_status, 4)))
        return KDA_ERR_INVALID_ARG;
    const size_t es = esize_of(qkv_dtype), n = static_cast<size_t>(N);
    const Range outs[] = {range_of(o, n * Hv * kHeadDim * es),
                          range_of(S, N > 0 ? static_cast<size_t>(num_slots) * Hv * kStateBytes : 0),
                          range_of(device_status, device_status ? 4 : 0)};
    const Range ins[] = {range_of(q, n * Hk * kHeadDim * es), range_of(k, n * Hk * kHeadDim * es),
                         range_of(v, n * Hv * kHeadDim * es), range_of(log_decay, n * Hv * 4),
                         range_of(beta, n * Hv * 4), range_of(state_indices, state_indices ? n * 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
        for (const Range& in : ins)
            if (overlap(outs[i], in)) return KDA_ERR_INVALID_ARG;
    }
    st = kda::device_check();
    if (st != KDA_OK) return st;
    return kda::launch_gdn_decode(qkv_dtype == KDA_DTYPE_F32, q, k, v, log_decay, beta, S, num_slots, state_indices, N,
                                  Hk, Hv, o, device_status, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"

// ================================================================ RMS norm ==
namespace {

kda_status norm_shape(kda_dtype t, int64_t rows, int32_t dim, float eps) {
    if (t != KDA_DTYPE_BF16 && t != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || rows > INT32_MAX || dim < 1 || dim > KDA_NORM_MAX_DIM || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}
// `out` may be `in` itself, else they do not overlap.
bool clash(Range out, Range in) { return out.lo != in.lo && overlap(out, in); }

}  // namespace

extern "C" {

kda_status kda_rms_norm(const void* x, const void* residual, kda_dtype dtype, const float* weight, float eps,
                        int64_t rows, int32_t dim, kda_norm_out out_type, int32_t group, void* y, float* scales,
                        void* residual_out, kda_stream_t stream) {
    kda_status st = norm_shape(dtype, rows, dim, eps);
    if (st != KDA_OK) return st;
    if (out_type != KDA_NORM_OUT_SAME && out_type != KDA_NORM_OUT_E4M3 && out_type != KDA_NORM_OUT_INT8)
        return KDA_ERR_UNSUPPORTED;
    const bool coded = out_type != KDA_NORM_OUT_SAME;
    if (coded ? (group != 0 && group != 128) || (group == 128 && dim % 128 != 0) : group != 0)
        return KDA_ERR_INVALID_ARG;
    if (coded != (scales != nullptr) && (scales || rows > 0)) return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(y, 16) ||
        !aligned(weight, 4) || !aligned(scales, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(rows) * dim, es = esize_of(dtype);
    const Range r_x = range_of(x, n * es), r_res = range_of(residual, residual ? n * es : 0);
    const Range r_w = range_of(weight, weight ? static_cast<size_t>(dim) * 4 : 0);
    const Range r_y = range_of(y, n * (coded ? 1 : es)), r_h = range_of(residual_out, residual_out ? n * es : 0);
    const Range r_s = range_of(scales, coded ? static_cast<size_t>(rows) * (group ? dim / group : 1) * 4 : 0);
    if (clash(r_h, r_x) || clash(r_h, r_res) || overlap(r_h, r_w) || overlap(r_h, r_y) || overlap(r_h, r_s))
        return KDA_ERR_INVALID_ARG;
    if ((coded ? overlap(r_y, r_x) : clash(r_y, r_x)) || overlap(r_y, r_res) || overlap(r_y, r_w) ||
        overlap(r_y, r_s))
        return KDA_ERR_INVALID_ARG;
    if (overlap(r_s, r_x) || overlap(r_s, r_res) || overlap(r_s, r_w)) return KDA_ERR_INVALID_ARG;
    st = kda::device_check();
    if (st != KDA_OK) return st;
    kda::NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.eps = eps;
    a.rows = rows;
    a.dim = dim;
    a.group = group;
    a.y = y;
    a.scales = scales;
    a.residual_out = residual_out;
    return kda::launch_rms_norm(dtype == KDA_DTYPE_F32, out_type, a, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

size_t kda_rms_norm_backward_workspace_bytes(int64_t rows, int32_t dim) {
    if (norm_shape(KDA_DTYPE_BF16, rows, dim, 0.f) != KDA_OK) return 0;
    const size_t parts = static_cast<size_t>(kda::rms_norm_backward_partials(rows));
    return round_up(std::max<size_t>(parts, 1) * dim * 4, kAlign);
}

kda_status kda_rms_norm_backward(const void* grad_y, const void* h, const void* grad_h, kda_dtype dtype,
                                 const float* weight, float eps, int64_t rows, int32_t dim, void* grad_x,
                                 float* grad_weight, void* workspace, size_t workspace_bytes, kda_stream_t stream) {
    kda_status st = norm_shape(dtype, rows, dim, eps);
    if (st != KDA_OK) return st;
    if (rows > 0 && (!grad_y || !h || !grad_x)) return KDA_ERR_INVALID_ARG;
    if (!aligned(grad_y, 16) || !aligned(h, 16) || !aligned(grad_h, 16) || !aligned(grad_x, 16) ||
        !aligned(weight, 4) || !aligned(grad_weight, 16) || !aligned(workspace, kAlign))
        return KDA_ERR_INVALID_ARG;
    const size_t need = grad_weight ? kda_rms_norm_backward_workspace_bytes(rows, dim) : 0;
    if (grad_weight && !workspace) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const size_t n = static_cast<size_t>(rows) * dim, es = esize_of(dtype), wb = static_cast<size_t>(dim) * 4;
    const Range r_dy = range_of(grad_y, n * es), r_h = range_of(h, n * es);
    const Range r_dh = range_of(grad_h, grad_h ? n * es : 0), r_w = range_of(weight, weight ? wb : 0);
    const Range r_dx = range_of(grad_x, n * es), r_dw = range_of(grad_weight, grad_weight ? wb : 0);
    const Range r_ws = range_of(workspace, need);
    if (clash(r_dx, r_dy) || clash(r_dx, r_dh) || overlap(r_dx, r_h) || overlap(r_dx, r_w) || overlap(r_dx, r_dw) ||
        overlap(r_dx, r_ws))
        return KDA_ERR_INVALID_ARG;
    for (const Range& in : {r_dy, r_h, r_dh, r_w})
        if (overlap(r_dw, in) || overlap(r_ws, in)) return KDA_ERR_INVALID_ARG;
    if (overlap(r_dw, r_ws)) return KDA_ERR_INVALID_ARG;
    st = kda::device_check();
    if (st != KDA_OK) return st;
    kda::NormBackwardArgs a;
    a.grad_y = grad_y;
    a.h = h;
    a.grad_h = grad_h;
    a.weight = weight;
    a.eps = eps;
    a.rows = rows;
    a.dim = dim;
    a.grad_x = grad_x;
    a.grad_weight = grad_weight;
    a.partial = static_cast<float*>(workspace);
    return kda::launch_rms_norm_backward(dtype == KDA_DTYPE_F32, a, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
