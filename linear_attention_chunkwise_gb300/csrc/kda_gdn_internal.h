// kda_gdn_internal.h -- interface between the C-ABI front end of the gated delta rule and of the RMS norm
// (kda_gdn_api.cu) and their kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kda_args.h"

namespace kda {

// ---- gated delta rule, one decay per (token, value head) ----
struct GdnArgs {
    const void* q = nullptr;  // [T, Hk, 128]
    const void* k = nullptr;
    const void* v = nullptr;  // [T, Hv, 128]
    const float* log_decay = nullptr;  // [T, Hv]
    const float* beta = nullptr;
    const float* S0 = nullptr;         // NULL: zeros
    const int32_t* cu_seqlens = nullptr;
    void* o = nullptr;
    float* S_final = nullptr;          // NULL: not stored
    int32_t* device_status = nullptr;
    int64_t total_tokens = 0;
    int32_t num_seqs = 0;
    int32_t Hk = 0, Hv = 0;
};
// Token by token in fp32 (kda_gdn_recurrent.cu).
cudaError_t launch_gdn_recurrent(bool f32_io, const GdnArgs& a, cudaStream_t stream);
// Chunkwise, bf16 (kda_gdn_prefill.cu, kda_gdn_backward.cu).
struct GdnWorkspace {
    int32_t* order = nullptr;    // sequences, longest first (NULL: in index order)
    int32_t* table = nullptr;    // chunk table (NULL: one sequence)
    uint8_t* images = nullptr;   // per (chunk, value head): the scans' operands
    uint8_t* records = nullptr;  // per (chunk, value head): states, adjoints, U and W (NULL: the prefill)
    int64_t chunks = 0;          // chunk entries: ceil(T / 64) + num_seqs
};
// Bytes of the workspace, and (w not NULL) its regions from `base`; bwd: the gradient's.
size_t gdn_workspace(int32_t num_seqs, int64_t total_tokens, int32_t Hv, bool bwd, uint8_t* base, GdnWorkspace* w);
cudaError_t launch_gdn_tables(const GdnArgs& a, const GdnWorkspace& w, cudaStream_t stream);
// Whether CTAs of 32 columns find an SM each (else the gradient's walks take 64, and sequences go by length).
bool gdn_narrow(int32_t num_seqs, int32_t Hv);
// tm_q, tm_k: maps of q and k with boxes of 64 tokens x 64 channels, 128B-swizzled.
cudaError_t launch_gdn_prep(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                            cudaStream_t stream);
cudaError_t launch_gdn_scan(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                            cudaStream_t stream);
cudaError_t launch_gdn_wide(const GdnArgs& a, const GdnWorkspace& w, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                            cudaStream_t stream);
struct GdnBackwardArgs {
    const void* grad_o = nullptr;          // [T, Hv, 128]
    const float* grad_S_final = nullptr;   // NULL: zeros
    void* grad_q = nullptr;                // [T, Hk, 128], the input type
    void* grad_k = nullptr;
    void* grad_v = nullptr;                // [T, Hv, 128]
    float* grad_log_decay = nullptr;       // [T, Hv]
    float* grad_beta = nullptr;
    float* grad_S0 = nullptr;              // NULL: not stored
};
// Token by token in fp32 (kda_gdn_recurrent.cu).
size_t gdn_recurrent_backward_workspace(int64_t total_tokens, int32_t Hk, int32_t Hv);
cudaError_t launch_gdn_recurrent_backward(const GdnArgs& a, const GdnBackwardArgs& b, void* workspace, cudaStream_t stream);
cudaError_t launch_gdn_backward(const GdnArgs& a, const GdnBackwardArgs& b, const GdnWorkspace& w, const CUtensorMap& tm_q,
                                const CUtensorMap& tm_k, cudaStream_t stream);
cudaError_t launch_gdn_decode(bool f32_io, const void* q, const void* k, const void* v, const float* log_decay,
                              const float* beta, float* S, int32_t num_slots, const int32_t* state_indices, int32_t N,
                              int32_t Hk, int32_t Hv, void* o, int32_t* device_status, cudaStream_t stream);

// ---- RMS norm (kda_rms_norm.cu) ----
struct NormArgs {
    const void* x = nullptr;
    const void* residual = nullptr;  // NULL: none
    const float* weight = nullptr;   // NULL: ones
    float eps = 0.f;
    int64_t rows = 0;
    int32_t dim = 0;
    int32_t group = 0;               // columns per scale (0: the row)
    void* y = nullptr;
    float* scales = nullptr;
    void* residual_out = nullptr;    // NULL: not stored
};
cudaError_t launch_rms_norm(bool f32_io, int32_t out_type, const NormArgs& a, cudaStream_t stream);
struct NormBackwardArgs {
    const void* grad_y = nullptr;
    const void* h = nullptr;
    const void* grad_h = nullptr;    // NULL: none
    const float* weight = nullptr;   // NULL: ones
    float eps = 0.f;
    int64_t rows = 0;
    int32_t dim = 0;
    void* grad_x = nullptr;
    float* grad_weight = nullptr;    // NULL: not computed
    float* partial = nullptr;        // [rms_norm_backward_partials(rows)][dim]
};
// Row blocks whose sums of the weight's gradient are added at the end.
int64_t rms_norm_backward_partials(int64_t rows);
cudaError_t launch_rms_norm_backward(bool f32_io, const NormBackwardArgs& a, cudaStream_t stream);

}  // namespace kda
