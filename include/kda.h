/*
 * kda.h -- C ABI of libkda: Kimi Delta Attention (KDA) recurrence on sm_103a.
 *
 * The operation (per head, state S is dk x dv, rows = key channels):
 *
 *   S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *   o_t = S_t^T q_t                         (read from the UPDATED state)
 *
 * Sources: the KDA equation in "Understanding Kimi Delta Attention"
 * (pyshine), section "The KDA Recurrence: Scalar Gate vs Channel-wise Gate";
 * per-row (key-channel) decay and the read o_t = S_t^T q_t in "kimi delta
 * attn from first principles" (aryagxr), section "KDA".  Page 1 of the
 * sources reads the state with k_t instead ("Understanding the
 * Recurrence"); this library follows the query read.
 *
 * Conventions shared by every entry point
 *   - alpha_t = exp(log_alpha_t) (natural log), one gate per key channel;
 *     beta_t is used as given (the sources give it as a sigmoid in [0, 1]).
 *   - No scaling or normalisation of q/k in the plain entry points: callers
 *     pass q and k already L2-normalised per (token, head), as the sources'
 *     "KDA Architecture" section describes (the _ex entry points can do it
 *     inside the kernels, see kda_fusion).
 *   - dk = dv = 128 only (the sources' 128 x 128 state); anything else
 *     returns KDA_ERR_UNSUPPORTED.
 *   - All tensors are dense, row-major, caller-owned DEVICE memory.  q, k,
 *     v, log_alpha, o and the states are 16-byte aligned; beta, cu_seqlens,
 *     state_indices and device_status 4-byte aligned; the prefill workspace
 *     256-byte aligned.  The library allocates no device memory, never
 *     synchronises the host, and enqueues all work on `stream` (a
 *     cudaStream_t; NULL = the legacy default stream).  It owns no streams,
 *     events or locks and keeps no state between calls except, per device,
 *     the kernels' attribute settings, how many clusters of a kernel fit, the
 *     entry points it looks up in the driver, and (kda_prefill_noalloc only)
 *     its fixed scratch array.
 *   - Argument errors are returned synchronously before anything is
 *     enqueued.  Data-dependent errors found on the device are OR-ed into
 *     *device_status (if non-NULL) as KDA_DEV_* bits; the affected sequences
 *     or slots are skipped and nothing is written out of bounds.  The caller
 *     reads *device_status after the stream completes and should zero it
 *     before the call.
 *   - Calls on different streams that write the same buffers race.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 1

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

typedef struct CUstream_st *kda_stream_t; /* same type as cudaStream_t */

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, illegal overlap */
    KDA_ERR_UNSUPPORTED = 2,   /* dk/dv other than 128, unknown dtype, device not sm_103 */
    KDA_ERR_CUDA = 3,          /* a CUDA runtime call failed (launch, attribute, ...) */
    KDA_ERR_WORKSPACE = 4      /* workspace smaller than kda_prefill_workspace_bytes() */
} kda_status;

typedef enum {
    KDA_DTYPE_BF16 = 0,
    KDA_DTYPE_F32 = 1
} kda_dtype;

/* Bits OR-ed into *device_status by the kernels. */
#define KDA_DEV_BAD_CU_SEQLENS 0x1  /* cu_seqlens not 0 .. total_tokens non-decreasing */
#define KDA_DEV_BAD_SLOT 0x2        /* state_indices entry outside [0, num_slots) */
#define KDA_DEV_TIMEOUT 0x4         /* an on-chip wait hit its iteration limit */
#define KDA_DEV_BAD_SNAPSHOT 0x8    /* kda_prefill_snapshots: a (sequence, position) entry is invalid */
#define KDA_DEV_BOUNDS 0x10         /* only in a library built with KDA_DEBUG_BOUNDS: a kernel derived a
                                       sequence, chunk, token or snapshot range outside its buffer and
                                       skipped that work (never set by a release build) */

/*
 * Fused prologue / epilogue (kda_prefill_ex, kda_decode_step_ex,
 * kda_decode_multi_ex): the elementwise steps around the recurrence that
 * "kimi delta attn from first principles" (aryagxr) lists -- q and k
 * L2-normalised ("KDA Architecture"),
 * the update gate beta as a sigmoid of its projection, and the output gate
 * (RMSNorm of o_t, then an elementwise product with g_t) ("KDA has three
 * gates").  The prologue runs inside the kernels (pass 1 of the prefill, the
 * decode kernels); the output gate runs inside the decode kernels and, for
 * the prefill, as one pass over o and the gate after the scan (the row's
 * mean square is taken from the row it scales).
 *
 *   KDA_FUSE_L2NORM_QK   q, k <- x / sqrt(sum_c x_c^2 + l2_eps), per (token, head)
 *   KDA_FUSE_BETA_SIGMOID  beta holds logits b; beta = 1 / (1 + exp(-b)) is used
 *   KDA_FUSE_OUT_GATE    the output is y = o / sqrt(mean_c o_c^2 + rms_eps)
 *                        * rms_weight * out_gate instead of o
 *
 * rms_weight: [dv] fp32 device (NULL = all ones); out_gate: [tokens, H, dv]
 * in qkv_dtype, device, 16-byte aligned (required with KDA_FUSE_OUT_GATE
 * unless tokens = 0; tokens = total_tokens for prefill, N for a decode step,
 * N x T for kda_decode_multi_ex).  l2_eps, rms_eps >= 0.
 * The state and S_final are those of the normalised q, k and sigmoid beta.
 */
#define KDA_FUSE_L2NORM_QK 0x1u
#define KDA_FUSE_BETA_SIGMOID 0x2u
#define KDA_FUSE_OUT_GATE 0x4u
typedef struct {
    uint32_t flags;
    float l2_eps;
    float rms_eps;
    const float *rms_weight;
    const void *out_gate;
} kda_fusion;

/* Version of this header the library was built from. */
KDA_API int32_t kda_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
KDA_API const char *kda_status_string(kda_status s);

/*
 * Workspace (device bytes, 256-byte aligned start) for kda_prefill's
 * two-pass path (the fast one): the sequence schedule, the chunk table, bf16
 * copies of q, k, v when qkv_dtype is KDA_DTYPE_F32, 67,072 bytes per
 * (chunk, head) of prepared operands, counting ceil(total_tokens/64) +
 * num_seqs chunks -- about 1.05 KB per token and head -- and one fp32 state
 * per (sequence, head), 64 KB each, that carries the state between the scan's
 * pieces when the call passes no S_final.  Returns 0 for invalid arguments.
 */
KDA_API size_t kda_prefill_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs,
                                   int64_t total_tokens, int32_t H,
                                   int32_t dk, int32_t dv);

/*
 * Smallest workspace kda_prefill accepts: the schedule (+ bf16 copies for
 * fp32 inputs).  With less than kda_prefill_workspace_bytes() it runs the
 * single-pass path, one CTA per (sequence, head), which is slower for few
 * long sequences.  Returns 0 for invalid arguments.
 */
KDA_API size_t kda_prefill_min_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs,
                                       int64_t total_tokens, int32_t H,
                                       int32_t dk, int32_t dv);

/*
 * kda_prefill -- chunkwise-parallel prefill over packed variable-length
 * sequences ("Understanding Kimi Delta Attention" (pyshine), section
 * "The Chunkwise DPLR Algorithm": fixed-size chunks, exactly equivalent to
 * the sequential recurrence).  Chunk size 64, fp32 state, bf16 tensor-core
 * operands with fp32 accumulation.
 *
 *   q, k       [total_tokens, H, dk]  qkv_dtype
 *   v          [total_tokens, H, dv]  qkv_dtype
 *   log_alpha  [total_tokens, H, dk]  fp32   (per key channel; see below)
 *   beta       [total_tokens, H]      fp32
 *   S0         [num_seqs, H, dk, dv]  fp32, or NULL for zero start states
 *   cu_seqlens [num_seqs + 1]         int32, device; 0 = c_0 <= ... <= c_N = total_tokens
 *   o          [total_tokens, H, dv]  qkv_dtype (out)
 *   S_final    [num_seqs, H, dk, dv]  fp32 (out), or NULL
 *   workspace  device scratch: >= kda_prefill_workspace_bytes(...) bytes
 *              selects the two-pass path (chunk preparation for all
 *              (chunk, head) pairs in parallel, then a scan over chunks per
 *              (sequence, head, 64-column slice of dv)); >=
 *              kda_prefill_min_workspace_bytes(...) selects the single-pass
 *              path; less returns KDA_ERR_WORKSPACE.  Both paths compute the
 *              same chunk algebra.
 *
 * Sequence n covers tokens [cu_seqlens[n], cu_seqlens[n+1]) and starts from
 * S0[n] (the prefix-cache state of "Kimi Delta Attention (KDA)"
 * (codewithdark), section "KV Caching Challenges & vLLM Contribution");
 * S_final[n] is its state after the last token (S0[n] for an empty
 * sequence).  S_final may alias S0 exactly; any other overlap between an
 * output and another buffer returns KDA_ERR_INVALID_ARG.  A malformed
 * cu_seqlens sets KDA_DEV_BAD_CU_SEQLENS; the single-pass path then skips the
 * sequences whose bounds are invalid, the two-pass path writes nothing.
 *
 * Range: the chunk factorisation takes exp(+-(g_r - g_ref)) of the
 * cumulative log-decay within a chunk, so log_alpha must be >= -2.5 per step
 * (documented precondition; values below it can overflow to inf/NaN).
 * q, k, v given as fp32 are rounded to bf16 operands.
 */
KDA_API kda_status kda_prefill(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                       const float *log_alpha, const float *beta, const float *S0,
                       const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                       int32_t H, int32_t dk, int32_t dv, void *o, float *S_final,
                       void *workspace, size_t workspace_bytes, int32_t *device_status,
                       kda_stream_t stream);

/*
 * kda_prefill_snapshots -- kda_prefill that also records the state at
 * caller-chosen positions inside the sequences: the prefix-cache boundaries
 * of "Kimi Delta Attention (KDA)" (codewithdark), section "KV Caching
 * Challenges & vLLM Contribution", where a cached prefix is resumed from its
 * state instead of being recomputed.
 *
 *   snap_seq   [num_snaps] int32, device: sequence index of each entry
 *   snap_pos   [num_snaps] int32, device: tokens of that sequence consumed,
 *              a multiple of 64 or the sequence length, 0 < pos <= length
 *   S_snap     [num_snaps, H, dk, dv] fp32 (out): entry i receives the
 *              state after the first snap_pos[i] tokens of sequence
 *              snap_seq[i] -- exactly the S_final a kda_prefill over that
 *              prefix alone would return
 *
 * Entries must be sorted by (sequence, position) with no repeats.  An entry
 * that breaks a rule sets KDA_DEV_BAD_SNAPSHOT; its S_snap slice may then be
 * left unwritten (never a write outside S_snap).  All other arguments and
 * errors are those of kda_prefill; snapshots need the two-pass workspace
 * (>= kda_prefill_workspace_bytes), else KDA_ERR_WORKSPACE.
 */
KDA_API kda_status kda_prefill_snapshots(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                 const float *log_alpha, const float *beta, const float *S0,
                                 const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                 int32_t H, int32_t dk, int32_t dv, void *o, float *S_final,
                                 const int32_t *snap_seq, const int32_t *snap_pos, int32_t num_snaps,
                                 float *S_snap, void *workspace, size_t workspace_bytes,
                                 int32_t *device_status, kda_stream_t stream);

/*
 * kda_prefill_ex -- kda_prefill with the fused prologue / epilogue of
 * `fusion` (host pointer; NULL or flags = 0 is kda_prefill).  With any flag
 * set the two-pass workspace is required (>= kda_prefill_workspace_bytes),
 * else KDA_ERR_WORKSPACE.  Unknown flags, a missing out_gate, or a negative
 * eps return KDA_ERR_INVALID_ARG; out_gate overlapping o returns it too.
 */
KDA_API kda_status kda_prefill_ex(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                          const float *log_alpha, const float *beta, const float *S0,
                          const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                          int32_t H, int32_t dk, int32_t dv, void *o, float *S_final,
                          const kda_fusion *fusion, void *workspace, size_t workspace_bytes,
                          int32_t *device_status, kda_stream_t stream);

/*
 * kda_prefill_backward -- reverse-mode gradient of kda_prefill (plain
 * inputs; no fusion) for the scalar loss
 *     L = sum_{t,h,j} o[t,h,j] grad_o[t,h,j] + sum_{n,h,i,j} S_final grad_S_final,
 * i.e. the vector-Jacobian product of the recurrence of "Understanding Kimi
 * Delta Attention" (pyshine), section "The KDA Recurrence", read in the
 * erase-then-write order of "kimi delta attn from first principles"
 * (aryagxr), section "KDA".  The pages train the layer but print no
 * backward; this is the exact derivative of that update, per token.
 *
 *   q, k, v, log_alpha, beta, S0, cu_seqlens, num_seqs, total_tokens, H,
 *   dk, dv     the forward's inputs, as kda_prefill (S0 may be NULL = zeros)
 *   grad_o        [total_tokens, H, dv] qkv_dtype, device (dL/do)
 *   grad_S_final  [num_seqs, H, dk, dv] fp32 device, or NULL (zeros)
 *   grad_q, grad_k, grad_v, grad_log_alpha  [total_tokens, H, 128] fp32 out
 *   grad_beta     [total_tokens, H] fp32 out
 *   grad_S0       [num_seqs, H, dk, dv] fp32 out, or NULL (not computed)
 *
 * The library reruns the chunkwise forward inside the call, recording the
 * state after every 64-token chunk, then computes the gradient chunkwise in
 * fp32: one walk of the state's adjoint back over the chunks of each
 * (sequence, head), and dense per-chunk products for everything else.  The
 * gradients are those of the fp32 recurrence on the given inputs; the only
 * bf16 step is the chunkwise forward that supplies the chunk-start states.
 * Results are bitwise repeatable.
 *
 * Workspace: >= kda_prefill_backward_workspace_bytes(...) device bytes,
 * 256-byte aligned (KDA_ERR_WORKSPACE below it).  Pointers: 16-byte aligned
 * (beta, grad_beta: 4).  The outputs overlap nothing: not each other, the
 * inputs or the workspace (KDA_ERR_INVALID_ARG).  Other errors are
 * kda_prefill's; a malformed cu_seqlens sets KDA_DEV_BAD_CU_SEQLENS and leaves
 * the gradients unspecified.  Asynchronous on `stream`.
 */
KDA_API size_t kda_prefill_backward_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs, int64_t total_tokens,
                                                    int32_t H, int32_t dk, int32_t dv);
KDA_API kda_status kda_prefill_backward(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                        const float *log_alpha, const float *beta, const float *S0,
                                        const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                        int32_t H, int32_t dk, int32_t dv, const void *grad_o,
                                        const float *grad_S_final, float *grad_q, float *grad_k, float *grad_v,
                                        float *grad_log_alpha, float *grad_beta, float *grad_S0,
                                        void *workspace, size_t workspace_bytes, int32_t *device_status,
                                        kda_stream_t stream);

/*
 * kda_prefill_backward_ex -- kda_prefill_backward through the fused prologue
 * of kda_prefill_ex: q, k are the raw projections (L2-normalised per (token,
 * head) with KDA_FUSE_L2NORM_QK, "KDA Architecture") and beta the logits
 * (KDA_FUSE_BETA_SIGMOID, "KDA has three gates").  grad_q, grad_k, grad_beta
 * are then the gradients with respect to those raw inputs:
 *     dx = (dx_hat - x_hat <x_hat, dx_hat>) / sqrt(|x|^2 + l2_eps),
 *     db = dbeta_hat sigma(b) (1 - sigma(b)),
 * the exact chain rule through the prologue, taken in fp32.  The call
 * writes the normalised q, k (in qkv_dtype) and sigmoid beta into the
 * workspace, runs the plain backward on them, and applies the chain rule in
 * place.  KDA_FUSE_OUT_GATE returns KDA_ERR_UNSUPPORTED (the output gate's
 * backward needs two more outputs: kda_prefill_backward_gated); fusion NULL
 * or flags 0 is kda_prefill_backward.
 *
 * Workspace: >= kda_prefill_backward_ex_workspace_bytes(...) (the plain
 * figure plus (2 x 128 x sizeof(qkv_dtype) + 12) bytes per (token, head)).
 * Other arguments, errors and overlap rules as kda_prefill_backward.
 */
KDA_API size_t kda_prefill_backward_ex_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs,
                                                       int64_t total_tokens, int32_t H, int32_t dk, int32_t dv);
KDA_API kda_status kda_prefill_backward_ex(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                           const float *log_alpha, const float *beta, const float *S0,
                                           const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                           int32_t H, int32_t dk, int32_t dv, const void *grad_o,
                                           const float *grad_S_final, float *grad_q, float *grad_k,
                                           float *grad_v, float *grad_log_alpha, float *grad_beta,
                                           float *grad_S0, const kda_fusion *fusion, void *workspace,
                                           size_t workspace_bytes, int32_t *device_status, kda_stream_t stream);

/*
 * kda_prefill_backward_gated -- kda_prefill_backward_ex for the layer output
 * y = o / sqrt(mean_c o_c^2 + rms_eps) * rms_weight * out_gate of
 * kda_prefill_ex with KDA_FUSE_OUT_GATE (the output gate of "kimi delta attn
 * from first principles" (aryagxr), section "KDA has three gates").  With
 * r = (sum_c o_c^2 / 128 + rms_eps)^(-1/2), w = rms_weight, g = out_gate and
 * dy = grad_y = dL/dy per (token, head) row:
 *     dL/do_c = r w_c g_c dy_c - (r^3 o_c / 128) sum_j dy_j o_j w_j g_j
 *     grad_out_gate_c  = dy_c o_c r w_c
 *     grad_rms_weight_c = sum over all (token, head) rows of dy_c o_c r g_c
 * and dL/do feeds the chunkwise backward in place of grad_o.  The o here is
 * the chunkwise forward's own (rerun inside the call, rounded to qkv_dtype
 * as kda_prefill_ex would output it); dL/do is rounded to qkv_dtype, as
 * grad_o is given to kda_prefill_backward.
 *
 *   grad_y           [total_tokens, H, dv] qkv_dtype device (dL/dy)
 *   grad_out_gate    [total_tokens, H, dv] fp32 out, 16-byte aligned
 *   grad_rms_weight  [dv] fp32 out, or NULL (not computed); summed over
 *                    rows in a fixed order (bitwise repeatable)
 *   fusion           required, with KDA_FUSE_OUT_GATE set (else
 *                    KDA_ERR_INVALID_ARG) and out_gate, rms_weight, rms_eps
 *                    as given to the forward; KDA_FUSE_L2NORM_QK and
 *                    KDA_FUSE_BETA_SIGMOID act as in kda_prefill_backward_ex.
 *
 * Workspace: >= kda_prefill_backward_gated_workspace_bytes(...) (the _ex
 * figure rounded up to 256 bytes, plus 592 x 128 x 4 bytes of partial sums).
 * grad_out_gate and grad_rms_weight overlap nothing (KDA_ERR_INVALID_ARG).
 * Other arguments, errors and overlap rules as kda_prefill_backward_ex.
 */
KDA_API size_t kda_prefill_backward_gated_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs,
                                                          int64_t total_tokens, int32_t H, int32_t dk, int32_t dv);
KDA_API kda_status kda_prefill_backward_gated(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                              const float *log_alpha, const float *beta, const float *S0,
                                              const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                              int32_t H, int32_t dk, int32_t dv, const void *grad_y,
                                              const float *grad_S_final, float *grad_q, float *grad_k,
                                              float *grad_v, float *grad_log_alpha, float *grad_beta,
                                              float *grad_S0, float *grad_out_gate, float *grad_rms_weight,
                                              const kda_fusion *fusion, void *workspace, size_t workspace_bytes,
                                              int32_t *device_status, kda_stream_t stream);

/*
 * kda_decode_step -- one fused recurrent step for N sequences
 * ("Understanding Kimi Delta Attention" (pyshine), section "The Chunkwise
 * DPLR Algorithm": the step-by-step "fused recurrent mode" for decode).
 * Each head's fp32 state is read once and written once, in place.
 *
 *   q, k       [N, H, dk]  qkv_dtype        v [N, H, dv] qkv_dtype
 *   log_alpha  [N, H, dk]  fp32             beta [N, H] fp32
 *   S          [num_slots, H, dk, dv] fp32, updated in place
 *   state_indices [N] int32 device, or NULL for slot = n.  Entries must be
 *              unique (duplicates race); out-of-range entries set
 *              KDA_DEV_BAD_SLOT and that sequence is skipped (its o row is
 *              left untouched).  Slots not named are never touched.
 *   o          [N, H, dv]  qkv_dtype (out)
 */
KDA_API kda_status kda_decode_step(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                           const float *log_alpha, const float *beta, float *S,
                           int32_t num_slots, const int32_t *state_indices, int32_t N,
                           int32_t H, int32_t dk, int32_t dv, void *o,
                           int32_t *device_status, kda_stream_t stream);

/*
 * kda_decode_step_ex -- kda_decode_step with the fused prologue / epilogue
 * of `fusion` (host pointer; NULL or flags = 0 is kda_decode_step).  Errors
 * as kda_prefill_ex; out_gate is [N, H, dv].
 */
KDA_API kda_status kda_decode_step_ex(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                              const float *log_alpha, const float *beta, float *S,
                              int32_t num_slots, const int32_t *state_indices, int32_t N,
                              int32_t H, int32_t dk, int32_t dv, void *o, const kda_fusion *fusion,
                              int32_t *device_status, kda_stream_t stream);

/*
 * kda_decode_multi -- T consecutive tokens per sequence in one launch: a
 * speculative-decoding verify step or a short continuation (the fused
 * recurrent mode of "Understanding Kimi Delta Attention" (pyshine), "The
 * Chunkwise DPLR Algorithm", over T steps; the speculative-decoding path of
 * its "Scaling to Kimi K3" section).  Each head's fp32 state is read once,
 * carried through the T updates on chip, and written once, in place.  The
 * per-token arithmetic is exactly kda_decode_step's.
 *
 *   q, k       [N, T, H, dk]  qkv_dtype        v [N, T, H, dv] qkv_dtype
 *   log_alpha  [N, T, H, dk]  fp32             beta [N, T, H] fp32
 *   S          [num_slots, H, dk, dv] fp32, updated in place to the state
 *              after all T tokens
 *   state_indices, device_status: as kda_decode_step
 *   o          [N, T, H, dv]  qkv_dtype (out), o[n, t] read after token t
 *   S_steps    [N, T, H, dk, dv] fp32 (out) or NULL: the state after each
 *              token, for rolling back to an accepted prefix
 * T = 0 is a no-op.
 */
KDA_API kda_status kda_decode_multi(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                    const float *log_alpha, const float *beta, float *S,
                                    int32_t num_slots, const int32_t *state_indices, int32_t N,
                                    int32_t T, int32_t H, int32_t dk, int32_t dv, void *o,
                                    float *S_steps, int32_t *device_status, kda_stream_t stream);

/*
 * kda_decode_multi_ex -- kda_decode_multi with the fused prologue / epilogue
 * of `fusion` per token (host pointer; NULL or flags = 0 is kda_decode_multi).
 * Errors as kda_prefill_ex; out_gate is [N, T, H, dv].
 */
KDA_API kda_status kda_decode_multi_ex(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                               const float *log_alpha, const float *beta, float *S,
                               int32_t num_slots, const int32_t *state_indices, int32_t N,
                               int32_t T, int32_t H, int32_t dk, int32_t dv, void *o, float *S_steps,
                               const kda_fusion *fusion, int32_t *device_status, kda_stream_t stream);

/*
 * kda_prefill_noalloc -- kda_prefill for callers that cannot allocate device
 * memory.  The sources have no counterpart to this entry point; it exists for
 * integration.  Some callers cannot hand the library a workspace: a plugin
 * that an inference engine gives only the tensors it owns, after the engine
 * has reserved all of HBM for its caches, or a latency-critical path where
 * cudaMalloc's implicit device synchronisation is not allowed.
 *
 * Same arguments and results as kda_prefill, minus the workspace.  Its
 * scratch lives in a fixed array in device global memory inside libkda:
 * KDA_NOALLOC_MAX_SEQS int32 (256 KiB), held on every GPU that loads the
 * library until the process exits.  That is passed to kda_prefill as its
 * workspace, so the single-pass path runs (the two-pass path only for inputs
 * small enough to fit).  It allocates nothing and calls no allocating
 * routine.
 *   - num_seqs > KDA_NOALLOC_MAX_SEQS returns KDA_ERR_WORKSPACE; fp32 q/k/v
 *     (which need token-sized scratch) return KDA_ERR_UNSUPPORTED.
 *   - The first call on each device looks up the array's device address
 *     (with that device current) and caches it; make that first call before
 *     any stream capture.
 *   - Every call shares the one array, which keeps the last call's contents
 *     (each call rewrites the part it reads before reading it).  Calls whose
 *     work overlaps on the GPU -- on different streams, or from different
 *     threads -- race on it: serialise them.
 */
#define KDA_NOALLOC_MAX_SEQS 65536

KDA_API kda_status kda_prefill_noalloc(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                       const float *log_alpha, const float *beta, const float *S0,
                                       const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                       int32_t H, int32_t dk, int32_t dv, void *o, float *S_final,
                                       int32_t *device_status, kda_stream_t stream);

/*
 * The gated delta rule: the recurrence with the scalar gate of "Understanding
 * Kimi Delta Attention" (pyshine), section "The KDA Recurrence: Scalar Gate vs
 * Channel-wise Gate", one decay per token and head instead of one per channel:
 *
 *   S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,  a_t = exp(log_decay_t)
 *   o_t = S_t^T q_t
 *
 * The kda_gdn_ entry points follow the conventions at the top of this file
 * (dense tensors, q and k normalised by the caller, beta as given, dk = dv =
 * 128) and add heads in groups: Hk heads of q and k, Hv of v, Hv a multiple of
 * Hk; value head h uses q/k head h / (Hv / Hk).  log_decay has no lower limit
 * (-inf, a decay of 0, included): decays enter as exp of differences that are
 * at most the largest decay.  States, decays and the sums over tokens are held
 * in fp32.  Token by token (below: short sequences, fp32 inputs, the decode
 * step) the products are fp32 too.  In chunks the products that make states and
 * fp32 gradients take operands of two bf16 terms, off by at most 2^-17: S_final
 * and those gradients agree with the recurrence to about 5e-6 of their 2-norm
 * (fp32 products: 1e-7 to 4e-7).  The products that make o, grad_q and grad_k
 * take some operands in one bf16 term: o is off by 3.3e-3, grad_q and grad_k by
 * 2.2e-3, where their own rounding to bf16 is 1.7e-3.
 */

/*
 * Workspace of kda_gdn_prefill (device bytes, 256-byte aligned start), enough
 * for every call with as many tokens and sequences or fewer (of the same heads).
 * Returns 0 for invalid arguments.
 */
KDA_API size_t kda_gdn_prefill_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs, int64_t total_tokens,
                                               int32_t Hk, int32_t Hv, int32_t dk, int32_t dv);

/*
 * kda_gdn_prefill -- the gated delta rule over packed variable-length sequences.
 *
 *   q, k       [total_tokens, Hk, dk]  qkv_dtype
 *   v          [total_tokens, Hv, dv]  qkv_dtype
 *   log_decay  [total_tokens, Hv]      fp32
 *   beta       [total_tokens, Hv]      fp32
 *   S0         [num_seqs, Hv, dk, dv]  fp32, or NULL for zero start states
 *   cu_seqlens [num_seqs + 1]          int32, device; 0 = c_0 <= ... <= c_N = total_tokens
 *   o          [total_tokens, Hv, dv]  qkv_dtype (out)
 *   S_final    [num_seqs, Hv, dk, dv]  fp32 (out), or NULL
 *   workspace  >= kda_gdn_prefill_workspace_bytes(...), else KDA_ERR_WORKSPACE
 *              (bf16: about 0.4 KB per token and value head and 26 KB per
 *              sequence and value head)
 *
 * Sequences, start and final states, aliasing (S_final may be S0 exactly, no
 * other overlap) and errors are those of kda_prefill.  A malformed cu_seqlens
 * sets KDA_DEV_BAD_CU_SEQLENS; sequences with invalid bounds are not written,
 * and others may not be.  Results are bitwise repeatable.
 * fp32 inputs and short sequences go token by token, and o is rounded once; in
 * chunks of 64 it is rounded to bf16 from products whose operands are.  Short
 * is one sequence of up to 16 tokens, and several of up to 8 tokens on average
 * and 240 + num_seqs * Hv / 8 in all: the same sequence may get either o,
 * depending on what it is packed with.
 * Inputs that are not finite reach the outputs of their token and of later ones
 * of their sequence, and in chunks also up to 15 earlier ones: those of the same
 * 16 tokens, counted from the sequence's start (the products with T and P go
 * over whole 16 x 16 blocks, and 0 times NaN is NaN).
 */
KDA_API kda_status kda_gdn_prefill(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                   const float *log_decay, const float *beta, const float *S0,
                                   const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t Hk,
                                   int32_t Hv, int32_t dk, int32_t dv, void *o, float *S_final, void *workspace,
                                   size_t workspace_bytes, int32_t *device_status, kda_stream_t stream);

/*
 * kda_gdn_prefill_backward -- reverse-mode gradient of kda_gdn_prefill for
 *     L = sum_{t,h,j} o[t,h,j] grad_o[t,h,j] + sum_{n,h,i,j} S_final grad_S_final.
 *
 *   q, k, v, log_decay, beta, S0, cu_seqlens, num_seqs, total_tokens, Hk, Hv,
 *   dk, dv        the forward's inputs (S0 may be NULL = zeros)
 *   grad_o        [total_tokens, Hv, dv] qkv_dtype, device (dL/do)
 *   grad_S_final  [num_seqs, Hv, dk, dv] fp32 device, or NULL (zeros)
 *   grad_q, grad_k  [total_tokens, Hk, dk] qkv_dtype out: the value heads of a
 *                   group are added in fp32 and rounded once
 *   grad_v        [total_tokens, Hv, dv] qkv_dtype out
 *   grad_log_decay, grad_beta  [total_tokens, Hv] fp32 out
 *   grad_S0       [num_seqs, Hv, dk, dv] fp32 out, or NULL (not computed)
 *
 * qkv_dtype is KDA_DTYPE_BF16 (else KDA_ERR_UNSUPPORTED).  The call reruns the
 * chunkwise forward, keeping the state before every 64-token chunk, walks the
 * state's adjoint back over the chunks, and forms everything else per chunk.
 * Up to two tokens a sequence and six more go token by token, in fp32, but no
 * more than 64 + num_seqs * Hv / 20 in all.
 * The fp32 gradients are accurate as S_final is; results are bitwise
 * repeatable.  The gradient of a log_decay at which the decay is 0 in fp32 is 0.
 *
 * Workspace: >= kda_gdn_prefill_backward_workspace_bytes(...) device bytes
 * (about 3.5 KB per token and value head and 220 KB per sequence and value
 * head; 64 KB per token and value head where it goes token by token), enough
 * for every call with as many tokens and sequences or fewer, 256-byte aligned.
 * q, k, v, grad_o, states and their gradients are 16-byte aligned, the others
 * 4.  The outputs overlap nothing (KDA_ERR_INVALID_ARG).  A malformed cu_seqlens sets
 * KDA_DEV_BAD_CU_SEQLENS and leaves the gradients unspecified.
 */
KDA_API size_t kda_gdn_prefill_backward_workspace_bytes(kda_dtype qkv_dtype, int32_t num_seqs, int64_t total_tokens,
                                                        int32_t Hk, int32_t Hv, int32_t dk, int32_t dv);
KDA_API kda_status kda_gdn_prefill_backward(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                            const float *log_decay, const float *beta, const float *S0,
                                            const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                            int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, const void *grad_o,
                                            const float *grad_S_final, void *grad_q, void *grad_k, void *grad_v,
                                            float *grad_log_decay, float *grad_beta, float *grad_S0,
                                            void *workspace, size_t workspace_bytes, int32_t *device_status,
                                            kda_stream_t stream);

/*
 * kda_gdn_decode_step -- one token of the gated delta rule for N sequences;
 * each head's state is read once and written once, in place.
 *
 *   q, k       [N, Hk, dk]  qkv_dtype        v [N, Hv, dv] qkv_dtype
 *   log_decay  [N, Hv] fp32                  beta [N, Hv] fp32
 *   S          [num_slots, Hv, dk, dv] fp32, updated in place
 *   state_indices, device_status             as kda_decode_step
 *   o          [N, Hv, dv]  qkv_dtype (out)
 */
KDA_API kda_status kda_gdn_decode_step(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                       const float *log_decay, const float *beta, float *S, int32_t num_slots,
                                       const int32_t *state_indices, int32_t N, int32_t Hk, int32_t Hv, int32_t dk,
                                       int32_t dv, void *o, int32_t *device_status, kda_stream_t stream);

/*
 * kda_rms_norm -- the norm in front of a layer's projections ("Inside one KDA
 * block" of "Understanding Kimi Delta Attention" (pyshine) begins with it),
 * with the residual stream's addition and an optional output in 8 bits:
 *
 *   h = round(x + residual)  (h = x when residual is NULL)
 *   y = h / sqrt(mean_c h_c^2 + eps) * weight
 *
 *   x, residual, residual_out  [rows, dim] dtype; residual_out (out, or NULL)
 *              receives h; it may be x or residual exactly
 *   weight     [dim] fp32 (NULL = all ones)
 *   y          [rows, dim] (out): KDA_NORM_OUT_SAME in dtype (may be x
 *              exactly); KDA_NORM_OUT_E4M3 or KDA_NORM_OUT_INT8 one byte each
 *   group      8-bit outputs: 0 = one scale for a row, 128 = one for every 128
 *              columns (dim a multiple of 128)
 *   scales     [rows, group ? dim / group : 1] fp32 (out), 8-bit outputs only:
 *              max(max |y| / qmax, 2^-126), qmax = 448 (e4m3) or 127 (int8).
 *              The code is y / scale rounded to nearest even (both quotients
 *              as products with the reciprocal, in fp32); it stands for
 *              code * scale.  Values that are not finite make the scale they
 *              share NaN (a y of infinity: infinite).
 *
 * x, residual, residual_out, y 16-byte aligned, weight and scales 4-byte; dim
 * from 1 to KDA_NORM_MAX_DIM.  Outputs overlap nothing but as said above
 * (KDA_ERR_INVALID_ARG).  Asynchronous on `stream`, no workspace; results are
 * bitwise repeatable.
 */
#define KDA_NORM_MAX_DIM (1 << 20)
typedef enum {
    KDA_NORM_OUT_SAME = 0,
    KDA_NORM_OUT_E4M3 = 1,
    KDA_NORM_OUT_INT8 = 2
} kda_norm_out;
KDA_API kda_status kda_rms_norm(const void *x, const void *residual, kda_dtype dtype, const float *weight, float eps,
                                int64_t rows, int32_t dim, kda_norm_out out_type, int32_t group, void *y,
                                float *scales, void *residual_out, kda_stream_t stream);

/*
 * kda_rms_norm_backward -- gradient of kda_rms_norm's y (KDA_NORM_OUT_SAME)
 * and h for L = <y, grad_y> + <h, grad_h>, with r = (mean_c h_c^2 + eps)^(-1/2):
 *     grad_x_c = r w_c dy_c - (r^3 h_c / dim) sum_j h_j w_j dy_j + grad_h_c
 * (the gradient of x and of residual alike) and grad_weight_c = sum over rows
 * of dy_c h_c r.
 *
 *   grad_y, h, grad_h  [rows, dim] dtype; h as the forward stored it; grad_h
 *                      may be NULL (zeros)
 *   grad_x             [rows, dim] dtype (out; may be grad_y or grad_h exactly)
 *   grad_weight        [dim] fp32 (out), 16-byte aligned, or NULL (not computed);
 *                      rows are added in a fixed order (bitwise repeatable)
 *   workspace          >= kda_rms_norm_backward_workspace_bytes(rows, dim) when
 *                      grad_weight is given, 256-byte aligned, else it may be NULL
 */
KDA_API size_t kda_rms_norm_backward_workspace_bytes(int64_t rows, int32_t dim);
KDA_API kda_status kda_rms_norm_backward(const void *grad_y, const void *h, const void *grad_h, kda_dtype dtype,
                                         const float *weight, float eps, int64_t rows, int32_t dim, void *grad_x,
                                         float *grad_weight, void *workspace, size_t workspace_bytes,
                                         kda_stream_t stream);

/*
 * The gated linear recurrence: the diagonal member of the family, a state of
 * one number for each channel instead of a 128 x 128 matrix for each head:
 *
 *   h_t = a_t h_{t-1} + s_t x_t       for every channel by itself
 *   a_t = exp(gate_t), or with KDA_GLR_SIGMOID 1 / (1 + exp(-gate_t))
 *   s_t = 1, or with KDA_GLR_COMPLEMENT 1 - a_t
 *
 * x, h [tokens, dim] in dtype; gate [tokens, dim] in gate_dtype, which is dtype
 * or KDA_DTYPE_F32 (else KDA_ERR_UNSUPPORTED); states [.., dim] fp32.  dim from
 * 1 to KDA_GLR_MAX_DIM, tokens, sequences and slots up to 2^31 - 65537.  Unknown
 * flags return KDA_ERR_INVALID_ARG.  Tensors and states are 16-byte aligned,
 * cu_seqlens, state_indices and device_status 4.
 *
 * States, decays and sums are fp32; every output is rounded once.  The step is
 * taken with 1 - a_t, held to 2^-20 of its value, so a channel with a memory of
 * many tokens keeps its accuracy; decays, 1 - a_t and slopes below fp32's normal
 * numbers count as 0.  Prefill and its gradient take up to 128 tokens
 * together: a state is off by a few 2^-24 of the largest one among the 128 tokens
 * before it (in the gradient: behind it), which is more than its own rounding
 * where a channel forgets a large state faster than that; decays of exactly 0
 * forget it exactly.  The single token (kda_glr_decode_step) keeps a_t h_{t-1} to
 * 2^-19 of its own value.  Results are bitwise repeatable.
 * Gates above 0 of the exp kind are growth.  Prefill and its gradient take them
 * while the product of any 128 consecutive tokens' decays is finite (gates that
 * add up to less than 88); beyond that they may give NaN where the recurrence is
 * finite, a state of 0 among them.  1 - a_t is then good to (22 + 1.25 gate_t)
 * 2^-24 of its value.
 * Inputs that are not finite reach the outputs of their token and of later ones
 * (in the gradient: earlier ones) of their sequence and channel; an infinite
 * state becomes NaN at the next token of prefill, while the single token has
 * a_t times it.
 */
#define KDA_GLR_SIGMOID 0x1u
#define KDA_GLR_COMPLEMENT 0x2u
#define KDA_GLR_MAX_DIM (1 << 20)
#define KDA_GLR_CHECKPOINT 64

/*
 * kda_glr_prefill -- the recurrence over packed variable-length sequences.
 *
 *   h0          [num_seqs, dim] fp32, or NULL for zero start states
 *   cu_seqlens  [num_seqs + 1] int32, device; 0 = c_0 <= ... <= c_N = total_tokens
 *   h           [total_tokens, dim] dtype (out)
 *   h_final     [num_seqs, dim] fp32 (out), or NULL; may be h0 exactly
 *   checkpoints [ceil(total_tokens / KDA_GLR_CHECKPOINT), dim] fp32 (out), or
 *               NULL: the state before every KDA_GLR_CHECKPOINT-th of the packed
 *               tokens (that of the sequence which the token before belongs to),
 *               for kda_glr_prefill_backward
 *
 * A sequence without tokens has h_final = h0.  No other overlap between an
 * output and another buffer (KDA_ERR_INVALID_ARG).  A malformed cu_seqlens sets
 * KDA_DEV_BAD_CU_SEQLENS and leaves the outputs unspecified.  One pass, no
 * workspace.
 */
KDA_API kda_status kda_glr_prefill(const void *x, kda_dtype dtype, const void *gate, kda_dtype gate_dtype, uint32_t flags,
                                   const float *h0, const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                   int32_t dim, void *h, float *h_final, float *checkpoints, int32_t *device_status,
                                   kda_stream_t stream);

/*
 * kda_glr_prefill_backward -- reverse-mode gradient of kda_glr_prefill for
 *     L = sum_{t,c} h[t,c] grad_h[t,c] + sum_{n,c} h_final grad_h_final.
 *
 *   x, gate, flags, h0, cu_seqlens, ..., dim   the forward's inputs
 *   grad_h        [total_tokens, dim] dtype, device (dL/dh)
 *   grad_h_final  [num_seqs, dim] fp32, device, or NULL (zeros)
 *   checkpoints   what the forward of these inputs stored, or NULL: the call then
 *                 runs it again for them, into its workspace
 *   grad_x        [total_tokens, dim] dtype (out)
 *   grad_gate     [total_tokens, dim] gate_dtype (out)
 *   grad_h0       [num_seqs, dim] fp32 (out), or NULL (not computed)
 *   workspace     without checkpoints: >= kda_glr_prefill_backward_workspace_bytes
 *                 device bytes, 256-byte aligned (KDA_ERR_WORKSPACE below it),
 *                 enough for every call with as many tokens or fewer; else it
 *                 may be NULL
 *
 * The outputs overlap nothing (KDA_ERR_INVALID_ARG).  A malformed cu_seqlens sets
 * KDA_DEV_BAD_CU_SEQLENS and leaves the gradients unspecified.
 */
KDA_API size_t kda_glr_prefill_backward_workspace_bytes(int64_t total_tokens, int32_t dim);
KDA_API kda_status kda_glr_prefill_backward(const void *x, kda_dtype dtype, const void *gate, kda_dtype gate_dtype,
                                            uint32_t flags, const float *h0, const int32_t *cu_seqlens, int32_t num_seqs,
                                            int64_t total_tokens, int32_t dim, const void *grad_h,
                                            const float *grad_h_final, const float *checkpoints, void *grad_x,
                                            void *grad_gate, float *grad_h0, void *workspace, size_t workspace_bytes,
                                            int32_t *device_status, kda_stream_t stream);

/*
 * kda_glr_decode_step -- one token of it for N sequences; each state is read
 * once and written once, in place.
 *
 *   x, h  [N, dim] dtype        gate [N, dim] gate_dtype
 *   state [num_slots, dim] fp32, updated in place
 *   state_indices, device_status   as kda_decode_step
 */
KDA_API kda_status kda_glr_decode_step(const void *x, kda_dtype dtype, const void *gate, kda_dtype gate_dtype,
                                       uint32_t flags, float *state, int32_t num_slots, const int32_t *state_indices,
                                       int32_t N, int32_t dim, void *h, int32_t *device_status, kda_stream_t stream);

/*
 * Products in 8-bit floats: e4m3 codes with an fp32 scale for every 128 of
 * them, as kda_rms_norm writes its rows (KDA_NORM_OUT_E4M3, group 128).  A code
 * stands for code * scale; the scales of a tensor [rows, cols] are
 *
 *   KDA_FP8_ROWS     [rows, ceil(cols / 128)]             128 of a row share one
 *   KDA_FP8_BLOCKS   [ceil(rows / 128), ceil(cols / 128)] 128 x 128 share one
 *   KDA_FP8_COLUMNS  kda_fp8_quantize only: the transposed codes [cols, rows]
 *                    with their KDA_FP8_ROWS scales [cols, ceil(rows / 128)]
 *
 * A layer's three products are y = x W^T, dx = dy W and dW = dy^T x, all of them
 * rows times rows: dx takes the transposed codes and scales of W (blocks stay
 * blocks), dW takes dy and x as KDA_FP8_COLUMNS makes them.  K, of which the
 * products take multiples of 16, is W's number of rows in dx and that of tokens
 * in dW: others are filled up with zeros before they are quantised (rows of W
 * and columns of dy; rows of dy and x), which changes no scale and no code.
 */
#define KDA_FP8_BLOCK 128
#define KDA_FP8_MAX_DIM (1 << 24)
typedef enum {
    KDA_FP8_BLOCKS = 0,
    KDA_FP8_ROWS = 1,
    KDA_FP8_COLUMNS = 2
} kda_fp8_scales;

/*
 * kda_fp8_matmul -- out = x w^T:
 *   out[m, n] = sum_b xs[m, b] ws[n, b] sum_{k in block b} x[m, k] w[n, k]
 *
 *   x         [M, K] e4m3            x_scales [M, ceil(K / 128)] fp32
 *   w         [N, K] e4m3            w_scales fp32, by w_form: KDA_FP8_BLOCKS or
 *             KDA_FP8_ROWS
 *   out       [M, N] out_dtype (out)
 *
 * M >= 0, N from 1 to KDA_FP8_MAX_DIM, K a multiple of 16 up to it (others:
 * KDA_ERR_UNSUPPORTED); x, w and out 16-byte aligned, the others 4.  A block's
 * products are summed by the tensor cores in fp32, blocks are added in fp32 after
 * their scales, and out is rounded once.  The two scales of a block are multiplied
 * with each other first: xs ws has to lie in fp32's range, below its normal
 * numbers it loses bits.  Results are bitwise repeatable.  A
 * scale or code that is not finite spoils the outputs of its row (column of out
 * for w) only.  out overlaps nothing (KDA_ERR_INVALID_ARG).  Asynchronous, no
 * workspace.
 */
KDA_API kda_status kda_fp8_matmul(const void *x, const float *x_scales, const void *w, const float *w_scales,
                                  kda_fp8_scales w_form, int64_t M, int32_t N, int32_t K, kda_dtype out_dtype, void *out,
                                  int32_t *device_status, kda_stream_t stream);

/*
 * kda_fp8_matmul_grouped -- the same for rows that are packed by expert:
 *   out[m] = x[m] w[e]^T for the rows offsets[e] <= m < offsets[e + 1] of expert e
 *
 *   x        [rows, K] e4m3          x_scales [rows, ceil(K / 128)] fp32
 *   w        [num_experts, N, K]     w_scales [num_experts, ..] as above for each
 *   offsets  [num_experts + 1] int32, device; 0 = o_0 <= ... <= o_E <= rows
 *   out      [rows, N] out_dtype (out); rows from o_E on are left as they are
 *
 * Malformed offsets set KDA_DEV_BAD_CU_SEQLENS and leave the outputs
 * unspecified; without rows nothing is launched and they are not read.  Else as
 * kda_fp8_matmul.
 */
KDA_API kda_status kda_fp8_matmul_grouped(const void *x, const float *x_scales, const void *w, const float *w_scales,
                                          kda_fp8_scales w_form, const int32_t *offsets, int32_t num_experts, int64_t rows,
                                          int32_t N, int32_t K, kda_dtype out_dtype, void *out, int32_t *device_status,
                                          kda_stream_t stream);

/*
 * kda_fp8_quantize -- x in e4m3 with its scales, as laid out above:
 *   scale = max(max |x| / 448, 2^-126) over what shares it, code = x / scale
 * rounded to nearest even (both fp32 quotients, rounded once; a code of zero may
 * have either sign).  A NaN makes the scale it shares NaN, an infinity infinite.
 *
 *   x       [rows, cols] dtype       codes  rows x cols bytes (out)
 *   scales  fp32 (out)
 * x and codes 16-byte aligned, scales 4.  The outputs overlap nothing
 * (KDA_ERR_INVALID_ARG).
 */
KDA_API kda_status kda_fp8_quantize(const void *x, kda_dtype dtype, int64_t rows, int64_t cols, kda_fp8_scales form,
                                    void *codes, float *scales, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
