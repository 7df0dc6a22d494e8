/*
 * kda.h -- C ABI of the MI355X (gfx950) Kimi Delta Attention forward library (libkda.so).
 *
 * The operation is the chunked forward pass of KDA as the "Kernel API" table of the
 * FlashKDA README ("MoonshotAI/FlashKDA" repository page) states it (plus, in kda_bwd,
 * its gradients):
 *
 *   fwd(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound,
 *       initial_state=None, final_state=None, cu_seqlens=None)
 *
 * with the in-kernel gate activation, q/k l2 normalisation and beta sigmoid that the
 * README section "Using FlashKDA as an FLA backend" switches on (use_gate_in_kernel,
 * use_qk_l2norm_in_kernel, use_beta_sigmoid_in_kernel, safe_gate) and the V-major state
 * layout it selects (transpose_state_layout).  Per (sequence, head) chain, per token:
 *   q^ = q/sqrt(|q|^2+1e-6), k^ = k/sqrt(|k|^2+1e-6), beta = sigmoid(beta_logit),
 *   a_c = lower_bound * sigmoid(exp(A_log[h]) * (g_c + dt_bias[h,c])),
 *   S <- S Diag(exp(a)),  S <- S + beta (v - S k^) k^T,  out = scale * S q^.
 * The library evaluates this in 16-token chunks (FlashKDA article index: "processes
 * 16-token chunks"; "Neumann-series expansion" for the intra-chunk inverse).
 *
 * Beside it: kda_gdn_*, the gated delta rule with one decay per head instead of one per channel, and kda_lin_*,
 * linear attention with one decay per head (no delta rule), each
 * forward, token by token and backward, on the same state layout; and kda_qk_rope*, the
 * normalisation of q and k with the rotation by positions, which prepares the inputs of either; and kda_gated_norm*,
 * kda_residual_norm*, what follows a mixer: the norm of its heads with their gate, and the step to the next block.
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers unless the name ends in _host.
 *   - The caller owns every buffer; the library allocates no device memory.  Scratch
 *     space comes from the caller's workspace (size from kda_fwd_workspace_size), except
 *     for kda_fwd_noalloc, which uses a static device array of the library.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream) and runs
 *     asynchronously; no entry point synchronises the host except kda_fwd_device_status.
 *   - Arguments are fully validated on the host before anything is launched; on any
 *     error nothing is launched and an error status is returned.  Nothing throws.
 *   - No global mutable state besides kda_fwd_noalloc's scratch and its per-device
 *     address; the other entry points are safe to call from several host threads on
 *     different streams with different workspaces.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_HEAD_DIM 128 /* K = V = 128 is the only supported head size (Kernel API table) */
#define KDA_CHUNK 16     /* tokens per chunk */

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_NULL = 1,        /* A_log or dt_bias is NULL (in-pass gate), or a token tensor is NULL while T > 0 */
    KDA_ERR_SHAPE = 2,       /* B < 1, T < 0, H < 1, N inconsistent or >= 2^29, or cu_seqlens with B != 1 */
    KDA_ERR_HEAD_DIM = 3,    /* K or V is not 128; kda_gated_norm*, kda_residual_norm*: D not supported */
    KDA_ERR_DTYPE = 4,       /* state dtype unknown, or initial/final state dtypes differ */
    KDA_ERR_LOWER_BOUND = 5, /* lower_bound not finite or outside [-5, 0] */
    KDA_ERR_SCALE = 6,       /* scale not finite */
    KDA_ERR_ALIGN = 7,       /* a pointer misses its alignment (see kda_fwd) */
    KDA_ERR_WORKSPACE = 8,   /* workspace NULL or smaller than kda_fwd_workspace_size */
    KDA_ERR_CU_SEQLENS = 9,  /* cu_seqlens_host given and cu[0] != 0, decreasing, or cu[N] != T */
    KDA_ERR_HIP = 10,        /* a HIP launch or query failed */
    KDA_ERR_ALIAS = 11,      /* out overlaps an input, or final_state overlaps a non-state input */
    KDA_ERR_FLAGS = 12,      /* kda_fwd_ex: unknown bits in the activation switch mask */
    KDA_ERR_SCRATCH = 13,    /* kda_fwd_noalloc: the call needs more than KDA_NOALLOC_SCRATCH_BYTES */
    KDA_ERR_HEADS = 14,      /* kda_lin_*, kda_gdn_*: H is not a multiple of Hk, or Hk < 1 */
    KDA_ERR_STRIDE = 15,     /* kda_lin_*, kda_gdn_*, kda_qk_rope*, norms: a stride is negative, no multiple of 16 bytes, or too large */
    KDA_ERR_ROTARY = 16      /* kda_qk_rope*: head size or rotary_dim not supported */
} kda_status;

typedef enum kda_state_dtype {
    KDA_STATE_NONE = 0, /* pointer is NULL: no initial state (zeros) / final state not written */
    KDA_STATE_BF16 = 1,
    KDA_STATE_FP32 = 2
} kda_state_dtype;

/*
 * kda_fwd -- chunked KDA forward pass (Kernel API table of the FlashKDA README).
 *
 *   q, k, g   bf16 [B, T, H, 128], contiguous, 16-byte aligned.  Query, key, gate before
 *             activation.
 *   v         bf16 [B, T, H, 128], contiguous, 16-byte aligned.
 *   beta      bf16 [B, T, H], contiguous, 2-byte aligned.  Beta logits (sigmoid applied here).
 *   scale     output scaling factor, finite.
 *   out       bf16 [B, T, H, 128], contiguous, 16-byte aligned; fully overwritten (every
 *             token of every sequence).  Must not overlap any input.
 *   A_log     fp32 [H], 4-byte aligned.   dt_bias  fp32 [H, 128], 16-byte aligned.
 *   lower_bound  gate lower bound in [-5, 0] (the table's stated range); the per-token
 *             log-decay lies in (lower_bound, 0].
 *   initial_state  NULL (zeros) or [N, H, 128(V), 128(K)] of initial_state_dtype, 16-byte aligned.
 *   final_state    NULL (not written) or [N, H, 128(V), 128(K)] of final_state_dtype,
 *             16-byte aligned.  May be the same buffer as initial_state (in-place state carry).
 *             bf16 states are widened on load and rounded (nearest-even) once on store.
 *   initial_state_dtype / final_state_dtype  KDA_STATE_NONE exactly when the pointer is NULL;
 *             when both states are given the two dtypes must be equal (KDA_ERR_DTYPE).
 *   cu_seqlens  NULL, or device int64 [N+1] cumulative sequence lengths (8-byte aligned);
 *             then B must be 1, T is the total length and sequence i is tokens
 *             [cu[i], cu[i+1]).  Without it each of the B batch rows is one sequence (N = B;
 *             pass N = B or N = 0).
 *   cu_seqlens_host  optional host copy of cu_seqlens.  When given, its content is checked
 *             synchronously (KDA_ERR_CU_SEQLENS).  Without it the device checks the content;
 *             an invalid cu_seqlens then turns every sequence into an empty one (out is not
 *             written, final_state = initial_state or zeros) and sets the device status word
 *             that kda_fwd_device_status reads.
 *   B, T, H, N  sizes as above.  K, V must both be 128.
 *   workspace, workspace_bytes  device scratch, 256-byte aligned, at least
 *             kda_fwd_workspace_size(B, T, H, N, cu_seqlens != NULL) bytes.  It must not be
 *             used by another call until this one has finished on the stream.
 *   stream    hipStream_t (NULL = default stream).
 * Returns KDA_OK once the work is enqueued, or the first validation error found.
 */
kda_status kda_fwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                   float scale, void *out, const float *A_log, const float *dt_bias,
                   float lower_bound, const void *initial_state, kda_state_dtype initial_state_dtype,
                   void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                   const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t H, int64_t N,
                   int64_t K, int64_t V, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Activation switches for kda_fwd_ex, after the use_gate_in_kernel, use_qk_l2norm_in_kernel
 * and use_beta_sigmoid_in_kernel flags the README section "Using FlashKDA as an FLA backend"
 * passes to chunk_kda (the pages name them and set all three; kda_fwd is the all-set case).
 * A switch that is off means that input arrives already activated:
 *   KDA_GATE_IN_KERNEL off:   g holds the per-token, per-channel natural-log decay a itself
 *                             (bf16 [B, T, H, 128]); the pass uses min(max(a, lower_bound), 0),
 *                             the range the in-pass gate produces.  A_log and dt_bias are
 *                             not read and may be NULL.
 *   KDA_QK_L2NORM_IN_KERNEL off: q and k are used as given (no l2 normalisation).
 *   KDA_BETA_SIGMOID_IN_KERNEL off: beta is the write strength itself (no sigmoid).
 */
#define KDA_GATE_IN_KERNEL 1u
#define KDA_QK_L2NORM_IN_KERNEL 2u
#define KDA_BETA_SIGMOID_IN_KERNEL 4u
#define KDA_ALL_IN_KERNEL 7u

/*
 * kda_fwd_ex -- kda_fwd with the activation switch mask `flags` (KDA_*_IN_KERNEL bits).
 * Same arguments, layouts, ownership and errors as kda_fwd, plus KDA_ERR_FLAGS for bits
 * outside KDA_ALL_IN_KERNEL.  With KDA_GATE_IN_KERNEL clear, A_log and dt_bias may be NULL
 * (they are then not checked for alignment either); lower_bound is still checked and
 * bounds the pre-activated log-decay.  kda_fwd(...) is kda_fwd_ex(..., KDA_ALL_IN_KERNEL).
 */
kda_status kda_fwd_ex(const void *q, const void *k, const void *v, const void *g, const void *beta,
                      float scale, void *out, const float *A_log, const float *dt_bias,
                      float lower_bound, const void *initial_state, kda_state_dtype initial_state_dtype,
                      void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                      const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t H, int64_t N,
                      int64_t K, int64_t V, void *workspace, size_t workspace_bytes, void *stream,
                      uint32_t flags);

/*
 * kda_fwd_recurrent -- the same forward pass evaluated token by token (the recurrence the
 * FlashKDA article index calls the linear-time recurrence), for short sequences: the decode
 * step (one token per sequence, state in and out, often in place) and sequences of a few
 * tokens.  Same arguments, layouts, ownership, errors and activation switches as kda_fwd_ex,
 * and the same workspace (kda_fwd_workspace_size).  One workgroup per (sequence, head)
 * keeps the 128 x 128 state in fp32 registers and walks the sequence's tokens in order, so
 * its time grows with the longest sequence; for sequences longer than a few chunks use
 * kda_fwd.  Results agree with kda_fwd to the same tolerance against the fp64 recurrence
 * (this path is all fp32; kda_fwd uses split-bf16 matrix products).
 */
kda_status kda_fwd_recurrent(const void *q, const void *k, const void *v, const void *g, const void *beta,
                             float scale, void *out, const float *A_log, const float *dt_bias,
                             float lower_bound, const void *initial_state,
                             kda_state_dtype initial_state_dtype, void *final_state,
                             kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                             const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t H, int64_t N,
                             int64_t K, int64_t V, void *workspace, size_t workspace_bytes, void *stream,
                             uint32_t flags);

/*
 * kda_fwd_recurrent_timed -- kda_fwd_recurrent with stage timing, for measurement: three
 * hipEvent_t handles (created by the caller) recorded on `stream` before the chunk-table
 * kernel, before the recurrent kernel and after it.  Returns KDA_ERR_NULL if any of the
 * three is NULL.
 */
kda_status kda_fwd_recurrent_timed(const void *q, const void *k, const void *v, const void *g,
                                   const void *beta, float scale, void *out, const float *A_log,
                                   const float *dt_bias, float lower_bound, const void *initial_state,
                                   kda_state_dtype initial_state_dtype, void *final_state,
                                   kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                                   const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t H,
                                   int64_t N, int64_t K, int64_t V, void *workspace,
                                   size_t workspace_bytes, void *stream, uint32_t flags,
                                   void *const *stage_events);

/*
 * kda_fwd_timed -- kda_fwd with stage timing, for measurement.  Same arguments and behaviour
 * as kda_fwd, plus stage_events: five hipEvent_t handles (created by the caller), recorded
 * on `stream`:
 *   [0] before the chunk-table kernel
 *   [1] before the first forward-kernel launch
 *   [2] after it (with the cut plan: after pass A and the transition runs)
 *   [3] after the cut scan (recorded right after [2] when there is none)
 *   [4] after pass B (right after [3] when there is none)
 * With the whole-chain plans (see kda_fwd_workspace_size) the forward kernel runs once;
 * with the cut plan, pass A, the transition runs, the scan and pass B.  hipEventElapsedTime
 * between consecutive events gives each stage's duration.  Returns KDA_ERR_NULL if any of
 * the five handles is NULL.
 */
kda_status kda_fwd_timed(const void *q, const void *k, const void *v, const void *g, const void *beta,
                         float scale, void *out, const float *A_log, const float *dt_bias,
                         float lower_bound, const void *initial_state,
                         kda_state_dtype initial_state_dtype, void *final_state,
                         kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                         const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t H, int64_t N,
                         int64_t K, int64_t V, void *workspace, size_t workspace_bytes, void *stream,
                         void *const *stage_events);

/*
 * kda_fwd_noalloc -- kda_fwd_ex for callers that cannot allocate device memory: code under
 * stream capture, tight serving loops, harnesses that forbid hipMalloc.  Same arguments,
 * layouts, ownership, activation switches, results and errors as kda_fwd_ex, without the
 * workspace arguments: the library's own static device scratch of KDA_NOALLOC_SCRATCH_BYTES
 * (64 MiB; one copy on every GPU the library runs on, held until the process ends) serves
 * as the workspace.  The call allocates nothing.
 *   - Returns KDA_ERR_SCRATCH, before any HIP call, when kda_fwd_workspace_size for these
 *     sizes exceeds KDA_NOALLOC_SCRATCH_BYTES (e.g. very many sequences).
 *   - The scratch belongs to the device of `stream` (the current device for NULL); its
 *     address is looked up once per device.  Calls on one GPU share it: two calls that
 *     overlap in time on one GPU (different streams, or host threads) race and give
 *     undefined results; serialise them.  Every word a call reads from the scratch is
 *     written earlier in the same call, so nothing needs clearing between calls.
 *   - kda_fwd_device_status cannot read this call's status word (it is not in a caller's
 *     buffer); validation errors are still returned.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
kda_status kda_fwd_noalloc(const void *q, const void *k, const void *v, const void *g, const void *beta,
                           float scale, void *out, const float *A_log, const float *dt_bias,
                           float lower_bound, const void *initial_state, kda_state_dtype initial_state_dtype,
                           void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                           const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t H, int64_t N,
                           int64_t K, int64_t V, void *stream, uint32_t flags);

/*
 * kda_fwd_workspace_size -- bytes of workspace kda_fwd needs: the status word, the
 * per-sequence chunk table (start, length, chunk offset), O(N) bytes, a fixed 2.25 KiB
 * table of the first unit of each workgroup and the unit list (8 bytes per sequence) that
 * spreads the sequences over the workgroups with about equal chunk counts (a long sequence
 * of a varlen batch may run as two units of 64 value columns each), and a fixed 3.25 KiB
 * cut table.  When sequences are long on average (at least 64 chunks of 16 tokens, about
 * ceil(T / 16) / N for varlen) and H <= 128, the cut plan gives each head P = min(256 / H,
 * C / 16) workgroups (C = the head's chunk count, ceil(T / 16) for varlen) that take equal
 * runs of its chunks, cutting sequences where needed (the state after a piece is affine
 * in the state before it); that adds three fp32 128 x 128 states per head and cut,
 * 3 * H * P * 64 KiB, plus 40 bytes per head and cut.  P is a deterministic function of
 * (B, T, H, N, has_cu_seqlens).  The per-chunk operands never leave the chip.  Returns 0
 * for invalid sizes.
 */
size_t kda_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens);

/*
 * kda_bwd -- gradients of kda_fwd_ex's outputs (out and final_state) with respect to its
 * inputs, for training.  The pages describe the forward pass only; this is the reverse-mode
 * derivative of the same per-token recurrence (stated in the comment at the top of this
 * file), under the same activation switches.  All arithmetic is fp32 (the products with the
 * states as three-term bf16 products with fp32 accumulation, about 16 significant bits per
 * factor, as in kda_fwd's chunk recurrence); the inputs q, k, v,
 * g, beta, scale, A_log, dt_bias, lower_bound, initial_state, cu_seqlens, B, T, H, N, K, V
 * and flags mean exactly what they mean for kda_fwd_ex.
 *   dout          bf16 [B, T, H, 128], 16-byte aligned: dL/dout.
 *   dfinal_state  NULL (zero) or fp32 [N, H, 128, 128], 16-byte aligned: dL/dfinal_state.
 *   dq, dk, dv, dg  fp32 [B, T, H, 128], 16-byte aligned, fully written: dL/dq, dL/dk,
 *                 dL/dv and dL/dg (with the gate switch off, g is the log-decay itself and
 *                 its gradient is zero where g lies outside (lower_bound, 0)).
 *   dbeta         fp32 [B, T, H], 4-byte aligned: dL/dbeta (the logit when the sigmoid runs
 *                 in the pass).
 *   dA_log        NULL or fp32 [H]; ddt_bias  NULL or fp32 [H, 128] (16-byte aligned):
 *                 summed over every token of every sequence.  Written only with the gate
 *                 switch on (KDA_GATE_IN_KERNEL); NULL = not written.
 *   dinitial_state  NULL (not written) or fp32 [N, H, 128, 128], 16-byte aligned: dL/d
 *                 initial_state (also when initial_state is NULL, i.e. zero).
 *   workspace     device scratch of at least kda_bwd_workspace_size(...) bytes, 256-byte
 *                 aligned.
 * An invalid cu_seqlens (found on the device) makes every sequence empty, as in kda_fwd:
 * dq, dk, dv, dg and dbeta are not written, dA_log and ddt_bias are zero, and
 * dinitial_state = dfinal_state (or zero); kda_fwd_device_status on the workspace reports it.
 * Outputs must not overlap any input or each other (KDA_ERR_ALIAS).  Same error codes as
 * kda_fwd_ex otherwise.  Work is enqueued on `stream`; nothing is allocated.  The pass runs
 * in 16-token chunks: the state runs forwards and dL/dS backwards over the chunks of each
 * (sequence, head), and the tokens' gradients are formed per chunk in parallel.  Where the
 * sequences are few and long (64 chunks or more on average), both walks are cut into pieces
 * that run in parallel and are joined by an affine scan (with the in-kernel l2norm and
 * sigmoid, a start state's share that has fallen below 2^-30 of a piece's own end state is
 * dropped, as in kda_fwd's cut plan).  Results are deterministic: fixed summation orders,
 * no atomics.
 */
kda_status kda_bwd(const void *q, const void *k, const void *v, const void *g, const void *beta, float scale,
                   const float *A_log, const float *dt_bias, float lower_bound, const void *initial_state,
                   kda_state_dtype initial_state_dtype, const void *dout, const float *dfinal_state, float *dq,
                   float *dk, float *dv, float *dg, float *dbeta, float *dA_log, float *ddt_bias,
                   float *dinitial_state, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host, int64_t B,
                   int64_t T, int64_t H, int64_t N, int64_t K, int64_t V, void *workspace,
                   size_t workspace_bytes, void *stream, uint32_t flags);

/*
 * kda_bwd_workspace_size -- bytes of workspace kda_bwd needs: the chunk table, then per
 * 16-token chunk of each head (counted as ceil(T / 16) per batch row, or ceil(T / 16) + N
 * with cu_seqlens) 33.5 KiB of chunk operands, one fp32 state (64 KiB: the state before the
 * chunk for the even chunks of a sequence, dL/dS after it for the odd ones) and the chunk's
 * V' and dL/dV' (8 KiB each), 16 bytes per chunk of location records and 64 KiB per head of
 * partial sums; when the pass cuts its walks into pieces, also three fp32 states per (piece,
 * head, direction) (pieces of L chunks, L = max(8, ceil(4 H C / 768)) with C the chunk count
 * above; at most ceil(C / L) + N pieces per head, N the number of sequences).  Returns 0 for
 * invalid sizes.
 */
size_t kda_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens);

/*
 * kda_lin_fwd -- linear attention with a decay for each head, chunked form (prompts, training).
 * Per (sequence, head), with the state S [V][K] of kda_fwd's layout:
 *   S <- e^g S + v k^T,   out = scale * S q.
 *
 *   q, k      bf16 [B, T, Hk, 128], 16-byte aligned.  H must be a multiple of Hk: value head h
 *             reads q/k head h / (H / Hk).
 *   v         bf16 [B, T, H, 128], 16-byte aligned.
 *   decay     fp32 natural-log decays g <= 0: [H] (decay_per_token 0), or contiguous [B, T, H]
 *             (decay_per_token 1; the decay of a token acts on the state before its write).
 *             Used as min(max(g, -1000), 0); from -87.34 on the factor is 0 (below 2^-126, the smallest
 *             normal fp32 number), -inf makes the head forget.  A NaN makes the sequence's head NaN from there on.
 *   scale     finite output factor.
 *   out       bf16 [B, T, H, 128], contiguous, 16-byte aligned; every token of every sequence
 *             is written.  Must not overlap an input.
 *   initial_state, final_state and their dtypes, cu_seqlens, cu_seqlens_host, B, T, N, K, V, workspace
 *             (256-byte aligned, kda_lin_fwd_workspace_size bytes) and stream: as in kda_fwd,
 *             including the in-place state carry and the handling of an invalid cu_seqlens
 *             (kda_fwd_device_status reads the status word of this workspace too).
 *   strides_host  NULL (q, k, v contiguous), or host int64 [9]: batch, token and head strides of
 *             q, k, v in elements; the 128 channels of a head are contiguous.  Each a
 *             multiple of 8, the token stride 128 .. 2^24 (views of one fused projection; batch and
 *             head strides may be 0).
 * Products take 24 bits of every factor and sum in fp32, whatever the states' dtypes; out and bf16 final
 * states are rounded once.  out does not depend on whether final_state is asked for.  A value that
 * is not finite reaches its own sequence and head alone, from the first token of its chunk
 * of 64 tokens on (of the workgroup's run of tokens, see kda_lin_fwd_workspace_size), and lasts; a k or v that is not
 * finite may be forgotten where the decays behind it come to a factor below 2^-150.
 * Deterministic: fixed summation orders, no atomics.
 */
kda_status kda_lin_fwd(const void *q, const void *k, const void *v, const float *decay, int decay_per_token,
                       float scale, void *out, const void *initial_state, kda_state_dtype initial_state_dtype,
                       void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                       const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                       int64_t K, int64_t V, const int64_t *strides_host, void *workspace, size_t workspace_bytes,
                       void *stream);

/*
 * kda_lin_fwd_recurrent -- the same operator token by token in fp32, for the decode step (one token
 * per sequence, state in and out, often in place) and sequences of a few tokens.  Same
 * arguments and results (to rounding) as kda_lin_fwd.  The workspace may be NULL without
 * cu_seqlens; with it, 256 bytes hold the status word.
 */
kda_status kda_lin_fwd_recurrent(const void *q, const void *k, const void *v, const float *decay,
                                 int decay_per_token, float scale, void *out, const void *initial_state,
                                 kda_state_dtype initial_state_dtype, void *final_state,
                                 kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                                 const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t Hk, int64_t H,
                                 int64_t N, int64_t K, int64_t V, const int64_t *strides_host, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * kda_lin_fwd_workspace_size -- 256 bytes, plus one fp32 128 x 128 state and one float per head and
 * segment where the tokens of a batch row (all tokens with cu_seqlens) are cut into segments
 * that run in parallel: when batch rows x heads leave the chip empty.  A function of
 * (B, T, H, N, has_cu_seqlens) alone.  Returns 0 for invalid sizes, among them (KDA_ERR_SHAPE in the
 * calls) batch rows x segments x heads of 2^23 or more; token by token the limit is N x heads of 2^24.
 */
size_t kda_lin_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens);

/*
 * kda_lin_bwd -- gradients of kda_lin_fwd's out and final_state.  q, k, v, decay, scale, initial_state,
 * cu_seqlens, sizes, strides_host and stream as there.
 *   dout          bf16 [B, T, H, 128], contiguous, 16-byte aligned: dL/dout.
 *   dfinal_state  NULL (zero) or fp32 [N, H, 128, 128], 16-byte aligned: dL/dfinal_state.
 *   dq, dk        bf16 [B, T, Hk, 128], dv bf16 [B, T, H, 128], contiguous, 16-byte aligned, fully
 *                 written; heads that share a q/k head are summed in fp32 and rounded once.
 *   ddecay        NULL (not wanted) or fp32, of decay's shape; a per-head decay's is summed over
 *                 all tokens.  0 where decay lies outside (-1000, 0].  It is a sum of differences that hold the token's own
 *                 write, so its error is some 1e-7 of q.dq, whatever the decay: a percent of a token's ddecay at a decay
 *                 of -8, all of it from -14 on (kda_gdn_bwd's keeps its digits).  Products as in kda_lin_fwd.  Asking for
 *                 it changes the order of dq's and dk's fp32 sums, so single values may round differently.
 *   dinitial_state  NULL or fp32 [N, H, 128, 128], 16-byte aligned (also when initial_state is NULL).
 *   workspace     kda_lin_bwd_workspace_size(..., ddecay != NULL) bytes, 256-byte aligned.
 * Outputs must not overlap inputs or each other (KDA_ERR_ALIAS).  An invalid cu_seqlens found on
 * the device leaves dq, dk, dv and a per-token ddecay unwritten, a per-head ddecay 0 and
 * dinitial_state = dfinal_state (or 0).  Deterministic.
 */
kda_status kda_lin_bwd(const void *q, const void *k, const void *v, const float *decay, int decay_per_token,
                       float scale, const void *initial_state, kda_state_dtype initial_state_dtype, const void *dout,
                       const float *dfinal_state, void *dq, void *dk, void *dv, float *ddecay,
                       float *dinitial_state, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host, int64_t B,
                       int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t K, int64_t V,
                       const int64_t *strides_host, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_lin_bwd_workspace_size -- 256 bytes; per head and segment (see kda_lin_fwd_workspace_size; at
 * most 512 tokens long when need_ddecay) two fp32 states; with Hk < H two fp32 [B, T, H, 128];
 * with need_ddecay two fp32 [B, T, H] and small sums.  Returns 0 for invalid sizes.
 */
size_t kda_lin_bwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int has_cu_seqlens,
                                  int need_ddecay);

/*
 * kda_gdn_fwd -- the gated delta rule with a decay for each head, chunked form (prompts, training).  Per (sequence,
 * head), with the state S [V][K] of kda_fwd's layout:
 *   S~ = e^g S,   S <- S~ + beta (v - S~ k) k^T,   out = scale * S q.
 *
 *   q, k, v   bf16 [B, T, Hk, 128], [B, T, Hk, 128], [B, T, H, 128], strides_host: as in kda_lin_fwd (value head h reads
 *             q/k head h / (H / Hk)).  They are used as given: kda_qk_rope with KDA_NORM_L2 makes keys of norm 1, which
 *             keep the rule from growing for beta in [0, 2].
 *   decay     fp32 [B, T, H], contiguous: natural-log decay of each token, used as min(max(g, -1000), 0); it acts on
 *             the state before the token's write.  Below about -87 the factor is 0: the head forgets.
 *   beta      fp32 [B, T, H], contiguous: write strength, used as given (0 writes nothing).
 *   scale     finite output factor.
 *   out       bf16 [B, T, H, 128], contiguous, 16-byte aligned; every token of every sequence is written.  Must not
 *             overlap an input.
 *   initial_state, final_state and their dtypes, cu_seqlens, cu_seqlens_host, B, T, N, K, V, workspace
 *             (256-byte aligned, kda_gdn_fwd_workspace_size bytes) and stream: as in kda_fwd, including the
 *             in-place state carry and the handling of an invalid cu_seqlens (kda_fwd_device_status reads the
 *             status word of this workspace too).
 * Products take 24 bits of every factor and sum in fp32, whatever the states' dtypes; a product of two factors of more
 * than 8 bits leaves out 2^-25.7 of itself root mean square, 2^-22.4 at most, on no side.  out and bf16 final states are
 * rounded once.  Where a row is cut into segments (kda_gdn_fwd_workspace_size), a finite state that has passed
 * transitions of a norm below 2^-150 in all counts as 0.  A value that is not finite (or a NaN gate) reaches its own
 * sequence and head alone, from the first token of its chunk of 32 tokens on; in the state it lasts, in k or v it may be
 * forgotten behind such transitions.
 * Deterministic: fixed summation orders, no atomics.
 * Errors: KDA_ERR_NULL, _SHAPE (also sizes whose launch would hold 2^32 threads), _HEAD_DIM, _DTYPE, _SCALE, _ALIGN,
 * _WORKSPACE, _CU_SEQLENS, _HIP, _ALIAS, _HEADS, _STRIDE.
 */
kda_status kda_gdn_fwd(const void *q, const void *k, const void *v, const float *decay, const float *beta, float scale,
                       void *out, const void *initial_state, kda_state_dtype initial_state_dtype, void *final_state,
                       kda_state_dtype final_state_dtype, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host,
                       int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t K, int64_t V,
                       const int64_t *strides_host, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_gdn_fwd_recurrent -- the same operator token by token in fp32, for the decode step (one token per sequence,
 * state in and out, often in place) and sequences of a few tokens.  Same arguments and results (to rounding) as
 * kda_gdn_fwd.  The workspace may be NULL without cu_seqlens; with it, 256 bytes hold the status word.
 */
kda_status kda_gdn_fwd_recurrent(const void *q, const void *k, const void *v, const float *decay, const float *beta,
                                 float scale, void *out, const void *initial_state, kda_state_dtype initial_state_dtype,
                                 void *final_state, kda_state_dtype final_state_dtype, const int64_t *cu_seqlens,
                                 const int64_t *cu_seqlens_host, int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N,
                                 int64_t K, int64_t V, const int64_t *strides_host, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * kda_gdn_fwd_workspace_size -- 256 bytes; 13 KiB per chunk of 32 tokens and head (T / 32 chunks in all, and one for each sequence);
 * where rows are cut into segments that run in parallel, three fp32 128 x 128 states and a word per segment and head and a word
 * per chunk and head.  A function of (B, T, H, N, has_cu_seqlens) alone.  Returns 0 for invalid sizes.
 */
size_t kda_gdn_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N, int has_cu_seqlens);

/*
 * kda_gdn_bwd -- gradients of kda_gdn_fwd's out and final_state.  q, k, v, decay, beta, scale, initial_state,
 * cu_seqlens, sizes, strides_host and stream as there.
 *   dout          bf16 [B, T, H, 128], contiguous, 16-byte aligned: dL/dout.
 *   dfinal_state  NULL (zero) or fp32 [N, H, 128, 128], 16-byte aligned: dL/dfinal_state.
 *   dq, dk        bf16 [B, T, Hk, 128], dv bf16 [B, T, H, 128], contiguous, 16-byte aligned, fully
 *                 written; heads that share a q/k head are summed in fp32 and rounded once.
 *   ddecay, dbeta fp32 [B, T, H], fully written.  ddecay is 0 where decay lies outside (-1000, 0].  It is the sum of
 *                 what crosses its token, all of it scaled by e^decay, and so are its errors (some 1e-6 of the sizes of
 *                 the summands); 0 below about -87.
 *   dinitial_state  NULL or fp32 [N, H, 128, 128], 16-byte aligned (also when initial_state is NULL).
 *   workspace     kda_gdn_bwd_workspace_size(...) bytes, 256-byte aligned.
 * Products as in kda_gdn_fwd.  A value that is not finite reaches the gradients of its own sequence alone, one of v, dout, a
 * gate or a state there those of its value head (dq and dk are sums over the heads that share a q/k head): any of their
 * tokens up to the end of its block of 64, and behind it where kda_gdn_fwd passes it on; beyond transitions of a norm below
 * 2^-150 it may be forgotten.  Outputs must not overlap inputs or each other (KDA_ERR_ALIAS).  An invalid cu_seqlens
 * found on the device leaves dq, dk, dv, ddecay and dbeta unwritten and makes dinitial_state = dfinal_state (or 0).
 * Deterministic.
 */
kda_status kda_gdn_bwd(const void *q, const void *k, const void *v, const float *decay, const float *beta, float scale,
                       const void *initial_state, kda_state_dtype initial_state_dtype, const void *dout,
                       const float *dfinal_state, void *dq, void *dk, void *dv, float *ddecay, float *dbeta,
                       float *dinitial_state, const int64_t *cu_seqlens, const int64_t *cu_seqlens_host, int64_t B,
                       int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t K, int64_t V, const int64_t *strides_host,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_gdn_bwd_workspace_size -- 256 bytes; 51 KiB per chunk of 32 tokens and head (T / 32 chunks in all, and one for each sequence) and
 * 128 KiB per block of 64; where rows are cut, what kda_gdn_fwd_workspace_size says of that; with Hk < H two fp32 [B, T, H, 128].
 * Returns 0 for invalid sizes.
 */
size_t kda_gdn_bwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int has_cu_seqlens);

typedef enum kda_dtype {
    KDA_DTYPE_BF16 = 1,
    KDA_DTYPE_FP32 = 2,
    KDA_DTYPE_FP16 = 3
} kda_dtype;

typedef enum kda_norm {
    KDA_NORM_NONE = 0,
    KDA_NORM_RMS = 1, /* x / sqrt(mean(x^2) + eps) */
    KDA_NORM_L2 = 2   /* x / sqrt(sum(x^2) + eps), the normalisation kda_fwd applies to q and k */
} kda_norm;

/*
 * kda_qk_rope -- normalises each head of q and k and rotates pairs of its first rotary_dim channels by the
 * token's position, in one pass over both tensors; out rounded once.
 *   n = norm(x) * weight;   for pair i, t = position * inv_freq[i]:
 *   (a, b) -> attention_factor * (a cos t - b sin t, a sin t + b cos t);  other channels pass as n.
 *
 *   q, q_out      [B, T, Hq, D], k, k_out [B, T, Hk, D], all of `dtype`, 16-byte aligned.  D a multiple
 *                 of 16 up to 512.  An output may be its input (same pointer and strides);
 *                 otherwise outputs overlap nothing.
 *   q_weight, k_weight  NULL (1) or fp32 [D], 4-byte aligned, shared by the tensor's heads.
 *   inv_freq      fp32 [rotary_dim / 2] angular frequencies (radians per position), any scaling
 *                 for long contexts already applied; NULL when rotary_dim is 0.
 *   positions     int64 [B, T], contiguous, or NULL: the token's index in its row.  Angles are formed in
 *                 fp64: exact to fp32 rounding for |position * inv_freq| below 2^27.
 *   rotary_dim    0 .. D, a multiple of 16.  interleaved: pairs (2i, 2i + 1) when 1, else
 *                 (i, i + rotary_dim / 2).
 *   norm, eps     eps finite and >= 0 (not used by KDA_NORM_NONE).
 *   strides_host  NULL (contiguous) or host int64 [12]: batch, token, head strides in elements of
 *                 q, k, q_out, k_out, each a multiple of 16 bytes.
 * Errors: KDA_ERR_NULL, _SHAPE, _ROTARY, _DTYPE, _FLAGS (norm, interleaved), _SCALE (eps, factor), _STRIDE,
 * _ALIGN, _ALIAS, _HIP.  T = 0 does nothing.
 */
kda_status kda_qk_rope(const void *q, const void *k, void *q_out, void *k_out, const float *q_weight,
                       const float *k_weight, const float *inv_freq, const int64_t *positions, int64_t B, int64_t T,
                       int64_t Hq, int64_t Hk, int64_t D, int64_t rotary_dim, kda_dtype dtype, kda_norm norm,
                       float eps, int interleaved, float attention_factor, const int64_t *strides_host,
                       void *stream);

/*
 * kda_qk_rope_bwd -- gradients of kda_qk_rope: dq, dk from dq_out, dk_out and the forward pass's inputs, and
 * (NULL = not wanted) dq_weight, dk_weight, fp32 [D], summed over tokens and heads in a
 * fixed order.  strides_host: int64 [18], q, k, dq_out, dk_out, dq, dk.  dq may be q or dq_out,
 * dk k or dk_out (same pointer and strides).  The workspace (kda_qk_rope_bwd_workspace_size
 * bytes, 256-byte aligned) is used, and may be NULL otherwise, when a weight gradient is wanted.
 */
kda_status kda_qk_rope_bwd(const void *q, const void *k, const void *dq_out, const void *dk_out, void *dq, void *dk,
                           const float *q_weight, const float *k_weight, float *dq_weight, float *dk_weight,
                           const float *inv_freq, const int64_t *positions, int64_t B, int64_t T, int64_t Hq,
                           int64_t Hk, int64_t D, int64_t rotary_dim, kda_dtype dtype, kda_norm norm, float eps,
                           int interleaved, float attention_factor, const int64_t *strides_host, void *workspace,
                           size_t workspace_bytes, void *stream);

/* Bytes of partial weight sums: 4 D for each of 1024 workgroups.  Returns 0 for invalid sizes. */
size_t kda_qk_rope_bwd_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D);

typedef enum kda_gate {
    KDA_GATE_SIGMOID = 0,
    KDA_GATE_SILU = 1 /* z * sigmoid(z) */
} kda_gate;

/*
 * kda_gated_norm -- the norm behind a mixer with its gate: out = x / sqrt(mean(x^2) + eps) * weight * act(gate), per token
 * and head, in fp32, rounded once.
 *   x, gate       [B, T, H, D] of `dtype`, 16-byte aligned.  D a multiple of 8 up to 512.
 *   weight        NULL (1) or fp32 [D], shared by the heads.
 *   out           [B, T, H, D], contiguous, 16-byte aligned.  May be x or gate where that is contiguous; else it overlaps
 *                 no input.
 *   activation    act: KDA_GATE_SIGMOID or KDA_GATE_SILU.   eps: finite and >= 0.
 *   strides_host  NULL (contiguous) or host int64 [6]: batch, token, head strides of x and gate in elements, each a
 *                 multiple of 16 bytes.
 * Errors: KDA_ERR_NULL, _SHAPE (also 2^31 rows or more), _HEAD_DIM (D), _DTYPE, _FLAGS (activation), _SCALE (eps), _STRIDE,
 * _ALIGN, _ALIAS, _HIP.  T = 0 does nothing.
 */
kda_status kda_gated_norm(const void *x, const void *gate, const float *weight, void *out, int64_t B, int64_t T, int64_t H,
                          int64_t D, kda_dtype dtype, kda_gate activation, float eps, const int64_t *strides_host,
                          void *stream);

/*
 * kda_gated_norm_bwd -- gradients of kda_gated_norm from its inputs and dout [B, T, H, D], contiguous: dx, dgate, contiguous,
 * and dweight (NULL = not wanted), fp32 [D], summed over tokens and heads in a fixed order.  The workspace
 * (kda_gated_norm_bwd_workspace_size bytes, 256-byte aligned) is used, and may be NULL otherwise, when dweight is wanted.
 * Outputs overlap nothing.
 */
kda_status kda_gated_norm_bwd(const void *x, const void *gate, const float *weight, const void *dout, void *dx, void *dgate,
                              float *dweight, int64_t B, int64_t T, int64_t H, int64_t D, kda_dtype dtype,
                              kda_gate activation, float eps, const int64_t *strides_host, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Bytes of partial weight sums: 4 D for each of up to 1024 workgroups.  Returns 0 for invalid sizes. */
size_t kda_gated_norm_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t D, kda_dtype dtype);

/*
 * kda_residual_norm -- from one block to the next: an optional norm of the block's output, its scale per channel, the
 * residual's sum and the norm before the next block, per token, in fp32:
 *   h = x, or x / sqrt(mean(x^2) + eps) * post_weight (post_norm KDA_NORM_RMS);   y = residual + scale * h;
 *   residual_out = y, rounded to its type;   out = y / sqrt(mean(y^2) + eps) * weight, from the sum before it is rounded.
 *   x, out        [B, T, D] of `dtype`; residual, residual_out [B, T, D] of `residual_dtype`: dtype or fp32.  All 16-byte
 *                 aligned; out and residual_out contiguous.  out may be x and residual_out may be residual where that is contiguous;
 *                 otherwise outputs overlap nothing.  D a multiple of 8 up to 8192.
 *   weight, scale, post_weight  NULL (1) or fp32 [D]; post_weight only with KDA_NORM_RMS.
 *   strides_host  NULL (contiguous) or host int64 [4]: batch and token strides of x and residual in elements, each a
 *                 multiple of 16 bytes.
 * Errors as in kda_gated_norm (_FLAGS: post_norm).
 */
kda_status kda_residual_norm(const void *x, const void *residual, const float *weight, const float *scale,
                             const float *post_weight, void *out, void *residual_out, int64_t B, int64_t T, int64_t D,
                             kda_dtype dtype, kda_dtype residual_dtype, kda_norm post_norm, float eps,
                             const int64_t *strides_host, void *stream);

/*
 * kda_residual_norm_bwd -- gradients of kda_residual_norm: dx (of dtype) and dresidual (of residual_dtype), contiguous, from
 * x, residual_out as the forward pass stored it (the gradients are those at the stored values), dout and
 * dresidual_out (NULL = zero), both contiguous; and (NULL = not wanted) dweight, dscale, dpost_weight, fp32 [D], summed over
 * tokens in a fixed order.  strides_host: int64 [4], of x and residual_out.  The workspace
 * (kda_residual_norm_bwd_workspace_size bytes, 256-byte aligned) is used, and may be NULL otherwise, when one of the
 * three is wanted.  Outputs overlap nothing.
 */
kda_status kda_residual_norm_bwd(const void *x, const void *residual_out, const void *dout, const void *dresidual_out,
                                 const float *weight, const float *scale, const float *post_weight, void *dx,
                                 void *dresidual, float *dweight, float *dscale, float *dpost_weight, int64_t B, int64_t T,
                                 int64_t D, kda_dtype dtype, kda_dtype residual_dtype, kda_norm post_norm, float eps,
                                 const int64_t *strides_host, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of partial weight sums: 12 D for each of up to 1024 workgroups.  Returns 0 for invalid sizes. */
size_t kda_residual_norm_bwd_workspace_size(int64_t B, int64_t T, int64_t D);

/* Human-readable name of a kda_status value (static string; never NULL). */
const char *kda_status_string(int status);

/*
 * kda_fwd_device_status -- after kda_fwd on `stream`, wait for the stream and read the
 * device status word from the workspace: 0 = inputs valid and the forward pass ran to
 * completion; otherwise a bit mask (1: cu[0] != 0, 2: cu decreasing somewhere,
 * 4: cu[N] != T, 0x100: a wavefront of the forward kernel gave up waiting for another
 * one -- results invalid; not expected to happen).  Synchronises the stream.
 */
kda_status kda_fwd_device_status(const void *workspace, int32_t *status_out, void *stream);

/*
 * kda_chunk_table -- run only the first stage of kda_fwd: the integer chunk table built
 * from cu_seqlens (or from B and T).  Writes into the workspace and, when the host
 * pointers are non-NULL, copies back (synchronising the stream):
 *   seq_off_host  int64 [N+1]  exclusive prefix sum of ceil(L_i / 16)
 *   n_total_host  int64        total number of chunks
 *   status_host   int32        device status word (as kda_fwd_device_status)
 * Used to check the integer indexing bit for bit.
 */
kda_status kda_chunk_table(const int64_t *cu_seqlens, int64_t B, int64_t T, int64_t H, int64_t N,
                           void *workspace, size_t workspace_bytes, int64_t *seq_off_host,
                           int64_t *n_total_host, int32_t *status_host, void *stream);

/* Library version, major * 10000 + minor * 100 + patch. */
int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
