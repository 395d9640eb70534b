/*
 * gdp.h -- C ABI of the MI355X (gfx950) chunked Gated DeltaProduct prefill library.
 *
 * The operation (FlashInfer docs, "flashinfer.gdp_prefill.chunk_gated_delta_product",
 * the recurrence display): for every sequence and every state head, per real
 * token t the K x V state S is first scaled by alpha_t = exp(g_log_t); then for
 * j = 0..n-1 on sub-token row r = t*n + j
 *     v_new_r = beta_r * (v_r - S^T k_r),   S += k_r v_new_r^T;
 * and after the last update o_t = scale * S^T q_t.  n = 1 is the gated delta rule.
 * The argument list follows the Megatron Core API docs, core.ssm.ops.gdp.chunk,
 * chunk_gated_delta_product_varlen (parameter list and the graph-capture note
 * after it), with outputs, workspace and stream appended.
 *
 * Conventions shared by every entry point
 *   - Every data pointer is DEVICE memory owned by the caller.  The library
 *     never allocates, frees or synchronises, never reads device memory on
 *     the host, and launches only on the stream it is given (a hipStream_t
 *     passed as void*; NULL is the default stream).  A call is therefore
 *     capturable into a HIP graph.
 *   - Return value: GDP_OK (0) or a negative gdp_status.  No exception ever
 *     crosses the ABI.  On failure gdp_last_error() returns a message (per
 *     calling thread).  Errors are detected from shapes, dtypes, strides and
 *     pointer ranges only; the contents of cu_seqlens, state_indices and
 *     caller-built descriptors are not checked (that would need a device to
 *     host read).  The kernels clamp what they index with them: sequence
 *     bounds to [0, T], cache slots outside [0, S) and chunk-state rows past
 *     the buffer are skipped, so bad contents give wrong numbers, never an
 *     out-of-bounds access.
 *   - Chunk size is fixed at 64 (Megatron Core page, the two-chunkings
 *     paragraph and the chunk_states description).
 */
#ifndef GDP_H
#define GDP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of gdp_tensor. */
enum gdp_dtype { GDP_F32 = 0, GDP_BF16 = 1, GDP_I32 = 2, GDP_I64 = 3, GDP_F16 = 4 };

/* Return codes. */
enum gdp_status {
  GDP_OK = 0,
  GDP_EINVAL = -1,       /* bad shape, dtype, stride, n < 1, Hv % Hqk != 0, missing argument */
  GDP_EUNSUPPORTED = -2, /* valid request this build does not serve (head dims, dtype mix) */
  GDP_EALIAS = -3,       /* an output overlaps an input or another output */
  GDP_EWORKSPACE = -4,   /* workspace missing or smaller than gdp_workspace_bytes() */
  GDP_EHIP = -5          /* a HIP launch failed; message from hipGetErrorString */
};

/* A strided view of device memory.  data == NULL means "absent" (None).
 * shape/stride hold ndim valid entries; strides are in ELEMENTS.  The
 * innermost dimension must be contiguous (stride 1, or a size of 1). */
typedef struct gdp_tensor {
  void *data;
  int32_t dtype;
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} gdp_tensor;

/* Chunk descriptors of the two chunkings (Megatron Core page: chunk_indices,
 * chunk_indices_dp, chunk_offsets).  Sequence i of length L_i has
 * ceil(L_i/64) token chunks and ceil(n*L_i/64) expanded chunks.
 *   chunk_indices    [nt_cap, 2]   int32 rows (i, c), sequence-major, c ascending,
 *                                  rows past the real count hold (-1, -1)
 *   chunk_indices_dp [ntdp_cap, 2] the same for the expanded stream
 *   chunk_offsets    [N+1]         int32 exclusive prefix sums of token-chunk counts
 *   chunk_offsets_dp [N+1]         the same for expanded-chunk counts
 * All four arrays are device memory owned by the caller. */
typedef struct gdp_descriptors {
  int32_t *chunk_indices;
  int32_t *chunk_indices_dp;
  int32_t *chunk_offsets;
  int32_t *chunk_offsets_dp;
  int64_t nt_cap;
  int64_t ntdp_cap;
} gdp_descriptors;

/* Host-only.  Capacities that bound the descriptor row counts for any
 * cu_seqlens with N sequences and T real tokens:
 *   nt_cap = floor((T + 63 N) / 64),  ntdp_cap = floor((n T + 63 N) / 64).
 * Padding to these makes every grid depend on (T, N, n) only (Megatron Core
 * page, the graph-capture note).  Returns GDP_EINVAL for negative sizes or n < 1. */
int gdp_descriptor_capacity(int64_t T, int64_t N, int32_t num_householder,
                            int64_t *nt_cap, int64_t *ntdp_cap);

/* Device.  Builds the descriptors of cu_seqlens ([N+1], int32 or int64,
 * device, contiguous) into out->*, padded to out->nt_cap / out->ntdp_cap, with
 * one kernel launch on `stream`.  T is the caller's real-token count; the
 * capacities must be at least gdp_descriptor_capacity(T, N, n) (GDP_EINVAL
 * otherwise).  Capturable; "built once per step" in the Megatron Core
 * page's words. */
int gdp_build_descriptors(const gdp_tensor *cu_seqlens, int32_t num_householder, int64_t T,
                          const gdp_descriptors *out, void *stream);

/* Host-only.  Workspace bytes gdp_chunk_prefill needs for T real tokens, N
 * sequences, n Householder rows per token, Hv state heads and input dtype
 * (GDP_BF16 or GDP_F32): the per-chunk WY matrices (64 x 64 per expanded
 * chunk and state head, at the input precision) or the buffers of the
 * segmented (chunk-parallel) path for few long sequences (bf16, K == V: per
 * segment of at least 256 tokens an f32 K x K map and two K x V states per
 * head), whichever is larger; plus room for the descriptors when the caller
 * passes none; plus an int32 work order of N x Hv entries when N x Hv > 256 and
 * N <= 4096; plus an int32 chunk counter per (sequence, state head) when
 * Hv > Hqk (the fused kernel paces the state heads that share a q/k head).
 * The size depends on host-known shapes only, so one allocation serves every
 * call of a captured batch shape, as the fixed-length descriptors do (Megatron
 * Core page, core.ssm.ops.gdp.chunk, the note on the descriptor arguments and
 * graph capture).  Returns 0 for invalid sizes or dtypes. */
size_t gdp_workspace_bytes(int64_t T, int64_t N, int32_t num_householder, int32_t Hqk,
                           int32_t Hv, int32_t K, int32_t V, int32_t dtype);

/* Device.  The chunked GDP prefill forward pass.
 *
 * Inputs (T real tokens, N sequences, n = num_householder, Hqk q/k heads,
 * Hv state heads = v/g/beta/output heads, head dims K and V):
 *   q            [T, Hqk, K]      bf16 or f32; rows may be strided
 *   k            [T*n, Hk, K]     same dtype as q; rows t*n..t*n+n-1 belong to token t;
 *                                 Hk = Hqk, or Hk = Hv (one k head per state head;
 *                                 FlashInfer page, k: num_k_heads equals the q or the
 *                                 v head count).  State head h reads q head
 *                                 h / (Hv / Hqk) and k head h / (Hv / Hk)
 *   v            [T*n, Hv, V]     same dtype as q
 *   g_log        [T, Hv]          f32 log decays (alpha_t = exp(g_log_t))
 *   beta         [T*n, Hv]        f32
 *   cu_seqlens   [N+1]            int32 or int64, contiguous, required
 *   scale        readout scale; 0 means K^-1/2 (FlashInfer page, scale)
 *   initial_state [N, Hv, K, V]   f32 contiguous, or data == NULL for zeros
 *   output_final_state            write final_state when nonzero
 *   use_qk_l2norm                 divide every q row and k sub-token row by
 *                                 sqrt(sum x^2 + 1e-6) inside the kernel
 *   state_cache  [S, Hv, K, V]    f32 contiguous, or NULL; when given, the final
 *                                 state of sequence i is written in place at
 *                                 slot state_indices[i]; -1 writes nothing
 *   state_indices [N]             int32 or int64; required with state_cache
 *   return_chunk_states           write chunk_states when nonzero
 * Outputs (caller-allocated device memory):
 *   o            [T, Hv, V]       same dtype as q; rows may be strided
 *   final_state  [N, Hv, K, V]    f32 contiguous; required iff output_final_state
 *   chunk_states [R, Hv, K, V]    f32 contiguous, R >= gdp_descriptor_capacity's
 *                                 nt_cap; row chunk_offsets[i] + c is the state of
 *                                 sequence i entering its token chunk c, i.e. after
 *                                 its first 64*c tokens (Megatron Core page,
 *                                 return_chunk_states).  Rows past the real count
 *                                 are left untouched.
 *   desc         caller-built descriptors (gdp_build_descriptors) or NULL; when
 *                NULL they are built into the workspace on `stream`.  Their
 *                capacities must be at least gdp_descriptor_capacity(T, N, n)
 *                (GDP_EINVAL otherwise: descriptors built for a smaller T or a
 *                different n would leave chunks out of the grids)
 *   workspace    device scratch, 256-byte aligned, of workspace_bytes >=
 *                gdp_workspace_bytes(...) (required: it holds the per-chunk WY
 *                matrices between the two kernels of the call)
 * Ownership/aliasing: no output may overlap an input or another output; in
 * particular final_state must not alias initial_state, because one sequence's
 * state is split over several workgroups (FlashInfer page, output_state).
 * Supported today: K, V in {64, 128}; f32 inputs need K = 64 (GDP_EUNSUPPORTED
 * otherwise).  Calls that overlap on one stream are ordered; calls on
 * different streams sharing an output race. */
int gdp_chunk_prefill(const gdp_tensor *q, const gdp_tensor *k, const gdp_tensor *v,
                      const gdp_tensor *g_log, const gdp_tensor *beta,
                      int32_t num_householder, const gdp_tensor *cu_seqlens, float scale,
                      const gdp_tensor *initial_state, int32_t output_final_state,
                      int32_t use_qk_l2norm, const gdp_tensor *state_cache,
                      const gdp_tensor *state_indices, int32_t return_chunk_states,
                      const gdp_tensor *o, const gdp_tensor *final_state,
                      const gdp_tensor *chunk_states, const gdp_descriptors *desc,
                      void *workspace, size_t workspace_bytes, void *stream);

/* Size of the static scratch array of gdp_chunk_prefill_noalloc, per GPU. */
#define GDP_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* Device.  gdp_chunk_prefill without a workspace argument, for callers that
 * cannot allocate device memory: code under graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  Arguments, results and errors are
 * those of gdp_chunk_prefill; the workspace is a file-scope device array of
 * GDP_NOALLOC_SCRATCH_BYTES (64 MiB) that every GPU the library runs on holds
 * until the process ends.  The call allocates nothing.  A call whose workspace
 * need exceeds the array returns GDP_EWORKSPACE with the size it needs.  The
 * fused path needs only the descriptors (when desc is NULL), the work order and
 * the pacing counters: 16 bytes per chunk row plus 8 per (sequence, state
 * head), under 1 MiB up to tens of millions of tokens; the split path's WY
 * matrices take 8 KiB (bf16) or 16 KiB (f32) per expanded chunk and state head,
 * and the segmented path 12 K V bytes per segment and state head.  All calls on one GPU share its array:
 * calls that overlap on one GPU (for instance on two streams) race; calls on
 * one stream are ordered.  No call depends on what an earlier one left in the
 * array. */
int gdp_chunk_prefill_noalloc(const gdp_tensor *q, const gdp_tensor *k, const gdp_tensor *v,
                              const gdp_tensor *g_log, const gdp_tensor *beta, int32_t num_householder,
                              const gdp_tensor *cu_seqlens, float scale, const gdp_tensor *initial_state,
                              int32_t output_final_state, int32_t use_qk_l2norm,
                              const gdp_tensor *state_cache, const gdp_tensor *state_indices,
                              int32_t return_chunk_states, const gdp_tensor *o,
                              const gdp_tensor *final_state, const gdp_tensor *chunk_states,
                              const gdp_descriptors *desc, void *stream);

/* Device.  The single-token recurrent decode step on the state cache, in place.
 *
 * The decode step of the blog page "Attention Cache and Sequence Parallelism"
 * (section "GDN: fixed state instead of a per-token cache": Sbar = lambda S,
 * vhat = Sbar^T k, e = beta (v - vhat), S = Sbar + k e^T, r = q^T S), with the
 * n Householder rows per token of the FlashInfer recurrence display and the
 * slot convention of the Megatron Core page (state / state_indices).  For
 * every entry i and state head h with slot = state_indices[i] in [0, S):
 *     S = state_cache[slot, h];  S *= exp(g_log[i, h]);
 *     for j = 0..n-1, r = i*n + j:  e = beta[r,h] (v[r,h] - S^T k[r]);  S += k[r] e^T;
 *     o[i, h] = scale * S^T q[i];  state_cache[slot, h] = S.
 * Entries whose index is negative (padding, -1) or past the cache get a zero
 * output row and leave the cache untouched.
 *   q [N, Hqk, K], k [N*n, Hk, K], v [N*n, Hv, V]    bf16 or f32 (one dtype); rows may be strided;
 *                                                    Hk = Hqk or Hv, as for gdp_chunk_prefill
 *   g_log [N, Hv], beta [N*n, Hv]                    f32 (log decays; alpha = exp(g_log))
 *   scale                                            0 means K^-1/2
 *   use_qk_l2norm                                    as for gdp_chunk_prefill
 *   state_cache [S, Hv, K, V]                        f32 contiguous, K-major states, read and written
 *   state_indices [N]                                int32 or int64
 *   o [N, Hv, V]                                     q's dtype, written
 * Two entries naming the same slot race (caller error; not checked: that needs
 * a device read).  o and the cache may not overlap the inputs or each other
 * (GDP_EALIAS).  K, V in {64, 128}.  One kernel launch on `stream`; nothing is
 * allocated, so the call is capturable. */
int gdp_recurrent_decode(const gdp_tensor *q, const gdp_tensor *k, const gdp_tensor *v,
                         const gdp_tensor *g_log, const gdp_tensor *beta, int32_t num_householder,
                         float scale, int32_t use_qk_l2norm, const gdp_tensor *state_cache,
                         const gdp_tensor *state_indices, const gdp_tensor *o, void *stream);

/* Host-only.  Workspace bytes gdp_chunk_prefill_backward needs, the larger of
 * its two paths' needs.  The chunked path: the descriptors, then per expanded
 * 64-row chunk and state head the float32 entering state and end-of-chunk state
 * gradient (2 x ntdp_cap x Hv x K x V floats) and a prep bundle (T^T and the
 * decayed scores in bfloat16, per-row factors).  The recurrent path: the
 * descriptors, the float32 state entering every token chunk (nt_cap x Hv x K x V),
 * an output buffer of the forward pass it reruns, the float32 L2-norm factors of
 * the q and k rows (T x Hqk and T*n x Hv at most), and that pass's workspace
 * (gdp_workspace_bytes).  Returns 0 for invalid sizes or dtypes. */
size_t gdp_backward_workspace_bytes(int64_t T, int64_t N, int32_t num_householder, int32_t Hqk, int32_t Hv,
                                    int32_t K, int32_t V, int32_t dtype);

/* Device.  Gradients of the prefill: with L = <o, d_o> + <final_state,
 * d_final_state>, writes dL/dq, dL/dk, dL/dv, dL/dg_log, dL/dbeta and (when
 * d_initial_state is given) dL/dinitial_state, for the same inputs and
 * conventions as gdp_chunk_prefill (no state cache, no chunk states).
 *
 * The pages give no backward formulas (the blog page "Attention Cache and
 * Sequence Parallelism", section "GDN: pass the state, not the KV", notes only
 * that the dependencies run in reverse); these are the gradients of the
 * recurrence itself, by reverse-mode differentiation.  Two paths give them:
 *   chunked (bfloat16 inputs, q/k/v/d_o 16-byte aligned with row and head
 *   strides multiples of 8): per
 *   64-row expanded chunk, a prep kernel forms the chunk's WY inverse and decayed
 *   scores, a forward walk stores each chunk's entering state and a reverse walk
 *   each chunk's end-of-chunk state gradient (both float32), and a gradient
 *   kernel forms every gradient of a chunk with matrix-core products;
 *   recurrent (everything else, or GDP_BACKWARD_PATH=recurrent in the
 *   environment): reruns the forward pass to obtain the state entering every
 *   64-token chunk, then walks each chain backwards token by token, recomputing
 *   the states in between.
 *   d_o            [T, Hv, V]      q's dtype, rows may be strided
 *   d_final_state  [N, Hv, K, V]   float32 contiguous, or data == NULL (zero)
 *   dq [T, Hqk, K], dk [T*n, Hk, K], dg_log [T, Hv], dbeta [T*n, Hv]
 *                                  float32, contiguous: the recurrent path
 *                                  accumulates them with float atomics over state
 *                                  heads and V tiles, so their last bits depend on
 *                                  the order of the adds; the chunked path stores
 *                                  each entry once
 *   dv [T*n, Hv, V]                float32, rows may be strided; the sub-rows no
 *                                  sequence covers (before cu_seqlens[0]*n or from
 *                                  cu_seqlens[N]*n on) are written as zeros, like
 *                                  the other gradients' rows there
 *   d_initial_state [N, Hv, K, V]  float32 contiguous, or data == NULL
 *   workspace      at least gdp_backward_workspace_bytes(...), 256-byte aligned
 * No gradient may overlap an input or another gradient (GDP_EALIAS).  K, V in
 * {64, 128}, num_householder <= 5 (GDP_EUNSUPPORTED otherwise).  Everything
 * runs on `stream` with no allocation and no host read of device memory. */
int gdp_chunk_prefill_backward(const gdp_tensor *q, const gdp_tensor *k, const gdp_tensor *v,
                               const gdp_tensor *g_log, const gdp_tensor *beta, int32_t num_householder,
                               const gdp_tensor *cu_seqlens, float scale, const gdp_tensor *initial_state,
                               int32_t use_qk_l2norm, const gdp_tensor *d_o, const gdp_tensor *d_final_state,
                               const gdp_tensor *dq, const gdp_tensor *dk, const gdp_tensor *dv,
                               const gdp_tensor *dg_log, const gdp_tensor *dbeta,
                               const gdp_tensor *d_initial_state, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Host-only.  Workspace bytes gdp_chunk_gated_delta_product needs: the gates
 * restated as float32 log decays and betas (4 (1 + n) T Hv bytes; the betas are
 * used only when they are not float32 already), a float32
 * K-major copy of each state it converts (4 N Hv d^2 bytes each, when an
 * initial state is given and when the final state is requested), and the
 * workspace of the prefill it runs (gdp_workspace_bytes); with float16 inputs
 * also bfloat16 copies of q, k, v and the output.  dtype is q's (GDP_BF16 or
 * GDP_F16).  Returns 0 for invalid sizes or dtypes. */
size_t gdp_fi_workspace_bytes(int64_t T, int64_t N, int32_t num_householder, int32_t Hq, int32_t Hv,
                              int32_t head_size, int32_t dtype, int32_t with_initial_state,
                              int32_t output_final_state);

/* Device.  The chunked GDP prefill in the FlashInfer convention (FlashInfer docs,
 * "flashinfer.gdp_prefill.chunk_gated_delta_product": its recurrence display and
 * parameter list, in the same order, with workspace and stream appended).
 * It computes what gdp_chunk_prefill computes; only the operands are stated
 * differently:
 *   q  [T, Hq, d], k [T*n, Hk, d] (Hk = Hq or Hv), v [T*n, Hv, d]   bfloat16 or
 *                  float16, rows may be strided; Hv a multiple of Hq (more q than v
 *                  heads is GDP_EUNSUPPORTED), d in {64, 128}.  float16 inputs
 *                  are copied to bfloat16 operands in the workspace (row and head
 *                  strides must be multiples of 8) and the output, formed in
 *                  bfloat16, is converted to float16
 *   g    [T, Hv]   the decay alpha itself (in (0, 1]), float32, bfloat16 or float16,
 *                  or data == NULL for no decay (alpha = 1)
 *   beta [T*n, Hv] float32 (read in place, strides honoured) or q's dtype, or
 *                  data == NULL for all ones
 *   scale          0 means d^-1/2
 *   initial_state  [N, Hv, d, d] V-major (entry [v][k]), float32 or bfloat16,
 *                  contiguous, or data == NULL for zero states
 *   output_final_state  write output_state when nonzero
 *   cu_seqlens     [N+1] int32 or int64, required
 *   use_qk_l2norm_in_kernel   as gdp_chunk_prefill's use_qk_l2norm
 *   output         [T, Hv, d] q's dtype, written
 *   output_state   [N, Hv, d, d] V-major, float32 or bfloat16, contiguous; required
 *                  iff output_final_state; it may not overlap initial_state or any
 *                  input (GDP_EALIAS; FlashInfer page, output_state)
 *   workspace      device scratch of at least gdp_fi_workspace_bytes(...), 256-byte
 *                  aligned
 * Everything runs on `stream` (conversion kernels, then the prefill), with no
 * host read of device memory and no allocation, so the call is capturable. */
int gdp_chunk_gated_delta_product(const gdp_tensor *q, const gdp_tensor *k, const gdp_tensor *v,
                                  const gdp_tensor *g, const gdp_tensor *beta, int32_t num_householder,
                                  float scale, const gdp_tensor *initial_state, int32_t output_final_state,
                                  const gdp_tensor *cu_seqlens, int32_t use_qk_l2norm_in_kernel,
                                  const gdp_tensor *output, const gdp_tensor *output_state, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Layers around the matrix-state recurrence: a per-channel (vector-state) gated
 * linear recurrence, and the group norm that follows either recurrence's
 * outputs.  The conventions above hold here too.
 * ------------------------------------------------------------------------ */

/* Rows of the token stream per recurrence checkpoint. */
#define GDP_SCAN_CHECKPOINT_ROWS 64

/* Host-only.  Workspace bytes gdp_gated_scan needs for T rows, N sequences and D
 * channels: a ticket counter and, per 128 rows and channel (and per 2048), one 8-byte
 * word through which the workgroups of a long sequence hand their states on.  The call writes
 * it before use and leaves nothing in it that a later call reads.  Returns 0 for
 * invalid sizes and where none is needed (up to 128 rows). */
size_t gdp_gated_scan_workspace_bytes(int64_t T, int64_t N, int64_t D);

/* Device.  The gated linear recurrence over packed sequences.  For every sequence
 * and channel d, from h = initial_state (or 0), per token t:
 *     h_t = a_t h_{t-1} + u_t,   a_t = exp(g_log[t, d]),   o[t, d] = h_t,
 *     u_t = x[t, d], or (1 - a_t) x[t, d] with complement_input.
 *   x            [T, D]    f32, bf16 or f16; rows may be strided
 *   g_log        [T, D]    f32 or x's dtype; log decays, g_log <= 0 (a positive
 *                          entry is served while the products of decays over 128
 *                          rows and fewer stay finite in float32, for any number of
 *                          channels); what such a product below 2^-126 leaves of a
 *                          state may be taken for 0; -inf drops the state before
 *                          (a state which is not finite may end at a -inf, or where
 *                          the product of its decays falls below 2^-126, or go on)
 *   cu_seqlens   [N+1]     int32 or int64, contiguous
 *   initial_state [N, D]   f32 contiguous, or data == NULL for zeros
 *   output_final_state     write final_state when nonzero
 *   state_cache  [S, D]    f32 contiguous, or NULL; when given, the final state of
 *                          sequence i is written at slot state_indices[i]; an index
 *                          outside [0, S) writes nothing, two sequences naming one slot
 *                          race (caller error)
 *   state_indices [N]      int32 or int64; required with state_cache
 *   return_checkpoints     write checkpoints when nonzero
 *   o            [T, D]    x's dtype, rows may be strided; the rows no sequence
 *                          covers are left as they are
 *   final_state  [N, D]    f32 contiguous; required iff output_final_state; of an
 *                          empty sequence its initial state
 *   checkpoints  [ceil(T / 64), D]  f32 contiguous: row c is the state entering
 *                          token row 64 c where that row continues a sequence, and
 *                          unspecified elsewhere; what gdp_gated_scan_backward reads
 *   workspace    at least gdp_gated_scan_workspace_bytes(...), 256-byte aligned
 * States are held in float32.  A non-finite x or g_log stays within its sequence
 * and channel.  No output may overlap an input or another output (GDP_EALIAS).
 * Calls that share a workspace must be ordered.  Two runs on the same inputs give
 * the same bits.  One or two launches on `stream`, no allocation: capturable. */
int gdp_gated_scan(const gdp_tensor *x, const gdp_tensor *g_log, const gdp_tensor *cu_seqlens,
                   int32_t complement_input, const gdp_tensor *initial_state, int32_t output_final_state,
                   const gdp_tensor *state_cache, const gdp_tensor *state_indices, int32_t return_checkpoints,
                   const gdp_tensor *o, const gdp_tensor *final_state, const gdp_tensor *checkpoints,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Device.  One token of the recurrence per entry, on the state cache in place:
 * for slot = state_indices[i] in [0, S),
 *     state_cache[slot] = a_i state_cache[slot] + u_i,   o[i] = state_cache[slot];
 * the other entries (padding, -1) get a zero output row and touch no state.
 *   x, g_log, o [N, D] as for gdp_gated_scan, state_cache [S, D] f32 contiguous,
 *   state_indices [N] int32 or int64.  Two entries naming one slot race (caller
 *   error).  One launch on `stream`; capturable. */
int gdp_gated_scan_decode(const gdp_tensor *x, const gdp_tensor *g_log, int32_t complement_input,
                          const gdp_tensor *state_cache, const gdp_tensor *state_indices, const gdp_tensor *o,
                          void *stream);

/* Host-only.  Workspace bytes gdp_gated_scan_backward needs (the forward scan's
 * words and, for calls without checkpoints, room for them).  0 for invalid sizes. */
size_t gdp_gated_scan_backward_workspace_bytes(int64_t T, int64_t N, int64_t D);

/* Device.  Gradients of gdp_gated_scan.  With L = <o, d_o> + <final_state,
 * d_final_state> and e_t the gradient of the state after token t (walking back from
 * d_final_state, or 0):
 *     e_t = d_o_t + a_{t+1} e_{t+1},   dx_t = e_t  or  (1 - a_t) e_t,
 *     dg_log_t = e_t a_t (h_{t-1}  or  h_{t-1} - x_t),   d_initial_state = a_0 e_0.
 *   x, g_log, cu_seqlens, complement_input, initial_state  the forward call's
 *   checkpoints  those of the forward call, or data == NULL: the states are then
 *                formed again first (x and g_log are read a second time)
 *   d_o          [T, D]  x's dtype, rows may be strided
 *   d_final_state [N, D] f32 contiguous, or data == NULL for zeros
 *   dx           [T, D]  float32 or x's dtype, rows may be strided
 *   dg_log       [T, D]  float32 or g_log's dtype, rows may be strided; the rows of dx
 *                        and dg_log that no sequence covers are written as zeros
 *   d_initial_state [N, D] f32 contiguous, or data == NULL; of an empty sequence its
 *                        d_final_state
 *   workspace    at least gdp_gated_scan_backward_workspace_bytes(...), 256-byte aligned
 * No gradient may overlap an input or another gradient (GDP_EALIAS).  No allocation,
 * everything on `stream`: capturable. */
int gdp_gated_scan_backward(const gdp_tensor *x, const gdp_tensor *g_log, const gdp_tensor *cu_seqlens,
                            int32_t complement_input, const gdp_tensor *initial_state,
                            const gdp_tensor *checkpoints, const gdp_tensor *d_o,
                            const gdp_tensor *d_final_state, const gdp_tensor *dx, const gdp_tensor *dg_log,
                            const gdp_tensor *d_initial_state, void *workspace, size_t workspace_bytes,
                            void *stream);

/* Activations of gdp_group_norm. */
enum gdp_activation { GDP_ACT_NONE = 0, GDP_ACT_SILU = 1, GDP_ACT_SIGMOID = 2 };

/* Device.  Group norm with an activation over the channels of each token, channels
 * last: the G groups of V channels are the heads of a recurrence's output [T, Hv, V].
 * For every token t and group:
 *     n = (x - mean) rstd weight + bias,   rstd = 1 / sqrt(mean((x - mean)^2) + eps),
 *     y = act(n) without a gate,   y = n act(gate) with one;
 * mean is the mean over the group's V channels, or 0 with subtract_mean == 0 (root
 * mean square norm).
 *   x            [T, G, V]  f32, bf16 or f16; tokens and groups may be strided
 *   weight       [V] (one for all groups) or [G, V], f32 or x's dtype, contiguous, or
 *                data == NULL for ones
 *   bias         as weight, or data == NULL for zeros; with a weight its shape and dtype
 *   gate         [T, G, V]  x's dtype, may be strided, or data == NULL
 *   activation   a gdp_activation
 *   eps          at least 2^-126, finite
 *   y            [T, G, V]  x's dtype, may be strided
 * Statistics and products are float32 (the squares of x - mean must stay finite
 * there); y is rounded once.  y may not overlap an input
 * (GDP_EALIAS).  V <= 16384 and G <= 65535 (GDP_EUNSUPPORTED otherwise).  One launch on
 * `stream`; capturable. */
int gdp_group_norm(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, const gdp_tensor *gate,
                   int32_t activation, int32_t subtract_mean, float eps, const gdp_tensor *y, void *stream);

/* Host-only.  Workspace bytes gdp_group_norm_backward needs where a weight or a bias
 * is given: partial sums of their gradients.  0 for invalid sizes. */
size_t gdp_group_norm_backward_workspace_bytes(int64_t T, int64_t G, int64_t V);

/* Device.  Gradients of gdp_group_norm (the same x, weight, bias, gate, activation,
 * subtract_mean and eps) for d_y [T, G, V] of x's dtype:
 *   dx, dgate    [T, G, V]  x's dtype, may be strided; dgate required iff a gate is given
 *   dweight, dbias          f32, contiguous, the shape of weight and bias; required iff
 *                           weight, respectively bias, is given: summed over the tokens
 *                           (and the groups that share them) in a fixed order
 *   workspace    at least gdp_group_norm_backward_workspace_bytes(...), 256-byte aligned;
 *                not used without weight and bias
 * The statistics are formed again from x.  No gradient may overlap an input or another
 * gradient (GDP_EALIAS).  Everything on `stream`, no allocation: capturable. */
int gdp_group_norm_backward(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias,
                            const gdp_tensor *gate, int32_t activation, int32_t subtract_mean, float eps,
                            const gdp_tensor *d_y, const gdp_tensor *dx, const gdp_tensor *dweight,
                            const gdp_tensor *dbias, const gdp_tensor *dgate, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * What stands around a recurrence in a layer: the short convolution before it, a
 * selective state space scan in its place, and the norms before and after the
 * block.  The conventions above hold here too.
 * ------------------------------------------------------------------------ */

/* Device.  Short causal convolution over packed sequences, channel by channel:
 *     v_t = bias + sum_{j < W} weight[d, j] x_{t-W+1+j},   y_t = act(v_t),
 * the W - 1 rows before a sequence's first being its initial state (or zeros).
 *   x            [T, D]    f32, bf16 or f16; rows may be strided; D <= 2^24
 *                          (GDP_EUNSUPPORTED otherwise)
 *   weight       [D, W]    f32 or x's dtype, contiguous; 2 <= W <= 8 (GDP_EUNSUPPORTED
 *                          otherwise)
 *   bias         [D]       weight's dtype, contiguous, or data == NULL for zeros
 *   activation   a gdp_activation
 *   cu_seqlens   [N+1]     int32 or int64, contiguous
 *   initial_state [N, W-1, D]  x's dtype, contiguous: the inputs before each sequence,
 *                          oldest first; or data == NULL for zeros
 *   output_final_state     write final_state when nonzero
 *   state_cache  [S, W-1, D]  x's dtype, contiguous, or NULL; when given, the final state
 *                          of sequence i is written at slot state_indices[i]; an index
 *                          outside [0, S) writes nothing, two sequences naming one slot
 *                          race (caller error)
 *   state_indices [N]      int32 or int64; required with state_cache
 *   y            [T, D]    x's dtype, rows may be strided; rows no sequence covers are left
 *                          as they are
 *   final_state  [N, W-1, D]  x's dtype, contiguous; required iff output_final_state: the
 *                          last W - 1 inputs (of a shorter sequence, its initial state's
 *                          last ones before them)
 * Products and sums are float32, y is rounded once, states are copied.  No output may
 * overlap an input or another output (GDP_EALIAS).  One launch on `stream`; capturable. */
int gdp_short_conv(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation,
                   const gdp_tensor *cu_seqlens, const gdp_tensor *initial_state, int32_t output_final_state,
                   const gdp_tensor *state_cache, const gdp_tensor *state_indices, const gdp_tensor *y,
                   const gdp_tensor *final_state, void *stream);

/* Device.  One token of the convolution per entry, on the state cache in place: for
 * slot = state_indices[i] in [0, S), y[i] from the slot's W - 1 inputs and x[i], which
 * then takes the place of the newest, the others moving up; the other entries (padding,
 * -1) get a zero output row and touch no state.
 *   x, y [N, D], weight, bias, activation as for gdp_short_conv; state_cache [S, W-1, D],
 *   state_indices [N].  Two entries naming one slot race (caller error).  One launch on
 *   `stream`; capturable. */
int gdp_short_conv_decode(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation,
                          const gdp_tensor *state_cache, const gdp_tensor *state_indices, const gdp_tensor *y,
                          void *stream);

/* Host-only.  Workspace bytes gdp_short_conv_backward needs: partial sums of the weights'
 * gradients.  0 for invalid sizes. */
size_t gdp_short_conv_backward_workspace_bytes(int64_t T, int64_t N, int64_t D, int64_t W);

/* Device.  Gradients of gdp_short_conv for d_y [T, D] of x's dtype and d_final_state
 * [N, W-1, D] f32 (or data == NULL for zeros):
 *   dx           [T, D]       x's dtype, rows may be strided; rows no sequence covers are
 *                             written as zeros
 *   dweight      [D, W], dbias [D] (iff a bias is given)  f32, contiguous, summed over the
 *                             tokens in a fixed order
 *   d_initial_state [N, W-1, D]  f32, contiguous, or data == NULL
 *   workspace    at least gdp_short_conv_backward_workspace_bytes(...), 256-byte aligned
 * v_t is formed again from x.  No gradient may overlap an input or another gradient
 * (GDP_EALIAS).  Calls that share a workspace must be ordered.  Everything on `stream`, no
 * allocation: capturable. */
int gdp_short_conv_backward(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation,
                            const gdp_tensor *cu_seqlens, const gdp_tensor *initial_state, const gdp_tensor *d_y,
                            const gdp_tensor *d_final_state, const gdp_tensor *dx, const gdp_tensor *dweight,
                            const gdp_tensor *dbias, const gdp_tensor *d_initial_state, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Rows of a sequence per checkpoint of the selective scan. */
#define GDP_SELECT_CHECKPOINT_ROWS 16

/* Host-only.  Workspace bytes gdp_selective_scan needs: the states at the ends of pieces of
 * long sequences, as many as the rows have, whatever N is.  0 for invalid sizes, and where
 * nothing is needed. */
size_t gdp_selective_scan_workspace_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S);

/* Device.  Selective state space scan over packed sequences, S states h per channel d:
 *     delta_t = softplus(dt_t + dt_bias)  or, without dt_softplus,  dt_t + dt_bias,
 *     h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,
 *     o_t = (C_t . h_t + skip u_t) silu(gate_t),
 * from h = initial_state (or 0) in every sequence; without a gate the last factor is 1.
 *   u            [T, D]    f32, bf16 or f16; rows may be strided; D <= 2^24
 *                          (GDP_EUNSUPPORTED otherwise)
 *   dt           [T, D]    f32 or u's dtype; rows may be strided
 *   A            [D, S]    f32, contiguous, negative (delta_t A > 0 is served while the
 *                          products of decays over 2048 rows stay finite in float32; what
 *                          such a product below 2^-126 leaves of a state may be taken
 *                          for 0); 1 <= S <= 32 (GDP_EUNSUPPORTED otherwise)
 *   B, C         [T, G, S] u's dtype, tokens and groups may be strided; channel d reads
 *                          group d / (D / G)
 *   skip, dt_bias [D]      f32, contiguous, or data == NULL for none
 *   gate         [T, D]    u's dtype, rows may be strided, or data == NULL
 *   cu_seqlens   [N+1]     int32 or int64, contiguous
 *   initial_state [N, D, S]  f32 contiguous, or data == NULL for zeros
 *   output_final_state, state_cache [S', D, S] f32, state_indices [N]  as for gdp_gated_scan
 *   return_checkpoints     write checkpoints when nonzero
 *   o            [T, D]    u's dtype, rows may be strided; rows no sequence covers are left
 *                          as they are
 *   final_state  [N, D, S] f32 contiguous; required iff output_final_state; of an empty
 *                          sequence its initial state
 *   checkpoints  [T / 16 + N, S, D]  f32 contiguous: row cu_seqlens[i] / 16 + i + k holds
 *                          the states entering row 16 k of sequence i, the other rows are
 *                          unspecified; what gdp_selective_scan_backward reads
 *   workspace    at least gdp_selective_scan_workspace_bytes(...), 256-byte aligned
 * States are float32, o is rounded once.  A non-finite input stays within its sequence,
 * and but for B and C within its channel; an infinite state times a product of decays below
 * 2^-126 may be NaN.  No output may overlap an input or another output
 * (GDP_EALIAS).  Calls that share a workspace must be ordered.  Two runs on the same inputs
 * give the same bits.  One to four launches on `stream`, no allocation: capturable. */
int gdp_selective_scan(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                       const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate, const gdp_tensor *dt_bias,
                       int32_t dt_softplus, const gdp_tensor *cu_seqlens, const gdp_tensor *initial_state,
                       int32_t output_final_state, const gdp_tensor *state_cache, const gdp_tensor *state_indices,
                       int32_t return_checkpoints, const gdp_tensor *o, const gdp_tensor *final_state,
                       const gdp_tensor *checkpoints, void *workspace, size_t workspace_bytes, void *stream);

/* Device.  One token of the selective scan per entry, on the state cache in place; entries
 * whose slot lies outside [0, S') (padding, -1) get a zero output row and touch no state.
 *   u, dt, gate, o [N, D], B, C [N, G, S] and the parameters as for gdp_selective_scan;
 *   state_cache [S', D, S] f32 contiguous, state_indices [N] int32 or int64.  Two entries
 *   naming one slot race (caller error).  One launch on `stream`; capturable. */
int gdp_selective_scan_decode(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                              const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate,
                              const gdp_tensor *dt_bias, int32_t dt_softplus, const gdp_tensor *state_cache,
                              const gdp_tensor *state_indices, const gdp_tensor *o, void *stream);

/* Host-only.  Workspace bytes gdp_selective_scan_backward needs; without the forward call's
 * checkpoints, room for them too.  0 for invalid sizes. */
size_t gdp_selective_scan_backward_workspace_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S,
                                                   int32_t with_checkpoints);

/* Device.  Gradients of gdp_selective_scan for d_o [T, D] of u's dtype and d_final_state
 * [N, D, S] f32 (or data == NULL for zeros):
 *   u .. initial_state   the forward call's
 *   checkpoints  those of the forward call, or data == NULL: the states are then formed
 *                again first
 *   du, dgate    [T, D]    u's dtype, rows may be strided (dgate iff a gate is given)
 *   ddt          [T, D]    dt's dtype, rows may be strided
 *   dA           [D, S]    f32, contiguous
 *   dB, dC       [T, G, S] u's dtype, contiguous: sums over the group's channels
 *   dskip, ddt_bias [D]    f32, contiguous; iff skip, respectively dt_bias, is given
 *   d_initial_state [N, D, S]  f32, contiguous, or data == NULL
 *   workspace    at least gdp_selective_scan_backward_workspace_bytes(...), 256-byte aligned
 * Rows no sequence covers are written as zeros; sums over tokens and channels are float32, in
 * a fixed order.  No gradient may overlap an input or another gradient (GDP_EALIAS).
 * Calls that share a workspace must be ordered.  Everything on `stream`, no allocation:
 * capturable. */
int gdp_selective_scan_backward(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                                const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate,
                                const gdp_tensor *dt_bias, int32_t dt_softplus, const gdp_tensor *cu_seqlens,
                                const gdp_tensor *initial_state, const gdp_tensor *checkpoints, const gdp_tensor *d_o,
                                const gdp_tensor *d_final_state, const gdp_tensor *du, const gdp_tensor *ddt,
                                const gdp_tensor *dA, const gdp_tensor *dB, const gdp_tensor *dC,
                                const gdp_tensor *dskip, const gdp_tensor *dgate, const gdp_tensor *ddt_bias,
                                const gdp_tensor *d_initial_state, void *workspace, size_t workspace_bytes,
                                void *stream);

/* Device.  The norms after a block and before the next one, with the block's gate, the
 * residual scale and the residual sum between them.  Per token, over all D channels:
 *     p = y rstd(y) post_weight,  or  y post_weight  without post_norm,
 *     r = x + residual_scale f(gate) p,      n = r rstd(r) pre_weight,
 * rstd(v) = 1 / sqrt(mean(v^2) + eps), f the gate's activation (1 without a gate).
 *   x            [T, D]  residual stream, f32 or y's dtype; rows may be strided
 *   y            [T, D]  block's output, f32, bf16 or f16; rows may be strided
 *   post_weight, pre_weight [D]  f32 or y's dtype (one dtype for both), contiguous, or
 *                data == NULL for ones; pre_weight only with pre_norm
 *   gate         [T, D]  y's dtype, rows may be strided, or data == NULL
 *   gate_activation  a gdp_activation; GDP_ACT_NONE without a gate
 *   eps          at least 2^-126, finite
 *   r            [T, D]  x's dtype, rows may be strided; it may be x itself (same address,
 *                dtype and strides), which is then updated in place
 *   n            [T, D]  y's dtype, rows may be strided; required iff pre_norm
 * Sums and products are float32 (the squares of y and r must stay finite there); r and n
 * are rounded once, n from the r before its rounding.  Otherwise no output may overlap
 * an input or another output (GDP_EALIAS).  D <= 16384 (GDP_EUNSUPPORTED otherwise).  One
 * launch on `stream`; capturable. */
int gdp_residual_norm(const gdp_tensor *x, const gdp_tensor *y, const gdp_tensor *post_weight,
                      const gdp_tensor *pre_weight, const gdp_tensor *gate, int32_t gate_activation, int32_t post_norm,
                      int32_t pre_norm, float residual_scale, float eps, const gdp_tensor *r, const gdp_tensor *n,
                      void *stream);

/* Host-only.  Workspace bytes gdp_residual_norm_backward needs where a weight is given:
 * partial sums of the weights' gradients.  0 for invalid sizes. */
size_t gdp_residual_norm_backward_workspace_bytes(int64_t T, int64_t D);

/* Device.  Gradients of gdp_residual_norm (the same inputs) for d_r [T, D] of x's dtype (or
 * data == NULL for zeros, with pre_norm) and d_n [T, D] of y's dtype (iff pre_norm):
 *   dx           [T, D]  x's dtype; dy, dgate (iff a gate is given) [T, D]  y's dtype; rows
 *                may be strided
 *   dpost_weight, dpre_weight [D]  f32, contiguous; iff the weight is given: summed over the
 *                tokens in a fixed order
 *   workspace    at least gdp_residual_norm_backward_workspace_bytes(...), 256-byte aligned;
 *                not used without weights
 * r is formed again from x, y and gate (a call that updated x in place has lost it).  No
 * gradient may overlap an input or another gradient (GDP_EALIAS).  Calls that share a
 * workspace must be ordered.  Everything on `stream`, no allocation: capturable. */
int gdp_residual_norm_backward(const gdp_tensor *x, const gdp_tensor *y, const gdp_tensor *post_weight,
                               const gdp_tensor *pre_weight, const gdp_tensor *gate, int32_t gate_activation,
                               int32_t post_norm, int32_t pre_norm, float residual_scale, float eps,
                               const gdp_tensor *d_r, const gdp_tensor *d_n, const gdp_tensor *dx,
                               const gdp_tensor *dy, const gdp_tensor *dpost_weight, const gdp_tensor *dpre_weight,
                               const gdp_tensor *dgate, void *workspace, size_t workspace_bytes, void *stream);

/* Debug validation of the data-dependent arguments.  These are not checked by
 * default, because checking them needs a read of device data.  A bad value stays
 * in bounds (every kernel clamps sequence ranges to [0, T] and skips slots
 * outside the cache), but the results are then undefined.  With the environment
 * variable GDP_DEBUG_VALIDATE=1, gdp_chunk_prefill (and the entries built on it),
 * gdp_recurrent_decode, the gated scan's, the short convolution's and the selective
 * scan's entries first launch a check on their stream.  The check ORs
 * these bits into a word kept per device:
 *   GDP_DBG_CU    cu_seqlens decreases somewhere, or an entry lies outside [0, T]
 *                 (Megatron Core page, chunk_gated_delta_product_varlen: the
 *                 cumulative sequence boundaries)
 *   GDP_DBG_SLOT  a state index below -1 or not below the number of cache slots
 *   GDP_DBG_DUP   two sequences (decode entries) share a non-negative state
 *                 index (same page, the state-cache arguments: -1 means no write)
 * The duplicate check is quadratic in the number of sequences: it is a
 * debugging aid, not for production steps. */
enum gdp_debug_bits { GDP_DBG_CU = 1, GDP_DBG_SLOT = 2, GDP_DBG_DUP = 4 };

/* Host-side: reads the current device's debug word into *word (host memory)
 * after the work queued on `stream` so far, then, if clear != 0, queues its
 * reset to 0 on `stream`.  Synchronises `stream`.  GDP_EINVAL if word is NULL,
 * GDP_EHIP on a runtime failure. */
int gdp_debug_status(uint32_t *word, int32_t clear, void *stream);

/* Message of the last failed call on this thread ("" if none).  A request the
 * library does not serve is declined with GDP_EUNSUPPORTED and its reason left
 * here rather than aborting the caller, the way the FlashInfer page
 * (flashinfer.gdp_prefill.chunk_gated_delta_product, requirements note) has an
 * engine decline a graph it cannot serve and log why. */
const char *gdp_last_error(void);

/* Library version string.  Informational; no passage of the pages defines it. */
const char *gdp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDP_H */
