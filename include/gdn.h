/*
 * gdn.h -- C ABI of libgdn, the MI355X (gfx950) gated delta-rule library.
 *
 * The method: per head, a d_k x d_v associative state S is carried over the
 * sequence and updated by a gated delta rule,
 *
 *     S_t = alpha_t (I - beta_t k_t kread_t^T) S_{t-1} + beta_t k_t v_t^T,
 *     o_t = S_t^T qread_t,
 *
 * where kread = k, qread = q for real data and kread = conj(k), qread = conj(q)
 * for complex data.  References for each piece:
 *   - rank-one delta write with a keyed readout and residual error:
 *     DeltaPhase README, section 2 "Complex Phase Matrix Delta Memory";
 *   - the data-dependent forget gate alpha_t: Sykra 0.3.3 README,
 *     "Architectural Highlights" (data-dependent forget gating); the gate
 *     scales the whole updated state (Gated DeltaNet ordering, named in the
 *     DeltaPhase lineage list);
 *   - beta in (0, 2) as the extended Householder range: DeltaPhase README,
 *     section 1 "Extended Householder Beta Range";
 *   - the chunkwise-parallel evaluation (WY / unit triangular transform) that
 *     gdn_chunk_fwd implements: Sykra README, "Architectural Highlights"
 *     (chunkwise parallel training), DeltaPhase README, section 1 "Fast
 *     Triangular Solve", and section 5 (log-space factorisation of the decay);
 *   - the O(d^2) single-token step of gdn_recurrent_step: Sykra README,
 *     "Computational Complexity" table (inference step time O(d^2), fixed state).
 * Around that forward: gdn_chunk_fwd_prologue folds the layer's input
 * transforms (L2 norms, gate logits) into it; gdn_chunk_bwd returns its
 * gradients; gdn_fwd_channel_decay replaces the scalar gate with a decay per
 * value channel (DeltaPhase README, section 5).
 *
 * Conventions shared by every entry point
 *   - All pointers are DEVICE pointers (memory the caller allocated on the
 *     current HIP device), except where stated.  The library allocates
 *     nothing and keeps no state besides a cached device-property query.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL means the null
 *     stream) and the call returns without synchronising.
 *   - Argument errors are reported synchronously, before anything is
 *     launched, and no output is touched.  A launch failure returns
 *     GDN_ERR_HIP.  Faults during execution surface at the caller's next
 *     synchronisation of the stream.  No C++ exception crosses this ABI.
 *   - Calls are thread-safe.  Two calls that write the same buffers must be
 *     ordered by the caller.
 *   - Element types: `dtype` selects the storage of q, k, v and out:
 *       GDN_F32  float32, GDN_BF16 bfloat16, GDN_C64 complex64 (interleaved
 *       re, im float32).  alpha and beta are always float32.  States (S0,
 *       S_final, S) are float32, or complex64 when dtype == GDN_C64.
 *       Gradients from gdn_chunk_bwd are float32.
 *   - Every pointer must be 16-byte aligned.
 *   - Size limits (GDN_ERR_SHAPE otherwise): no tensor above 2^40 elements;
 *     B * H below 2^20 for the chunk forwards, below 2^23 for the backward,
 *     below 2^22 for the channel-decay forward; N below 2^24 for the decode
 *     step.  These keep every launch under 2^32 work-items.
 *   - Preconditions not checked on the device (violations give undefined,
 *     typically non-finite, results): 0 < alpha <= 1, 0 <= beta <= 2, finite
 *     inputs.  Inputs and outputs must not overlap, except that S_final may
 *     equal S0.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
enum {
  GDN_OK = 0,
  GDN_ERR_NULL = 1,        /* a required pointer is NULL                     */
  GDN_ERR_SHAPE = 2,       /* a size is negative or the total is too large   */
  GDN_ERR_DTYPE = 3,       /* dtype is not one of GDN_F32, GDN_BF16, GDN_C64 */
  GDN_ERR_UNSUPPORTED = 4, /* valid but not supported (chunk, head dims)     */
  GDN_ERR_ALIGN = 5,       /* a pointer is not 16-byte aligned              */
  GDN_ERR_WORKSPACE = 6,   /* workspace missing or smaller than required     */
  GDN_ERR_HIP = 7          /* the HIP runtime reported an error on launch    */
};

/* Element types (the `dtype` argument). */
enum { GDN_F32 = 0, GDN_BF16 = 1, GDN_C64 = 2 };

/*
 * Bytes of device workspace gdn_chunk_fwd needs for these sizes; 0 means the
 * call may pass workspace = NULL.  Returns 0 also for unsupported arguments
 * (gdn_chunk_fwd then reports the error).
 *
 * GDN_BF16 and GDN_F32 need none.  GDN_C64 needs B * H * ceil(T / 64) * 57600
 * bytes: per chunk the factors -W and U, (diag(lambda) K)^T, the decay
 * prefix and the chunk-start state, handed between its three launches.  The
 * caller owns the workspace; its contents are scratch on entry and exit.  Two
 * calls may share one workspace only if they are ordered (same stream).
 */
size_t gdn_chunk_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, int chunk, int dtype);

/*
 * Chunkwise-parallel forward of the gated delta rule over whole sequences.
 *
 *   q, k      [B, T, H, dk]  dtype          queries and keys (row-major, d fastest)
 *   v         [B, T, H, dv]  dtype          values
 *   alpha     [B, T, H]      float32        forget gate, 0 < alpha <= 1
 *   beta      [B, T, H]      float32        write strength, 0 <= beta <= 2
 *   S0        [B, H, dk, dv] state type     initial state (row = key dim); NULL -> zeros
 *   chunk                                    chunk length C; 64 is supported
 *   out       [B, T, H, dv]  dtype          o_t for every token
 *   S_final   [B, H, dk, dv] state type     state after token T-1; NULL -> not written;
 *                                            may be the same buffer as S0
 *   workspace, workspace_bytes               device scratch, at least
 *                                            gdn_chunk_fwd_workspace_bytes(...) bytes
 *   stream                                   hipStream_t to enqueue on
 *
 * Supported: chunk == 64; dk == dv in {64, 128} for GDN_BF16; dk == dv == 64
 * for GDN_F32; dk == dv == 32 for GDN_C64.  Any T >= 0 (T % 64 != 0 is handled exactly:
 * the tail chunk is shorter).  B == 0, H == 0 or T == 0 with S_final given
 * copies S0 (or zeros) into S_final.
 *
 * Arithmetic: bf16 inputs are multiplied on bf16 matrix cores with fp32
 * accumulation; the state is carried in fp32.  fp32 and complex64 inputs use
 * fp32 matrix cores throughout.
 */
int gdn_chunk_fwd(const void *q, const void *k, const void *v, const float *alpha, const float *beta,
                  const void *S0, int chunk, void *out, void *S_final, int B, int T, int H, int dk,
                  int dv, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace gdn_chunk_fwd_prologue needs for these sizes (0:
 * workspace may be NULL; 0 also for unsupported arguments).  bf16: 0 where
 * gdn_chunk_fwd needs no workspace; otherwise (the two-launch path) what
 * gdn_chunk_fwd needs plus B * H * ceil(T / 64) * 256 bytes, the inverse key
 * norms handed from the first launch to the second.  GDN_F32 and GDN_C64: the
 * transformed q and k (B * T * H rows of 256 bytes each) and the two gates
 * (B * T * H floats each), each rounded up to 256 bytes, plus, for GDN_C64,
 * what gdn_chunk_fwd needs.  Ownership and sharing as for gdn_chunk_fwd.
 */
size_t gdn_chunk_fwd_prologue_workspace_bytes(int B, int T, int H, int dk, int dv, int chunk, int dtype);

/*
 * gdn_chunk_fwd for a layer's raw projections, with its input transforms
 * applied on the device:
 *
 *   q_t <- q_t / max(|q_t|, 1e-12),  k_t <- k_t / max(|k_t|, 1e-12)
 *          (L2 over the key dimension, per token and head; the unit-norm keys
 *          and queries the chunkwise form is usually run on; for complex
 *          rows the Hermitian norm, sum over i of |q_i|^2)
 *   beta_t  = beta_scale * sigmoid(b_t)
 *          (DeltaPhase README, section 1 "Extended Householder Beta Range":
 *          beta_scale = 2 gives beta in (0, 2); 1 gives (0, 1))
 *   alpha_t = exp(-softplus(a_t)) = 1 / (1 + e^{a_t})
 *          (the data-dependent forget gate of the Sykra README, "Architectural
 *          Highlights", as a logistic map of a logit into (0, 1))
 *
 *   q, k      [B, T, H, dk]  dtype      raw queries and keys
 *   v         [B, T, H, dv]  dtype      values
 *   a_logit   [B, T, H]      float32    forget-gate logits
 *   b_logit   [B, T, H]      float32    write-strength logits
 *   beta_scale                          finite, 0 <= beta_scale <= 2
 *   workspace  device memory of at least
 *              gdn_chunk_fwd_prologue_workspace_bytes(...) bytes, or NULL when
 *              that is 0
 *   S0, chunk, out, S_final, B, T, H, dk, dv, dtype, stream: as for
 *   gdn_chunk_fwd.
 *
 * Supported: the shapes gdn_chunk_fwd supports (bf16 d = 64 or 128, fp32
 * d = 64, complex64 d = 32; dk == dv; chunk == 64), except bf16 shapes with a
 * batch row of q, k, v or out of 2^31 bytes or more, and bf16 d = 128 grids of
 * 2^26 chunks (B * H * ceil(T / 64)) or more (GDN_ERR_UNSUPPORTED).
 *
 * bf16 fuses the transforms into the forward's kernels, so q, k and the
 * logits are read once, as stored, and the rows are never rewritten: 1/|k|
 * and 1/|q| scale the Gram tiles, the decay factors and the per-token gates
 * (on the two-launch path, d = 128 and long d = 64 sequences, the first
 * launch forms both and the second reads them).  fp32 and complex64
 * run one extra pass over the rows that writes the transformed q, k and gates
 * to the workspace; there alpha is kept at or above 2^-126 (a logit above 87
 * already gives a gate that wipes the state).
 */
int gdn_chunk_fwd_prologue(const void *q, const void *k, const void *v, const float *a_logit,
                           const float *b_logit, float beta_scale, const void *S0, int chunk, void *out,
                           void *S_final, int B, int T, int H, int dk, int dv, int dtype, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * Bytes of workspace gdn_chunk_bwd needs.  bf16 (the chunk form): per
 * (chain, 64-token chunk) two 6400-byte factor records, a bf16 start state and
 * a bf16 end gradient (2 * 6400 + 2 * 64 * 64 * 2 bytes), plus the forward's
 * segment maps when it splits long sequences (as gdn_chunk_fwd_workspace_bytes
 * reports them).  fp32 (d = 64) and complex64 (d = 32): the forward state
 * every 8 tokens, B * H * ceil(T / 8) * d * d * e bytes (e = 4 or 8), plus the
 * shares of dq, dk, dalpha and dbeta from each of the n column groups (n = 8:
 * d / 8 for fp32, d / 4 for complex64), n * B * T * H * (2 * d * e + 8) bytes.
 * 0 for an unsupported combination.
 */
size_t gdn_chunk_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, int dtype);

/*
 * Reverse-mode gradients of gdn_chunk_fwd: given the gradients grad_out of
 * out and grad_S_final of S_final, the gradients of the real loss
 * sum(out * grad_out) + sum(S_final * grad_S_final) with respect to q, k, v,
 * alpha, beta and S0.  For complex data the loss is
 * Re sum(conj(grad_out) out) + Re sum(conj(grad_S_final) S_final), and the
 * gradient of a complex value z is dL/dRe(z) + i dL/dIm(z) (the upstream
 * gradients are given the same way); alpha and beta stay real.  The forward is the recurrence of DeltaPhase README
 * section 2 with the data-dependent forget gate of the Sykra README
 * ("Architectural Highlights"), applied to the whole Householder-updated
 * state, as for gdn_chunk_fwd; the gradients follow it token by token in
 * reverse.  The pages train through this layer; they print no gradient
 * formula.
 *
 *   q, k, v, alpha, beta, S0   the forward's inputs, as for gdn_chunk_fwd
 *                              (S0 may be NULL: zero)
 *   grad_out      [B, T, H, dv]  dtype     gradient of out
 *   grad_S_final  [B, H, dk, dv] float32 (complex64 for GDN_C64)   gradient
 *                 of S_final (NULL: zero)
 *   grad_q, grad_k [B, T, H, dk], grad_v [B, T, H, dv]   float32 (complex64
 *                 for GDN_C64), written
 *   grad_alpha, grad_beta [B, T, H]                      float32, written
 *   grad_S0       [B, H, dk, dv] float32 (complex64 for GDN_C64), written
 *                 (NULL: not computed)
 *   (for GDN_C64 the float pointers hold complex64 as interleaved re, im)
 *   workspace     device memory of at least gdn_chunk_bwd_workspace_bytes(...)
 *                 bytes, owned by the caller, overwritten (may be NULL when
 *                 that is 0)
 *
 * Supported: GDN_F32 with dk == dv == 64, GDN_BF16 with dk == dv == 64 or
 * 128, GDN_C64 with dk == dv == 32, any T >= 0 with T * H * 4 < 2^31;
 * otherwise GDN_ERR_UNSUPPORTED.
 * bf16 inputs take the chunk form on the matrix cores (the same chunking as
 * gdn_chunk_fwd, run in reverse: the forward's chunk start states, then the
 * gradient carried from the last chunk to the first, then every chunk's
 * gradients at once), with bf16 operands and fp32 accumulation, like the
 * forward.  fp32 and complex64 inputs take a token-by-token reverse pass in
 * fp32 throughout (checkpoints every 8 tokens), split by groups of state
 * columns, 8 for fp32 and 4 for complex64 (the columns evolve independently;
 * a second launch adds the groups' shares of dq, dk, dalpha and dbeta).  The forward is recomputed inside the call, so
 * nothing from a forward call is needed.  Gradient outputs must not alias any
 * input.  alpha must be positive (the chunk form works with log alpha).
 * B * H == 0 is a no-op; T == 0 copies grad_S_final (or zeros) to grad_S0.
 * Errors as for gdn_chunk_fwd.
 */
int gdn_chunk_bwd(const void *q, const void *k, const void *v, const float *alpha, const float *beta,
                  const float *S0, const void *grad_out, const float *grad_S_final, float *grad_q,
                  float *grad_k, float *grad_v, float *grad_alpha, float *grad_beta, float *grad_S0,
                  int B, int T, int H, int dk, int dv, int dtype, void *workspace,
                  size_t workspace_bytes, void *stream);

/*
 * The forward with a per-output-channel decay in place of the scalar gate,
 * LaplacePhaseCore's gated-decay rule (DeltaPhase README, section 2: the
 * memory is read through the key BEFORE it decays, and the error is written
 * along the key; section 5: the decay diag(r_t) sits on the memory's output
 * rows, one factor per value channel).  With S [dk, dv] (row = key dim),
 * for every value channel j:
 *
 *   e_t[j] = v_t[j] - kr_t^T s_j,   s_j <- r_t[j] s_j + beta_t k_t e_t[j],
 *   o_t[j] = qr_t^T s_j            (the updated state)
 *
 * with kr = k, qr = q for real data and kr = conj(k), qr = conj(q) for
 * complex data (LaplacePhaseCore's keys are complex, e^{s dt}), i.e.
 * S_t = S_{t-1} diag(r_t) + beta_t k_t (v_t - S_{t-1}^T kr_t)^T.  With every
 * r_t[j] = 1 it is gdn_chunk_fwd at alpha = 1.  (With r < 1 it differs from
 * gdn_chunk_fwd's ordering, where the gate also scales the erased part.)
 *
 *   q, k     [B, T, H, dk]  dtype    keys of norm <= 1 for a stable update
 *   v        [B, T, H, dv]  dtype
 *   r        [B, T, H, dv]  float32  decay per token and value channel, in (0, 1]
 *   beta     [B, T, H]      float32
 *   S0       [B, H, dk, dv] state    may be NULL (zero)
 *   out      [B, T, H, dv]  dtype, written
 *   S_final  [B, H, dk, dv] state, written; may be NULL, may equal S0
 *
 * The state is float32 for real data and complex64 (interleaved re, im) for
 * GDN_C64.  Supported: dtype GDN_F32 or GDN_BF16 with dk == dv == 64, or
 * GDN_C64 with dk == dv == 32, any T >= 0; otherwise GDN_ERR_UNSUPPORTED.
 * fp32 arithmetic.  No workspace.  B * H == 0
 * is a no-op; T == 0 copies S0 (or zeros) to S_final.  Errors as for
 * gdn_chunk_fwd.
 */
int gdn_fwd_channel_decay(const void *q, const void *k, const void *v, const float *r, const float *beta,
                          const float *S0, void *out, float *S_final, int B, int T, int H, int dk, int dv,
                          int dtype, void *stream);

/*
 * gdn_chunk_fwd for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments and results as gdn_chunk_fwd, without the workspace: the
 * call takes it from a fixed device array that the library keeps per device,
 * from the first call on that device until the process ends.  The call
 * itself allocates nothing (no hipMalloc, hipFree or allocating library
 * routine).
 *
 * Limit: GDN_NOALLOC_MAX_WORKSPACE bytes (128 MiB), compared with
 * gdn_chunk_fwd_workspace_bytes(...) for the same sizes; a call that needs
 * more returns GDN_ERR_WORKSPACE before anything is launched.  Calls that need
 * no workspace (fp32, and bf16 d = 64 with enough chains) use none.
 *
 * All calls on one device share the array: calls that may overlap on one
 * device (different streams, unordered host threads) race and give wrong
 * results.  Order them (one stream) or use gdn_chunk_fwd with a workspace of
 * your own.  Other errors as for gdn_chunk_fwd; GDN_ERR_HIP if the array's
 * device address cannot be found.
 */
int gdn_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const float *alpha,
                          const float *beta, const void *S0, int chunk, void *out, void *S_final,
                          int B, int T, int H, int dk, int dv, int dtype, void *stream);
#define GDN_NOALLOC_MAX_WORKSPACE ((size_t)128 << 20)

/*
 * One single-token decode step on N independent states, in place.
 *
 *   q, k   [N, dk] dtype;  v [N, dv] dtype;  alpha, beta [N] float32
 *   S      [N, dk, dv] state type, read and overwritten with the new state
 *   out    [N, dv] dtype, o = S_new^T qread
 *
 * Supported: dk == dv == 64 or 128 for GDN_F32 / GDN_BF16; 32 for GDN_C64.
 * N == 0 is a no-op.  The state is read once and written once.
 */
int gdn_recurrent_step(const void *q, const void *k, const void *v, const float *alpha,
                       const float *beta, void *S, void *out, int N, int dk, int dv, int dtype,
                       void *stream);

/* ------------------------------------------------------------------------
 * Softmax attention: the layers of a hybrid model that stand between its
 * delta-rule layers (Sykra 0.3.3 README, "Architectural Highlights": one layer
 * in four).  Whole prompts and their gradients, and a paged 8-bit cache for
 * the tokens that follow.
 *
 * Shared by the entry points below
 *   - Hq query heads read Hkv key heads, Hq a multiple of Hkv: query head h
 *     reads key head h / (Hq / Hkv).  D, the head size, is 64 or 128.
 *   - q, k, v, out and gradients are bf16 (dtype GDN_BF16; others
 *     GDN_ERR_UNSUPPORTED).  A row (one token) holds its heads one after the
 *     other; the distance between rows is an argument, in elements, at least
 *     the row's length and a multiple of 8, so that the parts of one fused
 *     projection can be passed as they are.
 *   - scale is finite, of either sign (others GDN_ERR_SHAPE).  Scores (scale
 *     q.k) are float32 numbers and below 2^30 in magnitude: as they grow, their
 *     exponentials lose what their fraction does.
 *   - Softmax statistics and every sum are float32; probabilities are rounded
 *     to 16 bits where they enter a matrix product.
 *   - lse is the natural logarithm of a row's sum of exp(scale q.k), float32.
 *   - Lengths, offsets, tables and slots are int32 on the device.  Their
 *     values are not known to the call: entries that would lead outside the
 *     buffers are clamped or skipped as described, never followed.
 *   - A cache holds `num_blocks` blocks of `block_tokens` tokens (16, 32, 64
 *     or 128), stored [num_blocks, Hkv, block_tokens, D] in 8 bits with one
 *     float32 scale per (block, key head), stored [num_blocks, Hkv]; a value
 *     is its code times its scale.  num_blocks * block_tokens is below 2^31.
 *   - What a call writes overlaps nothing that it reads, but for the tables and
 *     caches that it updates in place.
 *   - Errors as for gdn_chunk_fwd.
 * ------------------------------------------------------------------------ */

/* Codes of a cache (the `cache_format` argument). */
enum { GDN_CACHE_I8 = 0,   /* signed integers in [-127, 127]                  */
       GDN_CACHE_E4M3 = 1  /* 8-bit floats, OCP e4m3, largest 448             */ };

/*
 * Block tables and slots of a step, from the requests' lengths.
 *
 *   seq_lens, new_lens  [R] tokens held, tokens that this step adds
 *   block_table [R, width]  row r: the blocks of request r in order; entries
 *               past those that seq_lens[r] tokens occupy are ignored.  The
 *               blocks that the new tokens need are appended in place.
 *   free_blocks [n_free]  blocks to hand out, taken from the front in the
 *               order of the requests
 *   slot_map [T]  written: for each new token (packed, request after request)
 *               block * block_tokens + offset; -1 behind the last token and
 *               for tokens of refused requests
 *   cu_seqlens [R + 1]  written: offsets of the requests' new tokens, at most T
 *   lens_after [R]  written: tokens held afterwards; may not alias seq_lens
 *   used [2]    written: how many free blocks were taken; how many requests
 *               were refused
 *
 * A request is refused if a length is negative, its blocks exceed the table's
 * width, its tokens exceed the slot map, or the free list does not reach its
 * blocks (the needs of every request before it count, refused or not, unless
 * their own lengths are at fault).  A refused request keeps its table row and
 * its length; a negative new length counts as no tokens.  A block outside
 * [0, num_blocks) gets slot -1.  R below 2^20, T below 2^31 - 2^12.  One launch.
 */
int gdn_block_tables(const int *seq_lens, const int *new_lens, int *block_table, const int *free_blocks,
                     int *slot_map, int *cu_seqlens, int *lens_after, int *used, int R, int width, int n_free,
                     int block_tokens, int num_blocks, int T, void *stream);

/*
 * Writes rows of keys and values into the cache.
 *
 *   k, v       [T] rows of Hkv * D bf16 values, k_stride and v_stride apart
 *   slot_map   [T] slots as from gdn_block_tables; tokens whose slot lies
 *              outside the cache are skipped
 *   k_cache, v_cache, k_scale, v_scale  updated in place
 *
 * For each (block, head) that new rows fall into, with a = max |x| over them
 * and M = 127 (int8) or 448 (e4m3):
 *     s = max(a (1 / M), old scale if older rows stand before the new ones, 2^-100)
 *     code = rne(x / s);   older codes = rne(code * old / s) if s grew.
 * a (1 / M) is the float32 product with the float32 reciprocal, x / s the float32
 * product x * (1 / s); old / s is a float32 quotient.
 * A value of int8 is off by at most s / 2 when it is written, and by as much
 * again, of the scale then, for each later call in which its block's scale grows:
 * k growths leave at most (k + 1) s / 2, or s where each at least doubles it.  For
 * e4m3 each of these roundings is 2^-4 of the value, or 2^-10 s if that is more.
 * Rows behind the new ones are left as they were.  A block whose first row is
 * new starts a scale of its own, whatever its scale was.  NaN is stored as
 * zero, infinities as the largest code of the largest bf16 value's scale.
 *
 * No two tokens may have the same slot, and the tokens of one block must
 * follow one another in the call with consecutive slots (each one more than the
 * one before it, none left out between), as gdn_block_tables gives them;
 * otherwise that block's contents and scale are undefined: rows behind a gap are
 * taken for a write of their own, at the same time as those before it.
 * T * Hkv below 2^28.
 */
int gdn_cache_append(const void *k, const void *v, const int *slot_map, void *k_cache, void *v_cache,
                     float *k_scale, float *v_scale, long long k_stride, long long v_stride, int T, int Hkv,
                     int D, int block_tokens, int num_blocks, int dtype, int cache_format, void *stream);

/*
 * Attention of one new token per request over the cache.
 *
 *   q          [R] rows of Hq * D, q_stride apart
 *   block_table [R, width], seq_lens [R]: request r attends to the first
 *              seq_lens[r] tokens of its blocks (at most width *
 *              block_tokens).  Blocks outside [0, num_blocks) are left out.
 *   out        [R, Hq, D] written;  lse [R, Hq] written, may be NULL
 *
 * A request without tokens gets zeros and an lse of -infinity.  What the cache
 * holds behind a request's last token is never used, whatever its bits.
 * A token's probability times its v scale is rounded to fp16: to 2^-11 of itself,
 * or 2^-40 of the request's largest where that is more (below e^-20 of it).
 * Scales are positive normal numbers; where scores pass 2^23, those of v lie
 * between 2^-16 and 2^16.  Workspace:
 * gdn_attn_decode_workspace_bytes, which is 0 where the table is narrow;
 * scratch on entry and exit, no clearing needed.  R is below 2^20, R * Hq below
 * 2^23, width * block_tokens below 2^31 - 2^12, R times the table's 128-token
 * units and one below 2^31.
 */
size_t gdn_attn_decode_workspace_bytes(int R, int Hq, int Hkv, int D, int block_tokens, int width);
int gdn_attn_decode(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                    const float *v_scale, const int *block_table, const int *seq_lens, void *out, float *lse,
                    float scale, long long q_stride, int R, int Hq, int Hkv, int D, int block_tokens,
                    int num_blocks, int width, int dtype, int cache_format, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * Causal attention over whole prompts, packed one after the other.
 *
 *   q, k, v    [T] rows of Hq * D, Hkv * D, Hkv * D
 *   cu_seqlens [R + 1] ascending: sequence r is the rows cu_seqlens[r] to
 *              cu_seqlens[r + 1] - 1; row i attends to the rows of its
 *              sequence up to itself.  Lengths of zero are fine.
 *   out        [T, Hq, D] written;  lse [Hq, T] written
 *
 * Rows in no sequence (before cu_seqlens[0], from cu_seqlens[R] on) are left
 * as they were in out and lse, or, where zero_rest is not 0, set to zero.
 * Values of masked keys and rows never reach a result, whatever they are.
 * T * Hq and the row strides are below 2^28 and 2^24.
 */
int gdn_attn_prompt(const void *q, const void *k, const void *v, const int *cu_seqlens, void *out, float *lse,
                    float scale, long long q_stride, long long k_stride, long long v_stride, int T, int R, int Hq,
                    int Hkv, int D, int dtype, int zero_rest, void *stream);

/*
 * Gradients of sum(out * grad_out) for gdn_attn_prompt's forward, from the out
 * and lse that it returned.
 *
 *   grad_out, grad_q  [T] rows of Hq * D;  grad_k, grad_v  [T] rows of Hkv * D,
 *              summed over the query heads that share them; bf16
 *
 * Each gradient is summed in float32 in a fixed order and rounded once, to
 * bf16; probabilities and score gradients are rounded to bf16 where they enter
 * a product (grad_q: score gradients in two parts, to 2^-16).  Rows in no sequence: as for the forward.  A non-finite value
 * of a row gives non-finite gradients where its row's probabilities reach, and
 * none outside its sequence.  Workspace: gdn_attn_prompt_bwd_workspace_bytes,
 * scratch on entry and exit, no clearing needed.
 */
size_t gdn_attn_prompt_bwd_workspace_bytes(int T, int Hq, int Hkv, int D);
int gdn_attn_prompt_bwd(const void *q, const void *k, const void *v, const void *out, const float *lse,
                        const void *grad_out, const int *cu_seqlens, void *grad_q, void *grad_k, void *grad_v,
                        float scale, long long q_stride, long long k_stride, long long v_stride,
                        long long grad_out_stride, long long grad_q_stride, long long grad_k_stride,
                        long long grad_v_stride, int T, int R, int Hq, int Hkv, int D, int dtype, int zero_rest,
                        void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * What stands around a recurrent layer's state update: the norm before its
 * projections, the short convolution behind them, and a selective state space
 * scan in the delta rule's place.
 *
 * Shared by the entry points below
 *   - Rows are packed: T tokens, one after the other; the distance between rows
 *     is an argument, in elements, at least the row's length and a multiple of 8,
 *     so that parts of one fused projection can be passed as they are.  Outputs
 *     without a stride are dense.
 *   - Rows are bf16 or float32 (dtype), parameters of the same type or float32
 *     (weight_dtype; float32 rows have float32 parameters).  All arithmetic is
 *     float32; results are rounded once, to nearest even.
 *   - cu_seqlens [R + 1] int32, ascending: sequence r is the rows cu_seqlens[r]
 *     to cu_seqlens[r + 1] - 1.  Lengths of zero are fine.  The values are not
 *     known to the call: what would lead outside the T rows is clamped.
 *     Rows in no sequence are left as they were, or, where zero_rest is not 0,
 *     set to zero; nothing that they hold reaches a result.
 *   - Sums over rows (gradients of parameters) are made in a fixed order.
 *   - What a call writes overlaps nothing that it reads, but for the states that
 *     a step updates in place, and the norm's rows: out and sum may be x or residual,
 *     grad_x may be sum, grad_out or grad_sum, where those rows are C apart.
 *     Otherwise results that are the very rows or states that are read are refused
 *     (GDN_ERR_UNSUPPORTED).
 *   - Errors as for gdn_chunk_fwd.
 * ------------------------------------------------------------------------ */

/*
 * Root-mean-square norm of rows, with the residual's addition:
 *
 *     s = round(x + residual),   out = s weight / sqrt(mean(s^2) + eps)
 *
 *   x, residual [T] rows of C values, x_stride and residual_stride apart;
 *              residual may be NULL: s is x
 *   weight     [C]
 *   out        [T, C] written;  sum [T, C] written: s (not without a residual)
 *
 * s is rounded to the rows' type before it is normalised: the norm is that of
 * what the next block reads.  C is a multiple of 8 and at most 16384, T below
 * 2^24; eps is finite and not negative.  Squares are summed in float32: rows
 * whose squares add up past its range come out as zeros.
 */
int gdn_rms_norm(const void *x, const void *residual, const void *weight, void *out, void *sum, float eps,
                 long long x_stride, long long residual_stride, int T, int C, int dtype, int weight_dtype,
                 void *stream);

/*
 * The same with an output in 8 bits (format: the codes of a cache), for a
 * product in 8 bits of the caller's: a value is its code times its scale.
 *
 *   codes [T, C] written;  scale written: [T, C / 128] where block is 128 (C a
 *   multiple of it), [T] where block is 0 (a scale to a row)
 *
 * With y the value that gdn_rms_norm would round, a = max |y| over a scale's
 * values and M = 127 (int8) or 448 (e4m3):
 *     scale = max(a (1 / M), 2^-100),   code = rne(y (1 / scale)).
 * Where a value is infinite or NaN so is the scale, and the values that it stands
 * for are NaN.
 */
int gdn_rms_norm_quant(const void *x, const void *residual, const void *weight, void *codes, float *scale,
                       void *sum, float eps, long long x_stride, long long residual_stride, int T, int C,
                       int block, int dtype, int weight_dtype, int format, void *stream);

/*
 * Gradients of gdn_rms_norm: of sum(out * grad_out) + sum(s * grad_sum).
 *
 *   sum        [T] rows, sum_stride apart: s as the forward wrote it (x without
 *              a residual)
 *   grad_out, grad_sum  [T] rows, their strides apart; grad_sum may be NULL
 *   grad_x     [T, C] written: the gradient of x, and of the residual
 *   grad_weight [C] written, of the weight's type
 *
 * Workspace: gdn_rms_norm_bwd_workspace_bytes (0 where T is 0), scratch on entry
 * and exit, no clearing needed.
 */
size_t gdn_rms_norm_bwd_workspace_bytes(int T, int C, int dtype);
int gdn_rms_norm_bwd(const void *sum, const void *weight, const void *grad_out, const void *grad_sum,
                     void *grad_x, void *grad_weight, float eps, long long sum_stride, long long grad_out_stride,
                     long long grad_sum_stride, int T, int C, int dtype, int weight_dtype, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * Depthwise causal convolution over packed sequences: with z the rows of a
 * sequence behind the W - 1 rows of its state,
 *
 *     p_t = bias + sum_j weight[:, j] z_{t + j},   out_t = p_t sigmoid(p_t), or p_t without silu
 *
 * so that tap W - 1 meets row t and tap 0 the row W - 1 before it.
 *
 *   x          [T] rows of C values, x_stride apart
 *   weight     [C, W], W from 2 to 4;  bias [C], may be NULL
 *   state      [R, W - 1, C] of the rows' type: the rows before each sequence,
 *              the latest last; may be NULL (zeros)
 *   out        [T, C] written
 *   state_final [R, W - 1, C] written: the last rows of z; may be NULL
 *
 * C is a multiple of 8 and at most 65536, T C below 2^34, R below 2^20, R C below
 * 2^31.
 */
int gdn_short_conv(const void *x, const void *weight, const void *bias, const int *cu_seqlens, const void *state,
                   void *out, void *state_final, long long x_stride, int T, int R, int C, int W, int dtype,
                   int weight_dtype, int silu, int zero_rest, void *stream);

/*
 * Its gradients: of sum(out * grad_out) + sum(state_final * grad_state_final).
 *
 *   grad_out   [T] rows, grad_out_stride apart;  grad_state_final [R, W - 1, C],
 *              may be NULL
 *   grad_x [T, C], grad_weight [C, W], grad_bias [C], grad_state [R, W - 1, C]
 *              written, each of the type of what it is the gradient of; the last
 *              two may be NULL
 *
 * Workspace: gdn_short_conv_bwd_workspace_bytes (0 where T is 0), scratch on
 * entry and exit, no clearing needed.
 */
size_t gdn_short_conv_bwd_workspace_bytes(int T, int C, int W);
int gdn_short_conv_bwd(const void *x, const void *weight, const void *bias, const void *grad_out,
                       const int *cu_seqlens, const void *state, const void *grad_state_final, void *grad_x,
                       void *grad_weight, void *grad_bias, void *grad_state, long long x_stride,
                       long long grad_out_stride, int T, int R, int C, int W, int dtype, int weight_dtype, int silu,
                       int zero_rest, void *workspace, size_t workspace_bytes, void *stream);

/*
 * One new row for each of R sequences: out [R, C] from x (R rows) and the state
 * [R, W - 1, C], which is moved on in place.
 */
int gdn_short_conv_step(const void *x, const void *weight, const void *bias, void *state, void *out,
                        long long x_stride, int R, int C, int W, int dtype, int weight_dtype, int silu,
                        void *stream);

/*
 * Selective state space scan.  For every head, with d = softplus(dt + dt_bias) and
 * a state S [N, P]:
 *
 *     S_t = exp(a d_t) S_{t-1} + d_t B_t x_t^T,   out_t = S_t^T C_t + D x_t
 *
 *   x          [T] rows of H * P bf16 values (dtype), x_stride apart
 *   dt         [T] rows of H values, bf16 or float32 (dt_dtype), dt_stride apart
 *              (any, from H on)
 *   a          [H], negative: the rate of decay;  D, dt_bias [H], may be NULL
 *              (zeros); all of param_dtype, bf16 or float32
 *   B, C       [T] rows of G * N bf16 values, B_stride and C_stride apart; head h
 *              reads group h / (H / G), H a multiple of G
 *   cu_seqlens [R + 1]
 *   S0         [R, H, N, P] float32: the states before, may be NULL (zeros)
 *   out        [T, H, P] bf16, written
 *   S_final    [R, H, N, P] float32, written; may be NULL
 *
 * P and N are 64 or 128 each.  States and every sum are float32; weights of rows and
 * the state are taken in two bf16 parts (2^-17) where they enter a product whose result
 * is out, and in three (2^-25) where it is a state.  Decays are float32 numbers:
 * where a token, or a piece of up to 64, keeps less than 2^-126 of the state, it keeps
 * nothing, and a weight within a piece is off by up to 9 E 2^-24 of itself, E the sum of
 * the piece's log2 decays, each counted up to 160.  Inputs are finite and a <= 0: others
 * give results that are undefined, typically non-finite, in their own sequence and
 * nowhere else.
 * Workspace: gdn_ssm_scan_workspace_bytes (0 for short T), scratch on entry and
 * exit, no clearing needed.  T is below 2^26, T * H below 2^31, R below 2^20, R * H
 * below 2^22, the strides of x, B and C below 2^24.
 */
size_t gdn_ssm_scan_workspace_bytes(int T, int H, int P, int G, int N);
int gdn_ssm_scan(const void *x, const void *dt, const void *a, const void *B, const void *C, const void *D,
                 const void *dt_bias, const int *cu_seqlens, const float *S0, void *out, float *S_final,
                 long long x_stride, long long dt_stride, long long B_stride, long long C_stride, int T, int R,
                 int H, int P, int G, int N, int dtype, int dt_dtype, int param_dtype, int zero_rest,
                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradients of gdn_ssm_scan: of sum(out * grad_out) + sum(S_final * grad_S_final).
 * The states are computed again inside the call.
 *
 *   grad_out, grad_x  [T] rows of H * P bf16 values, their strides apart
 *   grad_B, grad_C    [T] rows of G * N bf16 values, their strides apart, summed over
 *              the heads that share them
 *   grad_dt    [T, H] of dt_dtype
 *   grad_a, grad_D, grad_dt_bias [H] of param_dtype; the latter two may be NULL
 *   grad_S_final, grad_S0 [R, H, N, P] float32; may be NULL
 *
 * Sums are float32, in a fixed order, and rounded once.  Weights are taken in two bf16
 * parts; states and gradients of states, before and behind every 64 tokens, are rounded to
 * bf16 where they enter a product (grad_S0: as states of the forward are).  grad_dt,
 * grad_a and grad_dt_bias, sums of many terms that may cancel, are as exact as that
 * leaves their terms (2^-8 of each), also where they are float32.  Rows in no sequence:
 * as for the forward.  Workspace: gdn_ssm_scan_bwd_workspace_bytes, scratch on entry and
 * exit, no clearing needed; it holds two bf16 states for each head and 64 tokens, and
 * for each head and sequence.
 */
size_t gdn_ssm_scan_bwd_workspace_bytes(int T, int R, int H, int P, int G, int N);
int gdn_ssm_scan_bwd(const void *x, const void *dt, const void *a, const void *B, const void *C, const void *D,
                     const void *dt_bias, const void *grad_out, const int *cu_seqlens, const float *S0,
                     const float *grad_S_final, void *grad_x, void *grad_dt, void *grad_a, void *grad_B,
                     void *grad_C, void *grad_D, void *grad_dt_bias, float *grad_S0, long long x_stride,
                     long long dt_stride, long long B_stride, long long C_stride, long long grad_out_stride,
                     long long grad_x_stride, long long grad_B_stride, long long grad_C_stride, int T, int R, int H,
                     int P, int G, int N, int dtype, int dt_dtype, int param_dtype, int zero_rest, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * One token for each of R sequences, in place on their states S [R, H, N, P]
 * float32; x, dt, B, C have R rows.  The state and its sums are float32.
 */
int gdn_ssm_step(const void *x, const void *dt, const void *a, const void *B, const void *C, const void *D,
                 const void *dt_bias, float *S, void *out, long long x_stride, long long dt_stride,
                 long long B_stride, long long C_stride, int R, int H, int P, int G, int N, int dtype, int dt_dtype,
                 int param_dtype, void *stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char *gdn_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
