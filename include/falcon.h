/*
 * falcon.h -- C ABI of the MI355X (gfx950) implementation of Falcon
 * fast-weight attention: the chunk-parallel forward pass and the single-token
 * recurrent step, and the backward pass of the chunked form.
 *
 * Sources, cited by page title and section:
 *   [P1] zhouql-dev.github.io, "把状态更新写成一条学习规则：Falcon 家族重新对齐
 *        fast-weight 记忆": sections 本质 (prefix alignment), Falcon家族 (the
 *        family and the NLMS step), 三种等价形式 (recurrent / masked-parallel /
 *        chunked forms, positive-decay renormalisation), Figures 3 and 4.
 *   [P2] 59188saintaubert.com, "给记忆装一个“及时纠错”的开关：Falcon让循环模型
 *        学会边写边改": sections 一个被忽略的时间差, 把记忆更新变成一次梯度下降,
 *        六个变体, 正衰减钳制, 三种视角.
 *
 * What both entry points compute, per sequence (b, h) and step t = 1..T:
 *   x_t   = phi(k_{t-1})                  prefix-aligned key ([P1] 本质); x_1 = x_prev
 *   lam_t = max(exp(g_t), eps_gamma)      positive-decay clamp ([P2] 正衰减钳制)
 *   eta_t = beta_t / (eps_eta + |x_t|^2)  NLMS step ([P1] Falcon家族; [P2] 梯度下降)
 *   F1 : S_t = lam_t S_{t-1} + eta_t (v_t - S_{t-1} x_t) x_t^T
 *   F2 : as F1 with eta_t a vector over value channels (rows of S)
 *   F3 : S_t = lam_t S_{t-1} + (eta_t / Bw) sum_{j=t-Bw+1..t} (v_j - S_{t-1} x_j) x_j^T
 *   F1A/F2A/F3A: the same with the additive write (v_j instead of the residual)
 *   o_t   = S_t phi(q_t)                  read after write
 *   phi(a) = a / sqrt(|a|^2 + eps_phi)
 * The step definitions are [P1] Falcon家族 and [P2] 六个变体; the chunked
 * evaluation is [P1] 三种等价形式 form C / Figure 4-C (per-chunk Gram and WY
 * factors with a triangular solve) and [P2] 三种视角.
 *
 * Conventions shared by every entry point
 *   Layout   all arrays are dense, C order, no strides:
 *              q, k   [B, T, H, dk]   dtype (fp32 or bf16)
 *              v, o   [B, T, H, dv]   dtype
 *              beta   [B, T, H]  fp32, or [B, T, H, dv] for F2/F2A
 *              log_lambda (g) [B, T, H] fp32; any value <= 0 incl. -inf.
 *                     g > 0 (a decay above 1) is outside the contract and is
 *                     not checked: the chunked kernels factor every decay
 *                     exp(L_a - L_b), a >= b, as a number <= 1
 *              S      [B, H, dv, dk]  fp32, row i = value channel i
 *              x_prev [B, H, dk]      fp32
 *              win_x  [B, H, Bw-1, dk], win_v [B, H, Bw-1, dv] fp32, oldest first
 *            The single-step entry point drops the T axis.
 *   Memory   every pointer except `shape` and the state struct itself is a
 *            device pointer (hipMalloc / torch CUDA tensor).  The caller owns
 *            all memory; the library never allocates, frees, synchronises or
 *            keeps a pointer after the call returns.  Device pointers must be
 *            16-byte aligned.
 *   Streams  work is enqueued on `stream` (a hipStream_t, NULL = the null
 *            stream) and the call returns without waiting.  Buffers must stay
 *            alive until the stream reaches the work.
 *   Errors   the return value is a falcon_status_t.  Argument validation is
 *            done on the host before any HIP call, so an invalid call never
 *            touches the device.  A failed kernel launch returns
 *            FALCON_ERR_HIP; a fault inside a kernel shows up at the caller's
 *            next synchronisation.  NaN/Inf in the inputs are not checked;
 *            lam > 1 is outside the contract.
 *   Threads  no global mutable state: calls may be made from several threads.
 */
#ifndef FALCON_H
#define FALCON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FALCON_ABI_VERSION 4

typedef enum {
  FALCON_1 = 1,   /* scalar NLMS step, residual write            */
  FALCON_1A = 2,  /* scalar step, additive (inner-product) write  */
  FALCON_2 = 3,   /* per-value-channel step, residual write       */
  FALCON_2A = 4,  /* per-value-channel step, additive write       */
  FALCON_3 = 5,   /* window of Bw pairs, averaged residuals       */
  FALCON_3A = 6   /* window of Bw pairs, averaged additive write  */
} falcon_variant_t;

typedef enum { FALCON_F32 = 0, FALCON_BF16 = 1, FALCON_E4M3 = 2 } falcon_dtype_t;  /* of q, k, v, o: F32 or BF16;
 E4M3 (8 bits, largest number 448, no infinities): only where an entry point names it */

/* Which key the pair written at step t carries ([P1] 本质; [P2] 一个被忽略的时间差):
 * the prefix pair (phi(k_{t-1}), v_t), the method's alignment, or the same-step
 * pair (phi(k_t), v_t) the pages contrast it with.  Same-step calls do not read
 * the carried x_prev (they still write x_prev = phi(k_T)); window pairs are
 * (phi(k_j), v_j).  Same-step runs on the chunk-parallel kernels (with or without
 * a workspace where they are built) and on the decode step; other shapes return
 * FALCON_ERR_UNSUPPORTED. */
typedef enum { FALCON_ALIGN_PREFIX = 0, FALCON_ALIGN_SAME = 1 } falcon_align_t;

typedef enum {
  FALCON_OK = 0,
  FALCON_ERR_INVALID_ARG = 1,  /* null pointer, bad enum, non-positive size, ... */
  FALCON_ERR_UNSUPPORTED = 2,  /* valid but not built: head dim, chunk, window, dtype */
  FALCON_ERR_WORKSPACE = 3,    /* workspace smaller than falcon_chunk_fwd_workspace() */
  FALCON_ERR_HIP = 4           /* a HIP launch or runtime call failed */
} falcon_status_t;

typedef struct {
  int32_t variant;   /* falcon_variant_t */
  int32_t dtype;     /* falcon_dtype_t   */
  int32_t batch;     /* B >= 1 */
  int32_t seqlen;    /* T >= 1 (ignored by falcon_recurrent_step) */
  int32_t heads;     /* H >= 1 */
  int32_t dk;        /* key/query head dim: 32, 64 or 128 (fp32 inputs: 32 or 64).
                        The kernels are built for square states only: dk must
                        equal dv, else FALCON_ERR_UNSUPPORTED (every kernel tiles
                        both axes of S with the same 16-wide blocks and one
                        compile-time head dim).  fp32 at 128 is not built: its
                        tiles and staged rows do not fit a compute unit's LDS. */
  int32_t dv;        /* value head dim: equal to dk (see above) */
  int32_t chunk;     /* chunk length C: 16, 32 or 64; T need not be a multiple */
  int32_t window;    /* Bw for F3/F3A; must be 1 for the other variants.  The
                        decode step takes 1..8.  The chunked forms take 1, 2, 4
                        or 8 (Bw must divide 64: a system of 64 virtual rows
                        holds 64/Bw whole steps, and a step's Bw rows must not
                        straddle a 16-row MFMA block).  Larger windows (e.g. 16)
                        return FALCON_ERR_UNSUPPORTED: they are not built. */
  float eps_gamma;   /* decay floor, in (0, 1]; the pages' workloads use 1e-3 */
  float eps_phi;     /* feature-map epsilon, >= 0 (1e-6) */
  float eps_eta;     /* NLMS epsilon, > 0 (1e-6); 0 is FALCON_ERR_INVALID_ARG,
                        since a fresh sequence's first key is zero and its step
                        would divide by |x|^2 = 0 */
  int32_t align;     /* falcon_align_t */
} falcon_shape_t;

typedef struct {
  float *S;       /* [B, H, dv, dk]; required                                 */
  float *x_prev;  /* [B, H, dk] = phi(k) of the last consumed token; required  */
  float *win_x;   /* [B, H, Bw-1, dk], F3/F3A with Bw > 1 only, else ignored  */
  float *win_v;   /* [B, H, Bw-1, dv]                                         */
} falcon_state_t;

/* ABI version of the loaded library (FALCON_ABI_VERSION). */
int falcon_abi_version(void);

/* Static, human-readable name of a status code (never NULL). */
const char *falcon_status_string(int status);

/* Bytes of device workspace that enable the chunk-parallel path of
 * falcon_chunk_fwd for this shape; 0 when that path does not apply (the
 * forward then runs a fused kernel that needs no workspace).  The workspace
 * holds, per system of rows (a chunk of C steps; for F3/F3A with Bw > 1,
 * C/Bw steps of Bw pairs each), the key-side factors (Gram / score blocks,
 * diagonal-block inverses, per-row factors) that a prep kernel over all
 * systems writes and the state scan reads, plus a copy of each sequence's
 * incoming x_prev and window; its contents are scratch and need no
 * initialisation.  The path covers F1/F1A/F2/F2A (chunk 16, 32, 64) and
 * F3/F3A with Bw = 2, 4, 8 at chunk 64; d = 32, 64 (fp32, bf16), 128 (bf16).
 * F3A with Bw = 2, 4, 8 at d = 64, chunk 64 (fp32 and bf16 inputs) uses a workspace for its
 * banded-weight form (the window-averaged additive write of [P1] Falcon家族
 * as decayed score weights): each chunk's state increment, then the state
 * entering it, 16 KiB per chunk and sequence, plus the carried-state copy; the
 * returned size covers both.
 * Returns 0 for an invalid shape as well; validation is the forward call's job. */
size_t falcon_chunk_fwd_workspace(const falcon_shape_t *shape);

/* Chunked forward pass over T tokens ([P1] 三种等价形式 form C, Figure 4-C;
 * [P2] 三种视角).
 *   init         NULL: fresh sequences (S = 0, x_prev = 0, zero window).
 *                Otherwise S and x_prev (and the window for F3/F3A, Bw > 1)
 *                are read.  May alias final_state (in-place continuation).
 *   final_state  NULL: not written.  Otherwise receives S_T, x_prev =
 *                phi(k_T) and the last Bw-1 pairs.
 *   o            [B, T, H, dv] in dtype; must not alias any input.
 *   chunk_states NULL, or [B, H, ceil(T/C), dv, dk] fp32: S at the end of
 *                every chunk (the last one equals S_T).
 *   workspace    caller-owned device scratch, 16-byte aligned, or NULL.  NULL
 *                (or a shape whose workspace size is 0) selects the fused
 *                path; otherwise workspace_bytes must be at least
 *                falcon_chunk_fwd_workspace(shape) (else FALCON_ERR_WORKSPACE)
 *                and the chunk-parallel path runs.  Both paths compute the
 *                same function; calls that share one workspace on different
 *                streams race.
 * Results are deterministic: the same inputs give bit-identical outputs. */
int falcon_chunk_fwd(const falcon_shape_t *shape,
                     const void *q, const void *k, const void *v,
                     const float *beta, const float *log_lambda,
                     const falcon_state_t *init, falcon_state_t *final_state,
                     void *o, float *chunk_states,
                     void *workspace, size_t workspace_bytes, void *stream);

/* For callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.  The same computation as
 * falcon_chunk_fwd on its chunk-parallel path (prep kernel + state scan), with
 * the scratch that path needs taken from a fixed device array inside the library
 * (FALCON_STATIC_SCRATCH_BYTES per GPU, held from the first call on that GPU
 * until the process ends) instead of a caller's workspace.  The caller still
 * passes every input and output; the call allocates and frees nothing.
 *   Sizes  the shape must have that path (falcon_chunk_fwd_workspace(shape) > 0,
 *          else FALCON_ERR_UNSUPPORTED) and need at most
 *          FALCON_STATIC_SCRATCH_BYTES of it (else FALCON_ERR_WORKSPACE); e.g.
 *          the 130M-layer shape (B 8, H 12, T 2048, d 64, chunk 64) needs 41 MB.
 *   Races  every call on one GPU uses that GPU's one array: calls that overlap
 *          on a GPU (other streams, other threads) race and give wrong results.
 *          The scratch needs no initialisation; each call overwrites it.
 * Other arguments, aliasing and errors as falcon_chunk_fwd. */
#define FALCON_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
int falcon_chunk_fwd_static(const falcon_shape_t *shape,
                            const void *q, const void *k, const void *v,
                            const float *beta, const float *log_lambda,
                            const falcon_state_t *init, falcon_state_t *final_state,
                            void *o, float *chunk_states, void *stream);

/* Bytes of device workspace that enable the chunk-parallel path of
 * falcon_chunk_fwd_varlen for this packed shape (shape->batch = N sequences,
 * shape->seqlen = their total token count); 0 when that path does not apply
 * (as for falcon_chunk_fwd_workspace).  Per head it holds one image slot per
 * system the N sequences can have, at most total/S + N + 1 for systems of S
 * steps (sequence n's images start at slot cu_seqlens[n] / S + n, so the layout
 * follows from cu_seqlens on the device), plus each sequence's carried-state
 * copy; no initialisation needed. */
size_t falcon_chunk_fwd_varlen_workspace(const falcon_shape_t *shape);

/* Chunked forward pass over a packed batch of sequences of different lengths
 * (the same computation as falcon_chunk_fwd, one sequence per entry):
 *   shape->batch  = N, the number of sequences; shape->seqlen = the total
 *                   number of tokens, cu_seqlens[N].
 *   cu_seqlens    device int32 [N + 1]: sequence n holds tokens
 *                   cu_seqlens[n] .. cu_seqlens[n+1] - 1 (non-decreasing,
 *                   cu_seqlens[0] = 0; read on the device, not checked).
 *   q, k [total, H, dk], v, o [total, H, dv] in dtype; beta [total, H] (F2/F2A:
 *   [total, H, dv]) and log_lambda [total, H] fp32; the state arrays are per
 *   sequence ([N, H, ...]) as in falcon_chunk_fwd.
 *   workspace     NULL: the one-pass kernel, where it is built for the shape
 *                 (bf16 at d <= 64, fp32 at small chunks); a shape it does not
 *                 build returns FALCON_ERR_WORKSPACE when the chunk-parallel path
 *                 exists for it (pass a workspace) and FALCON_ERR_UNSUPPORTED
 *                 otherwise.  Non-NULL: at least
 *                 falcon_chunk_fwd_varlen_workspace(shape) bytes (else
 *                 FALCON_ERR_WORKSPACE), 16-byte aligned, and the chunk-parallel
 *                 path runs (this covers d = 128 in bf16).
 * Sequence n starts from init (its own S, x_prev and window) and ends in
 * final_state.  A sequence of length 0 is skipped: its final state is not
 * written.  No per-chunk states.  Same aliasing and stream rules as
 * falcon_chunk_fwd; calls sharing a workspace race. */
int falcon_chunk_fwd_varlen(const falcon_shape_t *shape, const int32_t *cu_seqlens,
                            const void *q, const void *k, const void *v,
                            const float *beta, const float *log_lambda,
                            const falcon_state_t *init, falcon_state_t *final_state,
                            void *o, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace falcon_chunk_fwd_segmented needs for this shape
 * and segment count; 0 when the segmented form is not built for them: nseg
 * must divide T, segments must hold at least Bw steps, the shape must have the
 * two-kernel chunk-parallel path (see falcon_chunk_fwd_workspace), and F2 is
 * excluded (its step differs per row of S, so a segment's map is not one
 * matrix).  The workspace holds that path's scratch for B*nseg sequences of
 * T/nseg steps plus six per-segment state arrays; it needs no initialisation. */
size_t falcon_chunk_fwd_segmented_workspace(const falcon_shape_t *shape, int32_t nseg);

/* The chunked forward pass with every sequence cut into nseg segments that run
 * in parallel: the same function as falcon_chunk_fwd (up to rounding), for
 * batches too small to fill the GPU.  A segment maps its incoming state S_0 to
 * S_0 M + N ([P1] 三种等价形式: the chunk maps are affine and compose; [P2]
 * 三种视角), so the call builds the key-side images of all B*nseg segments
 * once, then runs (1) the scan from S_0 = 0 (giving N) and (2) from S_0 = I
 * (giving M + N), both keeping end states only, (3) the composition
 * S_start[p] = S_start[p-1] M_{p-1} + N_{p-1} along each sequence, and (4) the
 * scan from S_start, which writes o and the final state.  The carried key
 * and window entering a segment come from the inputs.  The arrays are the same
 * as falcon_chunk_fwd's ([B, T, H, d] is read as [B*nseg, T/nseg, H, d]); no
 * per-chunk states.  init may alias final_state.  Errors: nseg < 1 or not
 * dividing T -> FALCON_ERR_INVALID_ARG; NULL or misaligned workspace ->
 * FALCON_ERR_INVALID_ARG; a shape or nseg the form is not built for ->
 * FALCON_ERR_UNSUPPORTED; a short workspace -> FALCON_ERR_WORKSPACE. */
int falcon_chunk_fwd_segmented(const falcon_shape_t *shape, int32_t nseg,
                               const void *q, const void *k, const void *v,
                               const float *beta, const float *log_lambda,
                               const falcon_state_t *init, falcon_state_t *final_state,
                               void *o, void *workspace, size_t workspace_bytes, void *stream);

/* One token of the recurrent form ([P1] 三种等价形式 form A; [P2] 三种视角):
 * reads q, k [B, H, dk], v [B, H, dv], beta [B, H] (F2/F2A: [B, H, dv]) and
 * log_lambda [B, H]; updates `state` in place (S, x_prev and, for F3/F3A with
 * Bw > 1, the window) and writes o [B, H, dv] in dtype.  shape->seqlen and
 * shape->chunk are ignored. */
int falcon_recurrent_step(const falcon_shape_t *shape,
                          const void *q, const void *k, const void *v,
                          const float *beta, const float *log_lambda,
                          falcon_state_t *state, void *o, void *stream);

/* Bytes of device workspace falcon_chunk_bwd needs for this shape; 0 when the
 * backward pass is not built for it (or the shape is invalid).  Built for every
 * shape the chunked forward pass builds with d_k = d_v: chunk 16, 32 or 64 (the
 * chunk of the forward call that wrote the per-chunk states), fp32 or bf16
 * inputs, either pairing, by one of two paths:
 *  - chunk-parallel (F1, F1A, F2, F2A, and F3 / F3A with one pair; d = 64): the
 *    kernels work in 64-step chunks and read the states at 64-step boundaries.
 *    The workspace holds, per chunk, the chunk's transition of the reverse
 *    recurrence (d x d), the state gradient the chunk's outputs inject and the
 *    state gradient at the chunk's end (3 x 16 KiB + 4 bytes); for F2, whose
 *    solves are per value channel, the keys, the decayed Gram matrix, the
 *    injected gradient, the end gradient and the per-channel steps (5 x 16 KiB)
 *    plus 516 bytes of per-row factors.
 *  - recurrent form (F3 / F3A windows of 2, 4 or 8 pairs; d = 32, or 128 with
 *    bf16 inputs; every variant): the states at every forward chunk are the
 *    checkpoints.  The workspace holds, per 16 value rows of every sequence,
 *    the row sums of each token (2 d + 2 floats) and of each carried window
 *    pair (d floats): d/16 x (B T H (2 d + 2) + B H (Bw - 1) d) x 4 bytes.
 * It needs no initialisation. */
size_t falcon_chunk_bwd_workspace(const falcon_shape_t *shape);

/* Backward pass of the chunked form ([P1] 三种等价形式 form C / Figure 4-C: the
 * form a training framework runs): the gradients of the scalar
 *     <d_o, o> + <d_final_S, S_T>
 * for the forward pass falcon_chunk_fwd(shape, q, k, v, beta, log_lambda, init)
 * with respect to q, k, v, beta, log_lambda and the initial state.  The
 * outgoing x_prev takes no gradient.  The decay clamp passes no gradient where
 * exp(g) <= eps_gamma (there the decay does not depend on g).
 * Windows ([P1] Falcon家族, [P2] 六个变体): every pair of a step's window takes
 * its share of the gradient, the carried window's pairs included.
 *   init         as given to the forward pass (NULL = fresh sequences); S,
 *                x_prev and, for F3/F3A with Bw > 1, the window are read.
 *   chunk_states [B, H, ceil(T/C), d, d] fp32: the per-chunk states the
 *                forward pass wrote for these inputs at shape->chunk = C.
 *   d_o          [B, T, H, d] in dtype.
 *   d_final_S    [B, H, d, d] fp32, or NULL for a zero gradient on S_T.
 *   dq, dk, dv   [B, T, H, d] fp32, written whole (under the prefix pairing
 *                dk of the last token is 0).
 *   dbeta, dg    [B, T, H] fp32 (F2/F2A: dbeta [B, T, H, dv], like their beta).
 *   d_init       NULL, or S [B, H, d, d] and x_prev [B, H, d] fp32 (and, for
 *                F3/F3A with Bw > 1, win_x and win_v [B, H, Bw-1, d]) that
 *                receive the gradients w.r.t. the initial state (x_prev: 0
 *                under the same-step pairing, which does not read it; the
 *                window's keys are features, so win_x takes their gradient
 *                as they are).
 *   workspace    at least falcon_chunk_bwd_workspace(shape) bytes, else
 *                FALCON_ERR_WORKSPACE; calls sharing a workspace race.
 * Outputs must not alias inputs.  Other shapes return FALCON_ERR_UNSUPPORTED.
 * Results are deterministic. */
int falcon_chunk_bwd(const falcon_shape_t *shape,
                     const void *q, const void *k, const void *v,
                     const float *beta, const float *log_lambda,
                     const falcon_state_t *init, const float *chunk_states,
                     const void *d_o, const float *d_final_S,
                     float *dq, float *dk, float *dv, float *dbeta, float *dg,
                     falcon_state_t *d_init,
                     void *workspace, size_t workspace_bytes, void *stream);

/* ======================================================================== */
/* Operators around the mixer                                               */
/* ======================================================================== */
/* What stands next to Falcon in a stack of recurrent and attention layers: a
 * gated linear recurrence with a vector state, the head norm and rotary
 * positions of queries and keys, and causal softmax attention.  Memory, stream,
 * error and thread conventions are those of the entry points above; packed
 * sequences are given by the same device offsets (int32, non-decreasing, first
 * 0, last at most the given token count; read on the device, not checked there).
 * Tokens behind the last sequence are not written.  Gradients with
 * respect to activations have the activations' dtype; those with respect to
 * parameters and states are fp32.  Sums, states, softmax statistics and norms
 * are fp32, and results are deterministic.  NaN and infinities stay in their own
 * sequence.  A workspace needs no initialisation and serves one call at a time.
 * Sizes past the limits given here, or past a launch (2^32 threads), are
 * FALCON_ERR_UNSUPPORTED. */

/* ---- Gated linear recurrence ---------------------------------------------
 * Per sequence and channel, with lam_t = exp(log_lambda_t):
 *   h_t = lam_t h_{t-1} + u_t,  u_t = x_t            (FALCON_SCAN_ADD)
 *                               u_t = (1 - lam_t) x_t (FALCON_SCAN_MIX)
 * There is no decay floor: log_lambda = -inf is an exact reset (lam = 0).
 * log_lambda > 0 grows the state; the product of the lam of FALCON_SCAN_CHUNK
 * steps then has to stay in fp32's range.  (Steps are composed before they are
 * applied: behind an infinite state a later one may be NaN.) */
typedef enum { FALCON_SCAN_ADD = 0, FALCON_SCAN_MIX = 1 } falcon_scan_input_t;

typedef struct {
  int32_t dtype;   /* falcon_dtype_t of x, log_lambda, h and their gradients */
  int32_t batch;   /* sequences, 1 .. 2^30 */
  int32_t seqlen;  /* steps of every sequence, >= 1; packed: all tokens (>= 1) */
  int32_t width;   /* channels, a multiple of 8, at most 2^20 */
  int32_t input;   /* falcon_scan_input_t */
} falcon_scan_shape_t;

#define FALCON_SCAN_CHUNK 256   /* steps between the states the forward keeps */

/* Bytes of workspace of falcon_scan_fwd and falcon_scan_bwd (the same for both);
 * `packed` is nonzero for calls with cu_seqlens.  0 when the steps fit one chunk
 * (then workspace may be NULL), and for invalid shapes. */
size_t falcon_scan_workspace(const falcon_scan_shape_t *shape, int packed);

/* The recurrence over T steps.
 *   cu_seqlens   NULL: x, log_lambda, h are [B, T, D].  Otherwise [B + 1] offsets
 *                and the arrays are [T, D], T = all tokens.
 *   init         [B, D] fp32, or NULL for zeros.
 *   final_state  [B, D] fp32, or NULL; may alias init.  An empty sequence's is
 *                its initial state.
 *   chunk_states [B, ceil(T / FALCON_SCAN_CHUNK), D] fp32 (packed: of the one
 *                packed time axis, [1, ...]), or NULL: h after every chunk, for
 *                the backward pass.
 *   workspace    at least falcon_scan_workspace bytes, else FALCON_ERR_WORKSPACE.
 * Outputs must not overlap inputs otherwise. */
int falcon_scan_fwd(const falcon_scan_shape_t *shape, const int32_t *cu_seqlens, const void *x, const void *log_lambda,
                    const float *init, float *final_state, void *h, float *chunk_states,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Gradients of <d_h, h> + <d_final, final_state> with respect to x, log_lambda
 * and init, from the chunk_states the forward wrote for the same arguments.
 * d_final [B, D] fp32 or NULL (zeros); dx, dg like x; d_init [B, D] fp32 or NULL.
 * Outputs must not alias inputs. */
int falcon_scan_bwd(const falcon_scan_shape_t *shape, const int32_t *cu_seqlens, const void *x, const void *log_lambda,
                    const float *init, const float *chunk_states, const void *d_h, const float *d_final,
                    void *dx, void *dg, float *d_init, void *workspace, size_t workspace_bytes, void *stream);

/* One step: x, log_lambda, h [B, D]; state [B, D] fp32 is updated in place.
 * shape->seqlen is ignored. */
int falcon_scan_step(const falcon_scan_shape_t *shape, const void *x, const void *log_lambda, float *state, void *h,
                     void *stream);

/* ---- Query / key norm with rotary positions ------------------------------
 * For every head x (d entries) of q and k of every token:
 *   z = x w / sqrt(mean(x^2) + eps)   (norm != 0; z = x otherwise)
 * then the first `rot` entries turn in pairs (a, b) by the angle
 * position * inv_freq[j], times rot_scale:
 *   y_a = z_a cos - z_b sin,  y_b = z_b cos + z_a sin
 * with a = j, b = j + rot / 2 (FALCON_ROPE_HALF) or a = 2 j, b = 2 j + 1
 * (FALCON_ROPE_INTERLEAVED); the other entries are z.  Longer contexts scale
 * inv_freq and rot_scale; the angle is formed in 64 bits, the mean of squares in
 * 32 (entries over 2^63 overflow it: z = 0; with eps = 0, z of a row of zeros, or
 * of entries under 2^-75, is not finite). */
typedef enum { FALCON_ROPE_HALF = 0, FALCON_ROPE_INTERLEAVED = 1 } falcon_rope_layout_t;

typedef struct {
  int32_t dtype;     /* falcon_dtype_t of q, k and the outputs */
  int32_t tokens;    /* 1 .. 2^31 - 1 - 2^20 */
  int32_t heads_q;   /* >= 1 */
  int32_t heads_k;   /* >= 1; both together at most 2^20 */
  int32_t d;         /* 32, 64 or 128 */
  int32_t rot;       /* rotated entries: a multiple of 16, 0 .. d */
  int32_t layout;    /* falcon_rope_layout_t */
  int32_t norm;      /* 0 or 1 */
  float eps;         /* finite, >= 0 */
  float rot_scale;   /* finite */
  int32_t grad_dtype; /* falcon_dtype_t of the backward's dq_out, dk_out: dtype, or FALCON_F32 */
} falcon_qk_shape_t;

/* [tokens, heads, d] with dense heads: the elements from one token to the next,
 * a multiple of 16 bytes and at least heads * d.  So q and k may be views of
 * one projection's output. */
typedef struct { const void *data; int64_t token_stride; } falcon_heads_t;
typedef struct { void *data; int64_t token_stride; } falcon_heads_out_t;

/* q_out, k_out: may be q, k themselves (same pointer and stride), else must not
 * overlap the inputs.  q_weight, k_weight: [d] fp32, or NULL for ones (ignored
 * without norm).  positions: [tokens] int32.  inv_freq: [rot / 2] fp64, radians
 * per position (NULL allowed when rot is 0). */
int falcon_qk_norm_rope(const falcon_qk_shape_t *shape, falcon_heads_t q, falcon_heads_t k,
                        const float *q_weight, const float *k_weight, const int32_t *positions,
                        const double *inv_freq, falcon_heads_out_t q_out, falcon_heads_out_t k_out, void *stream);

/* Bytes of workspace of the backward pass (the workgroups' weight-gradient
 * sums); 0 without norm and for invalid shapes. */
size_t falcon_qk_norm_rope_bwd_workspace(const falcon_qk_shape_t *shape);

/* Gradients of <dq_out, q_out> + <dk_out, k_out>: dq, dk in dtype (without norm
 * q and k are not read and may be {NULL, 0}); dq_weight, dk_weight [d] fp32 or
 * NULL.  dq, dk may be dq_out, dk_out themselves when the dtypes agree. */
int falcon_qk_norm_rope_bwd(const falcon_qk_shape_t *shape, falcon_heads_t q, falcon_heads_t k,
                            const float *q_weight, const float *k_weight, const int32_t *positions,
                            const double *inv_freq, falcon_heads_t dq_out, falcon_heads_t dk_out,
                            falcon_heads_out_t dq, falcon_heads_out_t dk, float *dq_weight, float *dk_weight,
                            void *workspace, size_t workspace_bytes, void *stream);

/* ---- Causal softmax attention --------------------------------------------
 * The queries of a sequence are the last Lq of its Lk tokens: query i sees keys
 * j <= i + Lk - Lq.  Query head h reads key head h / (heads_q / heads_k).
 *   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  lse_i = ln sum_j e^{scale q_i . k_j}
 * A query that sees no key (Lq > Lk), or whose scores are all -inf, has o = 0,
 * lse = -inf and no gradients.
 * Infinite or NaN keys and values do not reach o and lse of the queries that do
 * not see them; any gradient of a sequence that holds some may be NaN. */
typedef struct {
  int32_t dtype;     /* falcon_dtype_t of every array but lse */
  int32_t batch;     /* sequences, 1 .. 2^30 */
  int32_t seqlen_q;  /* query tokens of every sequence, >= 1; packed: all of them */
  int32_t seqlen_k;  /* key tokens of every sequence, >= 1; packed: all of them */
  int32_t heads_q;   /* a multiple of heads_k, at most 2^20 */
  int32_t heads_k;   /* >= 1; query tokens * heads_q / heads_k at most 2^31 - 4097 */
  int32_t d;         /* 32, 64 or 128 */
  float scale;       /* finite, > 0 */
} falcon_attn_shape_t;

/* Bytes of workspace of the forward: partial results, where the keys are split
 * over workgroups because there are few queries; 0 where they are not (then
 * workspace may be NULL).  `packed`: nonzero for calls with offsets. */
size_t falcon_attn_fwd_workspace(const falcon_attn_shape_t *shape, int packed);

/* q [tokens, heads_q, d], k, v [tokens, heads_k, d] (token strides as above, at
 * most 2^25 bytes), o dense [tokens, heads_q, d], lse [tokens, heads_q] fp32 or
 * NULL; they must not overlap the inputs.
 *   cu_q, cu_k  both NULL (batch * seqlen tokens) or both [batch + 1] offsets.
 * Either way the tokens of a sequence follow those of the one before: there is no
 * form for keys kept with room to grow between the sequences. */
int falcon_attn_fwd(const falcon_attn_shape_t *shape, const int32_t *cu_q, const int32_t *cu_k,
                    falcon_heads_t q, falcon_heads_t k, falcon_heads_t v, void *o, float *lse,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace of the backward: two fp32 numbers per query and head, and, where
 * few key tiles meet many queries, partial sums of dk and dv. */
size_t falcon_attn_bwd_workspace(const falcon_attn_shape_t *shape, int packed);

/* Gradients of <d_o, o> with respect to q, k, v, from the forward's o and lse (o
 * dense; the stride of d_o at most 2^25 bytes).  Outputs must not alias inputs. */
int falcon_attn_bwd(const falcon_attn_shape_t *shape, const int32_t *cu_q, const int32_t *cu_k,
                    falcon_heads_t q, falcon_heads_t k, falcon_heads_t v, const void *o, const float *lse,
                    falcon_heads_t d_o, falcon_heads_out_t dq, falcon_heads_out_t dk, falcon_heads_out_t dv,
                    void *workspace, size_t workspace_bytes, void *stream);

/* ======================================================================== */
/* Operators of a state-space block                                         */
/* ======================================================================== */
/* What a block of a recurrent model is made of besides its mixer: the norm of the
 * residual stream, the projections, the short causal convolution, and the
 * selective state-space scan.  Conventions as for the operators around the mixer
 * (packed sequences, gradients' types, determinism, workspaces, refusals).
 * Arrays are dense unless given as falcon_heads_t, with one head of the array's
 * width: then tokens may be further apart, as in a view of a wider projection.
 * Outputs must not overlap inputs, but where an entry point allows it; the same pointer is
 * FALCON_ERR_INVALID_ARG where that would be a race. */

typedef enum { FALCON_ACT_NONE = 0, FALCON_ACT_SILU = 1, FALCON_ACT_GELU = 2 } falcon_activation_t;
/* silu(p) = p / (1 + e^-p);  gelu(p) = p (1 + erf(p / sqrt 2)) / 2 */

/* ---- Norm of the residual stream ------------------------------------------
 * Per token, of `width` entries:
 *   s = x + residual, rounded to dtype          (residual NULL: s = x)
 *   y = s w / sqrt(mean(s^2) + eps)             (norm = 0: y = s w)
 * The norm is of the rounded stream, which the backward pass differentiates.
 * out = FALCON_E4M3: y in 8 bits, y = q scale with one fp32 scale a token,
 *   scale = max(max |y|, 1e-30) / 448, q = y / scale rounded to nearest even
 * (the fp32 quotient, of the unrounded y; with norm = 0 and no weight this quantises
 * x's rows).  A row with a NaN has a NaN scale; one with an infinity (norm = 0) an infinite one.
 * The mean of squares is formed in fp32: as in the query / key norm, entries over
 * 2^63 overflow it, and with eps = 0 a row of zeros is not finite. */
typedef struct {
  int32_t dtype;   /* falcon_dtype_t of x, residual and the stream: F32 or BF16 */
  int32_t tokens;  /* 1 .. 2^31 - 1 - 2^20 */
  int32_t width;   /* a multiple of 8; at most 32768 (BF16) or 16384 (F32) */
  int32_t norm;    /* 0 or 1 */
  int32_t out;     /* falcon_dtype_t of y: dtype or E4M3 */
  float eps;       /* finite, >= 0 */
} falcon_norm_shape_t;

/* weight [width] fp32 or NULL (ones).  stream: receives s; may be NULL, and may be
 * x or residual itself; not written without residual.  y may be x or residual
 * itself if it has their type and is not the stream.  scale: [tokens] fp32, for E4M3. */
int falcon_rms_norm(const falcon_norm_shape_t *shape, const void *x, const void *residual, const float *weight,
                    void *stream_out, void *y, float *scale, void *stream);

/* Bytes of workspace of the backward pass (the workgroups' sums for the weight's
 * gradient); 0 for invalid shapes. */
size_t falcon_rms_norm_bwd_workspace(const falcon_norm_shape_t *shape);

/* The gradient dx, which is x's and the residual's alike, of <d_y, y> + <d_stream, s>,
 * from the stream s (x itself where there was no residual).  shape->norm must be 1, and
 * out is ignored: d_y, d_stream (NULL: zeros) and dx have dtype.  dweight [width] fp32 or
 * NULL (then workspace may be NULL).  dx may be d_y or d_stream itself. */
int falcon_rms_norm_bwd(const falcon_norm_shape_t *shape, const void *s, const float *weight, const void *d_y,
                        const void *d_stream, void *dx, float *dweight, void *workspace, size_t workspace_bytes,
                        void *stream);

/* ---- Short causal convolution ----------------------------------------------
 * Per sequence and channel, with one filter of `taps` weights a channel:
 *   y_t = act(bias + sum_j w_j x_{t - taps + 1 + j}),  j = 0 .. taps - 1
 * The inputs before a sequence's first token are its initial state (oldest first),
 * its last taps - 1 inputs (those of the initial state included) its final one. */
typedef struct {
  int32_t dtype;       /* falcon_dtype_t of x, y, the states and their gradients: F32 or BF16 */
  int32_t batch;       /* sequences, >= 1 */
  int32_t seqlen;      /* tokens of every sequence, >= 1; packed: all tokens.  At most 2^31 - 1 - 4096 in all */
  int32_t width;       /* channels, a multiple of 8, at most 2^20 */
  int32_t taps;        /* 2, 3 or 4 */
  int32_t activation;  /* FALCON_ACT_NONE or FALCON_ACT_SILU */
} falcon_conv_shape_t;

/*   cu_seqlens   NULL: x, y are [B, T, D].  Otherwise [B + 1] offsets, and they are [T, D].
 *   weight       [D, taps] fp32;  bias [D] fp32 or NULL.
 *   init         [B, taps - 1, D] in dtype, or NULL for zeros.
 *   final_state  the same, or NULL.  An empty sequence's is its initial state.
 * Outputs must not overlap inputs. */
int falcon_conv_fwd(const falcon_conv_shape_t *shape, const int32_t *cu_seqlens, falcon_heads_t x, const float *weight,
                    const float *bias, const void *init, void *final_state, void *y, void *stream);

/* Bytes of workspace of the backward pass; `packed` is nonzero for calls with
 * cu_seqlens.  0 for invalid shapes. */
size_t falcon_conv_bwd_workspace(const falcon_conv_shape_t *shape, int packed);

/* Gradients of <d_y, y> + <d_final, final_state>: dx, d_init (or NULL) in dtype, the sums
 * rounded once; dweight [D, taps], dbias [D] fp32, or NULL (both NULL: workspace may be
 * NULL).  d_final as the final state, or NULL.  Outputs must not alias inputs. */
int falcon_conv_bwd(const falcon_conv_shape_t *shape, const int32_t *cu_seqlens, falcon_heads_t x, const float *weight,
                    const float *bias, const void *init, const void *d_y, const void *d_final, falcon_heads_out_t dx,
                    float *dweight, float *dbias, void *d_init, void *workspace, size_t workspace_bytes, void *stream);

/* One token of every sequence: x [B, D] (batch the tokens), y [B, D]; state
 * [B, taps - 1, D] in dtype, state_out the same (may be state itself).  shape->seqlen is
 * ignored. */
int falcon_conv_step(const falcon_conv_shape_t *shape, falcon_heads_t x, const float *weight, const float *bias,
                     const void *state, void *state_out, void *y, void *stream);

/* ---- Selective state-space scan --------------------------------------------
 * Per sequence, channel d and state n, with delta_t = softplus(dt_t + dt_bias)
 * (softplus = 0: delta_t = dt_t + dt_bias):
 *   h_t = exp(delta_t A[d][n]) h_{t-1} + delta_t x_t B_t[n]
 *   y_t = (sum_n C_t[n] h_t[n] + D[d] x_t) silu(z_t)         (z NULL: no gate)
 * B_t and C_t are shared by the channels.  Token strides are at most 2^24 bytes.  A is
 * finite; where delta_t A > 0 the state grows, and its growth over 64 steps (where
 * sequences are cut into segments, over a segment) has to stay in fp32's range.  States,
 * sums and delta are fp32.  An infinity in B or C stays in its state n; gradients of that
 * state may be NaN where the formula's are infinite. */
typedef struct {
  int32_t dtype;     /* falcon_dtype_t of x, dt, B, C, z, y and their gradients: F32 or BF16 */
  int32_t batch;     /* sequences, >= 1 */
  int32_t seqlen;    /* tokens of every sequence, >= 1; packed: all tokens.  At most 2^31 - 1 - 4096 in all */
  int32_t width;     /* channels, a multiple of 8, at most 2^20 */
  int32_t state;     /* N: 16, 32 or 64 */
  int32_t softplus;  /* 0 or 1 */
} falcon_ssm_shape_t;

#define FALCON_SSM_CHUNK(state) (1024 / (state))   /* steps between the states the forward keeps */

/* Bytes of workspace of the forward: the maps of segments, where few long sequences are
 * cut to run in parallel; 0 where none may be (then workspace may be NULL), and for invalid
 * shapes.  `packed` is nonzero for calls with cu_seqlens. */
size_t falcon_ssm_fwd_workspace(const falcon_ssm_shape_t *shape, int packed);

/* Chunks of K = FALCON_SSM_CHUNK(N) steps that the forward keeps a state of: batch ceil(T / K),
 * or packed floor(T / K) + batch (chunk c of sequence n, which begins at token s, is number
 * floor(s / K) + n + c; some stay unused).  0 for invalid shapes. */
int falcon_ssm_chunks(const falcon_ssm_shape_t *shape, int packed);

/*   cu_seqlens   NULL: x, dt, z, y are [B, T, D] and Bm, Cm [B, T, N].  Otherwise [B + 1] offsets,
 *                and they are [T, ...].
 *   A            [D, N] fp32;  D, dt_bias  [D] fp32, or NULL (zeros).
 *   z            {NULL, 0}: no gate.
 *   init         [B, D, N] fp32, or NULL for zeros.
 *   final_state  [B, D, N] fp32, or NULL.  An empty sequence's is its initial state.
 *   chunk_states [falcon_ssm_chunks, D, N] fp32, or NULL: h before every chunk of a sequence,
 *                for the backward pass.
 * Outputs must not overlap inputs (final_state may not be init). */
int falcon_ssm_fwd(const falcon_ssm_shape_t *shape, const int32_t *cu_seqlens, falcon_heads_t x, falcon_heads_t dt,
                   const float *A, falcon_heads_t Bm, falcon_heads_t Cm, const float *D, falcon_heads_t z,
                   const float *dt_bias, const float *init, float *final_state, void *y, float *chunk_states,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace of the backward: partial sums of dB and dC for every 32 channels and of the
 * parameters' gradients, and the maps of segments.  0 for invalid shapes. */
size_t falcon_ssm_bwd_workspace(const falcon_ssm_shape_t *shape, int packed);

/* Gradients of <d_y, y> + <d_final, final_state>, from the chunk_states the forward wrote for
 * the same arguments (the initial state among them).  d_y [.., D] dense in dtype; d_final
 * [B, D, N] fp32 or NULL (zeros).  dx, ddt, dz (ignored without z), dB, dC in dtype; dA [D, N],
 * dD, ddt_bias [D] fp32 (dD, ddt_bias may be NULL); d_init [B, D, N] fp32 or NULL.  Outputs must
 * not alias inputs. */
int falcon_ssm_bwd(const falcon_ssm_shape_t *shape, const int32_t *cu_seqlens, falcon_heads_t x, falcon_heads_t dt,
                   const float *A, falcon_heads_t Bm, falcon_heads_t Cm, const float *D, falcon_heads_t z,
                   const float *dt_bias, const float *chunk_states, const void *d_y, const float *d_final,
                   falcon_heads_out_t dx, falcon_heads_out_t ddt, float *dA, falcon_heads_out_t dB,
                   falcon_heads_out_t dC, float *dD, falcon_heads_out_t dz, float *ddt_bias, float *d_init,
                   void *workspace, size_t workspace_bytes, void *stream);

/* One step of every sequence: x, dt, z, y [B, D], Bm, Cm [B, N]; state, state_out [B, D, N] fp32
 * (state_out may be state itself).  shape->seqlen is ignored. */
int falcon_ssm_step(const falcon_ssm_shape_t *shape, falcon_heads_t x, falcon_heads_t dt, const float *A,
                    falcon_heads_t Bm, falcon_heads_t Cm, const float *D, falcon_heads_t z, const float *dt_bias,
                    const float *state, float *state_out, void *y, void *stream);

/* ---- Projections -----------------------------------------------------------
 *   p = x W^T (x_scale, weight_scale) + bias,  y = act(p) + residual
 * with x [tokens, in] and W [out, in] in dtype.  E4M3: entry (t, o) of the product is scaled by
 * x_scale[t] weight_scale[o], as falcon_rms_norm and its form without norm leave rows.  Sums
 * are fp32 and y is rounded once; but E4M3 with y in BF16 and without pre is summed by the matrix
 * unit's 8-bit products, which drop what lies 13 bits behind the largest of a group of them. */
typedef struct {
  int32_t dtype;       /* falcon_dtype_t of x and W: F32, BF16 or E4M3 */
  int32_t tokens;      /* 1 .. 2^31 - 4097 */
  int32_t in;          /* a multiple of 16, at most 2^20 */
  int32_t out;         /* a multiple of 8, at most 2^20 */
  int32_t activation;  /* falcon_activation_t */
  int32_t out_dtype;   /* falcon_dtype_t of y and residual: dtype; for E4M3 F32 or BF16 */
} falcon_linear_shape_t;

/* Bytes of workspace of the forward: the sums of workgroups that split `in`, where there are few
 * tokens; 0 where none do (then workspace may be NULL), and for invalid shapes. */
size_t falcon_linear_fwd_workspace(const falcon_linear_shape_t *shape);

/*   x             token stride at most 2^23 bytes;  weight dense.
 *   x_scale, weight_scale  [tokens], [out] fp32 for E4M3, else NULL.
 *   bias          [out] fp32, or NULL;  residual [tokens, out] in out_dtype, or NULL.
 *   y             [tokens, out]; may be the residual itself.
 *   pre           [tokens, out] fp32: receives p, for the backward pass of an activation; or
 *                 NULL.  Outputs must not overlap inputs otherwise. */
int falcon_linear_fwd(const falcon_linear_shape_t *shape, falcon_heads_t x, const void *weight, const float *x_scale,
                      const float *weight_scale, const float *bias, const void *residual, void *y, float *pre,
                      void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace of the backward: the gradient of p, and partial sums. */
size_t falcon_linear_bwd_workspace(const falcon_linear_shape_t *shape);

/* Gradients of <d_y, y> (the residual's is d_y itself), for F32 and BF16: with
 * d = d_y act'(pre), dx = d W and dweight = d^T x in dtype, dbias = the sum of d over tokens, fp32;
 * any may be NULL (dx: {NULL, 0}).  For BF16 with an activation the products take d rounded to
 * BF16 (dbias the unrounded d).  pre as the forward wrote it (without an activation it is
 * ignored).  Strides of x and d_y at most 2^23 bytes.  Outputs must not alias inputs. */
int falcon_linear_bwd(const falcon_linear_shape_t *shape, falcon_heads_t x, const void *weight, const float *pre,
                      falcon_heads_t d_y, falcon_heads_out_t dx, void *dweight, float *dbias,
                      void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FALCON_H */
