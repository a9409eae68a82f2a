/*
 * naju.h -- C ABI of libnaju.so, the MI355X (gfx950) implementation of the
 * Naju native-discrete selective state scan and of the mixer-block pieces
 * fused around it.
 *
 * The operation (Naju reproduction README of arXiv 2607.21000, section
 * "Core equations"): for each batch row and channel c, with state row
 * x[c, 0..N-1] (N = d_state),
 *
 *     x_n[c,s] = f_n[c] x_{n-1}[c,s] + i_n[c] h_n[c] B_n[s],
 *     f_n = sigma(a_n),  i_n = sigma(b_n)            (retain / write gates)
 *     ys_n[c]  = (1/sqrt(N)) sum_s x_n[c,s] C_n[s] + D[c] h_n[c]
 *
 * using the post-update state in the readout.  The gates and h are given per
 * (token, channel); B_n and C_n are one N-vector per (batch, token), shared by
 * every channel (the page's "token-dependent B/C directions").
 *
 * The block entry points add the front end and the output modulation of the
 * same page's block flowchart: h = SiLU(causal depthwise conv1d(u)) with
 * d_conv taps and no bias, and y = ys * SiLU(z).  The convolution is a
 * cross-correlation whose last tap multiplies the current token:
 *     pre_n[c] = sum_{k<K} conv_w[c,k] u_{n-K+1+k}[c]
 * with u_m for m < 0 taken from conv_state (zeros if conv_state is NULL).
 *
 * The backward entry points are the reverse mode of these definitions.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  Layouts   row-major, contiguous, no strides:
 *              per (token, channel) tensors: [batch][seqlen][d_inner]
 *              per token tensors B, C, dB, dC: [batch][seqlen][d_state]
 *              states x0, x_final, dx_final, dx0: [batch][d_inner][d_state] fp32
 *              D, dD: [d_inner] fp32;  conv_w, dconv_w: [d_inner][d_conv] fp32
 *              conv_state, conv_state_out, dconv_state: [batch][d_conv-1][d_inner]
 *                (the d_conv-1 inputs that precede u_0, oldest first), io dtype
 *  Dtypes    activations and their gradients use dims->io (fp32 or bf16);
 *            parameters, states, checkpoints and dD/dconv_w are fp32.  Device
 *            arithmetic is fp32; bf16 results are rounded to nearest even.
 *  Pointers  every data pointer is a device pointer (hipMalloc'd or a torch
 *            tensor), aligned to its element size; outputs must not alias
 *            inputs.  `dims` is a host pointer.  Optional pointers may be NULL
 *            as documented per argument.
 *  Ownership the caller owns every buffer.  The library never allocates device
 *            memory; it uses only the caller's workspace.
 *  Stream    `stream` is a hipStream_t (NULL = the default stream).  Every call
 *            only enqueues work on that stream and returns; nothing is
 *            synchronised.  The stream and every device pointer belong to the
 *            calling thread's current device.
 *  Workspace `ws` of at least naju_workspace_bytes(op, dims) bytes, zero-filled
 *            before its first use (naju_workspace_init, or any zero fill).
 *            Each call leaves it in a reusable state when its work completes,
 *            for further calls of the same entry point with the same dims.
 *            Zero-fill it again before using it for another entry point or
 *            other dims.  Calls that share one workspace must be ordered (same
 *            stream or explicit dependencies); concurrent calls need separate
 *            workspaces.
 *  Errors    arguments are validated before anything is enqueued: any status
 *            other than NAJU_OK and NAJU_EHIP means nothing was enqueued.
 *            NAJU_EHIP reports a HIP launch error.  naju_last_error() returns a
 *            thread-local message describing the last failure.
 *  Sizes     batch, seqlen, d_inner >= 0 (any zero makes the call a no-op
 *            except for the state outputs: with seqlen == 0, x_final = x0 and
 *            conv_state_out = conv_state).  d_state in {16, 64}; d_conv == 4
 *            for the block entry points.
 */
#ifndef NAJU_H
#define NAJU_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NAJU_OK = 0,
    NAJU_EINVAL = 1,       /* bad argument: NULL pointer, bad size, misalignment */
    NAJU_EUNSUPPORTED = 2, /* valid but not built: d_state or d_conv not instantiated */
    NAJU_EWORKSPACE = 3,   /* ws NULL or smaller than naju_workspace_bytes() */
    NAJU_EHIP = 4          /* the HIP runtime reported an error */
} naju_status_t;

typedef enum { NAJU_F32 = 0, NAJU_BF16 = 1 } naju_dtype_t;

/* Added to naju_adamw_step()'s state_bits 8. */
enum { NAJU_STOCHASTIC = 256 };

typedef enum {
    NAJU_OP_SCAN_FWD = 0,
    NAJU_OP_SCAN_BWD = 1,
    NAJU_OP_BLOCK_FWD = 2,
    NAJU_OP_BLOCK_BWD = 3
} naju_op_t;

typedef struct {
    int64_t batch;   /* Bt */
    int64_t seqlen;  /* L */
    int64_t d_inner; /* Di: channels */
    int64_t d_state; /* N: 16 or 64 */
    int32_t d_conv;  /* K: 4 (block entry points; ignored by the scan ones) */
    int32_t io;      /* naju_dtype_t of activations and their gradients */
} naju_dims_t;

/* Bytes of workspace the entry point `op` needs for `dims` (0 if dims invalid). */
size_t naju_workspace_bytes(naju_op_t op, const naju_dims_t *dims);

/* Bytes of the optional forward checkpoint buffer (fp32 chunk-boundary states
 * written by the forward and read by the backward).  Its layout is private to
 * the library; it is valid only for the same dims. */
size_t naju_ckpt_bytes(const naju_dims_t *dims);

/* Zero-fills a workspace on `stream` (with a kernel, so it may be captured). */
naju_status_t naju_workspace_init(void *ws, size_t ws_bytes, void *stream);

/* Synchronises `stream`, then reads the workspace's device-side error word:
 * *flags = 0 if every cross-workgroup wait of the previous calls completed,
 * nonzero if one gave up after its bounded spin (results are then invalid).
 * Every kernel that waits on another workgroup takes its work items from an
 * in-order counter (the matrix-core forward by default), so a
 * wait is always on an item already held by a running workgroup and ends
 * however many workgroups the device runs at once; the bound (about 0.4 s of
 * polling) only catches a device stalled for longer than that. */
naju_status_t naju_workspace_check(const void *ws, size_t ws_bytes, void *stream,
                                   uint32_t *flags);

/*
 * Scan forward: y = ys (readout + feedthrough), x_final = x_L.
 *   h, a, b   [Bt][L][Di] io          token activations, forget and write
 *                                     gate pre-activations
 *   B, C      [Bt][L][N]  io          write / read directions
 *   D         [Di] fp32               direct feedthrough
 *   x0        [Bt][Di][N] fp32 or NULL (= zeros)  initial state
 *   y         [Bt][L][Di] io          output (written)
 *   x_final   [Bt][Di][N] fp32 or NULL            final state (written)
 *   ckpt      naju_ckpt_bytes() or NULL           checkpoints for the backward
 */
naju_status_t naju_scan_fwd(const naju_dims_t *dims, const void *h, const void *a,
                            const void *b, const void *B, const void *C, const float *D,
                            const float *x0, void *y, float *x_final, float *ckpt, void *ws,
                            size_t ws_bytes, void *stream);

/*
 * Scan backward.  Inputs are the forward's inputs plus
 *   ckpt      from naju_scan_fwd on the same inputs, or NULL (recomputed)
 *   dy        [Bt][L][Di] io          dLoss/dy
 *   dx_final  [Bt][Di][N] fp32 or NULL (= zeros)  dLoss/dx_final
 * Outputs (written, not accumulated):
 *   dh, da, db [Bt][L][Di] io;  dB, dC [Bt][L][N] io;  dD [Di] fp32;
 *   dx0 [Bt][Di][N] fp32 or NULL (skipped)
 */
naju_status_t naju_scan_bwd(const naju_dims_t *dims, const void *h, const void *a,
                            const void *b, const void *B, const void *C, const float *D,
                            const float *x0, const float *ckpt, const void *dy,
                            const float *dx_final, void *dh, void *da, void *db, void *dB,
                            void *dC, float *dD, float *dx0, void *ws, size_t ws_bytes,
                            void *stream);

/*
 * Block forward: y = ScanReadout(SiLU(conv(u)), a, b, B, C, D) * SiLU(z).
 *   u, z          [Bt][L][Di] io      conv input and modulation input
 *   conv_w        [Di][K] fp32        depthwise taps (no bias)
 *   conv_state    [Bt][K-1][Di] io or NULL (= zeros)  inputs preceding u_0
 *   a, b, B, C, D, x0                 as naju_scan_fwd
 *   y             [Bt][L][Di] io      output (written)
 *   x_final       [Bt][Di][N] fp32 or NULL
 *   conv_state_out [Bt][K-1][Di] io or NULL: last K-1 rows of [conv_state; u]
 *   ckpt          naju_ckpt_bytes() or NULL
 */
naju_status_t naju_block_fwd(const naju_dims_t *dims, const void *u, const void *z,
                             const float *conv_w, const void *conv_state, const void *a,
                             const void *b, const void *B, const void *C, const float *D,
                             const float *x0, void *y, float *x_final, void *conv_state_out,
                             float *ckpt, void *ws, size_t ws_bytes, void *stream);

/*
 * Block backward.  Inputs: the block forward's inputs, ckpt (or NULL), dy and
 * dx_final (or NULL).  Outputs (written):
 *   du, dz, da, db [Bt][L][Di] io;  dB, dC [Bt][L][N] io;
 *   dconv_w [Di][K] fp32;  dD [Di] fp32;
 *   dconv_state [Bt][K-1][Di] io or NULL;  dx0 [Bt][Di][N] fp32 or NULL
 */
naju_status_t naju_block_bwd(const naju_dims_t *dims, const void *u, const void *z,
                             const float *conv_w, const void *conv_state, const void *a,
                             const void *b, const void *B, const void *C, const float *D,
                             const float *x0, const float *ckpt, const void *dy,
                             const float *dx_final, void *du, void *dz, float *dconv_w,
                             void *dconv_state, void *da, void *db, void *dB, void *dC,
                             float *dD, float *dx0, void *ws, size_t ws_bytes, void *stream);

/*
 * Decode step: one token of the scan for every batch row, with the state
 * carried in place -- the streaming-generation form of the same recurrence
 * and readout (naju_scan_fwd on one token with x0 = x, x_final written back
 * to x).  dims->seqlen is not used; no workspace.
 *   h, a, b   [Bt][Di] io         this token's activation and gate pre-activations
 *   B, C      [Bt][N]  io
 *   D         [Di] fp32
 *   x         [Bt][Di][N] fp32, 16-byte aligned: the state before the token on
 *             entry, after it on return (read and written by the call)
 *   y         [Bt][Di] io         output (written)
 * batch <= 65535.
 */
naju_status_t naju_scan_step(const naju_dims_t *dims, const void *h, const void *a,
                             const void *b, const void *B, const void *C, const float *D,
                             float *x, void *y, void *stream);

/*
 * Block decode step: one token of the block (naju_block_fwd on one token with
 * x0 = x and conv_state, both updated in place).
 *   u, z          [Bt][Di] io
 *   conv_w        [Di][K] fp32
 *   conv_state    [Bt][K-1][Di] io: the K-1 inputs before u (oldest first) on
 *                 entry; shifted by one token (u appended) on return
 *   a, b, B, C, D, x, y   as naju_scan_step
 */
naju_status_t naju_block_step(const naju_dims_t *dims, const void *u, const void *z,
                              const float *conv_w, void *conv_state, const void *a,
                              const void *b, const void *B, const void *C, const float *D,
                              float *x, void *y, void *stream);

/*
 * Mixer layer forward (bf16 io only): the block flowchart of the same page
 * ("Background and main changes") around the scan -- input projection, causal
 * depthwise conv + SiLU, forget / write gate and B/C projections, the block
 * scan with readout, feedthrough and SiLU(z) modulation, output projection and
 * residual.  Per token, with row vectors and weights stored [in][out]:
 *     u = xn W_u;  z = xn W_z;  h = SiLU(conv(u))             (conv as naju_block_fwd)
 *     a = h W_a + a_bias;  b = h W_b + b_bias;  B = h W_B;  C = h W_C
 *     y = naju_block_fwd(u, z, conv_w, conv_state, a, b, B, C, D)
 *     out = y W_out + res
 * u, z, h, a, b, B, C and y are bf16 intermediates in the workspace (each
 * rounded to nearest even from fp32); the projections read the bf16 h, the
 * scan recomputes h from u in fp32.  The projections run through hipBLASLt
 * (fp32 accumulation); its handle is created on a device's first call and
 * kept for the process.
 *   dims          batch, seqlen, d_inner, d_state as elsewhere; d_conv == 4;
 *                 io == NAJU_BF16; d_inner % 8 == 0
 *   d_model       width of the layer's input and output, % 8 == 0
 *   xn            [Bt][L][d_model] bf16     normalized tokens
 *   res           [Bt][L][d_model] bf16 or NULL (= no residual)
 *   W_u, W_z      [d_model][d_inner] bf16   input projection (conv branch, gate branch)
 *   conv_w        [d_inner][4] fp32;  conv_state [Bt][3][d_inner] bf16 or NULL
 *   W_a, W_b      [d_inner][d_inner] bf16;  a_bias, b_bias [d_inner] fp32
 *   W_B, W_C      [d_inner][d_state] bf16
 *   D             [d_inner] fp32
 *   W_out         [d_inner][d_model] bf16
 *   out           [Bt][L][d_model] bf16 (written)
 *   ws            naju_mixer_workspace_bytes() bytes, 256-byte aligned, zero-filled
 *                 before first use (as for the other entry points)
 * Matrices, conv_w and conv_state must be 16-byte aligned; batch <= 65535,
 * seqlen <= 16 * 65535.  The first call for a shape asks hipBLASLt's heuristic
 * for each projection's algorithm (host work only) and caches it.  A hipBLASLt
 * failure returns NAJU_EHIP; work already enqueued is not undone.
 */
size_t naju_mixer_workspace_bytes(const naju_dims_t *dims, int64_t d_model);
naju_status_t naju_mixer_fwd(const naju_dims_t *dims, int64_t d_model, const void *xn,
                             const void *res, const void *W_u, const void *W_z,
                             const float *conv_w, const void *conv_state, const void *W_a,
                             const float *a_bias, const void *W_b, const float *b_bias,
                             const void *W_B, const void *W_C, const float *D,
                             const void *W_out, void *out, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * Mixer layer backward: the reverse mode of naju_mixer_fwd for the upstream
 * gradient d_out = dLoss/dout.  The call recomputes the layer's forward
 * intermediates (u, z, h, a, b, B, C, y and the scan checkpoints) in its
 * workspace, then runs the output projection's, the block scan's (the
 * naju_block_bwd kernels), the gate / B / C projections', the projection
 * path's conv + SiLU and the input projections' reverse modes.  The stored
 * bf16 intermediates pass gradients unchanged (rounding taken as the
 * identity); dy and the block backward's gradients are kept in bf16, the
 * projections' sums in fp32.  The residual's gradient is d_out itself.
 *   inputs        as naju_mixer_fwd (no res), and
 *   d_out         [Bt][L][d_model] bf16
 * outputs (written, fp32 unless noted):
 *   dxn [Bt][L][d_model];  dW_u, dW_z [d_model][d_inner];  dconv_w [d_inner][4];
 *   dconv_state [Bt][3][d_inner] bf16 or NULL (needs conv_state);
 *   dW_a, dW_b [d_inner][d_inner];  da_bias, db_bias [d_inner];
 *   dW_B, dW_C [d_inner][d_state];  dD [d_inner];  dW_out [d_inner][d_model]
 *   fwd_ws        NULL (the forward intermediates are recomputed), or the workspace
 *                 of the naju_mixer_fwd call on the same inputs, untouched since
 *                 (it holds u, z, h, a, b, B, C, y and the scan's checkpoints, so
 *                 the recomputation is skipped); fwd_ws_bytes its size
 *   ws            naju_mixer_bwd_workspace_bytes() bytes, as for the forward
 * Output buffers must be 16-byte aligned (dD 4-byte).
 */
size_t naju_mixer_bwd_workspace_bytes(const naju_dims_t *dims, int64_t d_model);
naju_status_t naju_mixer_bwd(const naju_dims_t *dims, int64_t d_model, const void *xn,
                             const void *W_u, const void *W_z, const float *conv_w,
                             const void *conv_state, const void *W_a, const float *a_bias,
                             const void *W_b, const float *b_bias, const void *W_B,
                             const void *W_C, const float *D, const void *W_out,
                             const void *d_out, float *dxn, float *dW_u, float *dW_z,
                             float *dconv_w, void *dconv_state, float *dW_a, float *da_bias,
                             float *dW_b, float *db_bias, float *dW_B, float *dW_C, float *dD,
                             float *dW_out, const void *fwd_ws, size_t fwd_ws_bytes, void *ws,
                             size_t ws_bytes, void *stream);

/*
 * Scan forward without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Same arguments, outputs and results as
 * naju_scan_fwd; it allocates nothing, neither itself nor through a library.
 * Its scratch is a 64 MiB device array inside the library, one per GPU, zero
 * at load and held until the process ends; shapes whose forward workspace
 * (naju_workspace_bytes(NAJU_OP_SCAN_FWD, dims)) exceeds it return
 * NAJU_EWORKSPACE before anything is enqueued.  Every call on a GPU shares that
 * GPU's scratch: calls that overlap on one GPU (different streams, or host
 * threads) race and must not be issued.
 *   flags  device uint32 or NULL: receives the call's error word (0: every
 *          cross-workgroup wait completed; nonzero: one gave up and the
 *          results are invalid), which the call then clears in the scratch
 */
naju_status_t naju_scan_fwd_noalloc(const naju_dims_t *dims, const void *h, const void *a,
                                    const void *b, const void *B, const void *C, const float *D,
                                    const float *x0, void *y, float *x_final, float *ckpt,
                                    uint32_t *flags, void *stream);

/*
 * ---- Around the mixer layer: tokens in, losses and tokens out ----
 * The entry points below serve the two ends of a language model built from
 * mixer layers and its decode step.  The conventions above hold, with sizes as
 * plain arguments: contiguous row-major tensors unless a row stride is given,
 * `io` the type of activations, arguments checked before anything is enqueued.
 * Token ids are int32.
 */

/*
 * Token embedding: out[t] = scale * W[ids[t]], and zeros where ids[t] lies
 * outside [0, vocab) (padding).  No workspace.
 *   ids  [tokens] int32;  W [vocab][d_model] io;  out [tokens][d_model] io (written)
 * tokens <= 2^28, vocab <= 2^30, d_model <= 2^20.
 */
naju_status_t naju_embed_fwd(int64_t tokens, int64_t vocab, int64_t d_model, int32_t io,
                             const int32_t *ids, const void *W, float scale, void *out,
                             void *stream);

/*
 * Gradient of the embedding with respect to W:
 *     dW[v] = scale * sum over t with ids[t] == v of dout[t]
 * summed in fp32 in the order of t within runs, without floating-point
 * atomics: equal inputs give equal bits.  Ids outside [0, vocab) contribute
 * nothing.
 *   dout  [tokens][d_model] io
 *   accumulate  0: dW is written, rows of tokens that do not occur with zeros;
 *               nonzero: the sums are added to dW and the other rows are not
 *               touched (an output layer that shares W has its gradient there)
 *   dW    [vocab][d_model] fp32
 *   ws    naju_embed_bwd_workspace_bytes() bytes, 256-byte aligned (no initial
 *         contents needed; not used when tokens == 0)
 */
size_t naju_embed_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d_model);
naju_status_t naju_embed_bwd(int64_t tokens, int64_t vocab, int64_t d_model, int32_t io,
                             const int32_t *ids, const void *dout, float scale,
                             int32_t accumulate, float *dW, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * Distillation from a teacher's top logits.  Per row, with student logits s,
 * teacher entries (i_j, t_j), j < k, and temperature tau:
 *     x_v = s_v / tau,  lse = log sum_v exp x_v
 *     p   = softmax over the valid entries of t_j / tau
 *     loss = tau^2 sum_j p_j (log p_j - (x_{i_j} - lse))
 * An entry is valid when i_j lies in [0, vocab) and t_j is not -inf; shorter
 * lists are filled up with either.  A row without a valid entry has loss 0 and
 * gradient 0.  An index that a row lists more than once counts each time.  A
 * student logit of -inf has probability 0 (a teacher probability above 0 there
 * makes the loss +inf); NaN, and +inf, make the row's results NaN.  With k == 1
 * and tau == 1 the loss is the cross entropy of a hard label.  No workspace.
 *   logits    [rows][ld] io, the first vocab of every row's ld >= vocab elements
 *   t_ids     [rows][k] int32;  t_logits [rows][k] fp32;  k <= 512
 *   temperature  > 0, finite, with a finite reciprocal (5e-39 and more)
 *   loss, lse [rows] fp32 (written); lse is infinite where it leaves fp32 (a row of
 *             nothing but fp32's lowest value at temperatures below 1)
 * Finite logits and teacher values may lie anywhere in their types' ranges: a
 * maximum is taken off before a difference is scaled.
 * rows, vocab <= 2^30.
 */
naju_status_t naju_distill_fwd(int64_t rows, int64_t vocab, int64_t k, int32_t io,
                               const void *logits, int64_t ld, const int32_t *t_ids,
                               const float *t_logits, float temperature, float *loss, float *lse,
                               void *stream);

/*
 * Its gradient for the upstream gradient g of each row's loss:
 *     dlogits_v = g tau ([any valid entry] exp(x_v - lse) - sum_{j : i_j = v} p_j)
 * A row with g == 0 gets zeros, whatever it holds.
 *   lse       [rows] fp32 from naju_distill_fwd on the same inputs (where it is
 *             larger than 16384, too coarse to form exp(x_v - lse) from, it is formed
 *             again from the row)
 *   g         [rows] fp32
 *   dlogits   [rows][ld_d] io: the first vocab elements of every row are written,
 *             the others are not touched
 */
naju_status_t naju_distill_bwd(int64_t rows, int64_t vocab, int64_t k, int32_t io,
                               const void *logits, int64_t ld, const int32_t *t_ids,
                               const float *t_logits, float temperature, const float *lse,
                               const float *g, void *dlogits, int64_t ld_d, void *stream);

/*
 * Loss and gradient in one call, for upstream gradients that are known before
 * the loss is (a mean or a weighted sum over rows).  Arguments as above.
 */
naju_status_t naju_distill_fwd_bwd(int64_t rows, int64_t vocab, int64_t k, int32_t io,
                                   const void *logits, int64_t ld, const int32_t *t_ids,
                                   const float *t_logits, float temperature, const float *g,
                                   float *loss, float *lse, void *dlogits, int64_t ld_d,
                                   void *stream);

/*
 * Logits made ready for the choice of a token.  Per row, with c_v the number of
 * times v occurs among the first lengths[row] entries of the row's history:
 *     x = l_v
 *     where c_v > 0:  x = x > 0 ? x / repetition : x * repetition;
 *                     x = x - frequency c_v;  x = x - presence
 *     x = x + bias of v
 *     x = -inf where bit v of the row's mask is 0
 *     out_v = x;  best = the lowest v whose x is largest
 * in fp32, every operation rounded by itself.  best is -1 where no x is above
 * -inf (NaN is never best).
 *   logits    [rows][ld] io, the first vocab of every row's ld >= vocab elements
 *   history   [rows][history_len] int32, entries outside [0, vocab) ignored
 *             (NULL with history_len 0); history_len < 2^20
 *   lengths   [rows] int32 (taken into [0, history_len]), or NULL (= history_len)
 *   repetition, presence, frequency  [rows] fp32, each may be NULL (= none)
 *   bias_ids, bias  [rows][n_bias] int32 and fp32: pairs of a token and what is
 *             added to it (-inf forbids it); ids outside [0, vocab) are ignored; of
 *             several pairs that name one token the first counts; n_bias < 4095
 *   mask      [rows][ceil(vocab / 32)] uint32 or NULL (= all allowed): bit v % 32
 *             of word v / 32, 1 = allowed; bits past vocab are ignored
 *   out       [rows][vocab] fp32 (written)
 *   best      [rows] int32 (written) or NULL
 *   ws        naju_logits_workspace_bytes() bytes, 256-byte aligned, zero-filled
 *             before its first use and left reusable for calls with up to that
 *             many rows; may be NULL when best is
 * rows <= 2^24, vocab <= 2^30.
 */
size_t naju_logits_workspace_bytes(int64_t rows);
naju_status_t naju_logits_process(int64_t rows, int64_t vocab, int32_t io, const void *logits,
                                  int64_t ld, const int32_t *history, int64_t history_len,
                                  const int32_t *lengths, const float *repetition,
                                  const float *presence, const float *frequency,
                                  const int32_t *bias_ids, const float *bias, int64_t n_bias,
                                  const uint32_t *mask, float *out, int32_t *best, void *ws,
                                  size_t ws_bytes, void *stream);

/*
 * Linear layer with 4-bit weights, for the few rows of a decode step:
 *     y[r][n] = sum_k x[r][k] (q[n][k] - z[n][k / group]) s[n][k / group]
 *               + bias[n] + res[r][n]
 * summed in fp32, one rounding to bf16.  No workspace.
 *   x         [rows][d_in] bf16
 *   qweight   [d_out][d_in / 2] uint8: the code of input 2i in the low half of byte
 *             i, that of input 2i + 1 in the high half (any alignment)
 *   scales    [d_out][ceil(d_in / group)] bf16
 *   zeros     [d_out][ceil(d_in / group)] uint8, or NULL (= 8 everywhere)
 *   bias      [d_out] fp32 or NULL;  res [rows][d_out] bf16 or NULL
 *   y         [rows][d_out] bf16 (written)
 * d_in even, at most 2^24; d_out <= 2^26; group 32, 64 or 128 (the last group of a
 * row may be shorter).  Any number of rows up to 2^20; the weights are read once
 * for every 64 of them.  An infinite or NaN x makes its row of y NaN or infinite, and
 * so does a group of inputs whose magnitudes add up to more than 2e36.
 */
naju_status_t naju_w4_linear(int64_t rows, int64_t d_in, int64_t d_out, int64_t group,
                             const void *x, const uint8_t *qweight, const void *scales,
                             const uint8_t *zeros, const float *bias, const void *res, void *y,
                             void *stream);

/*
 * Quantises weights stored [in][out], as the mixer layer's are, into that
 * layout.  Per output and group, to the nearest code: without zeros
 * s = max|w| / 7 and codes 8 + round(w / s); with them s = (max(w, 0) -
 * min(w, 0)) / 15, z = round(-min / s) and codes z + round(w / s), into 0 .. 15.
 * The scale is rounded to bf16 before the codes are formed.
 *   W         [d_in][d_out] io (fp32 or bf16), finite
 *   qweight, scales (written);  zeros (written) or NULL (codes around 8)
 */
naju_status_t naju_w4_quantize(int64_t d_in, int64_t d_out, int64_t group, int32_t io,
                               const void *W, uint8_t *qweight, void *scales, uint8_t *zeros,
                               void *stream);

/*
 * ---- The rest of a layer: norms, a second token mixer, the update ----
 * The conventions of the section above hold.
 */

/*
 * The norms before and after a block, with the block's gate and residual scale.
 * Per token, over d_model channels:
 *     n  = y / sqrt(mean y^2 + eps) * w_post      (y itself without w_post)
 *     x' = x + scale * n * SiLU(z)                (without scale, z: 1)
 *     xn = x' / sqrt(mean x'^2 + eps) * w_pre
 * in fp32, each output rounded once (xn is formed from the unrounded x').
 *   x         [tokens][d_model] x_io  the residual stream
 *   y         [tokens][d_model] io    the block's output, or NULL: x' = x, and z,
 *             scale, w_post and x_new are NULL too
 *   z         [tokens][d_model] io    gate pre-activation, or NULL
 *   scale, w_post, w_pre  [d_model] fp32, each may be NULL (w_pre: no xn)
 *   x_new     [tokens][d_model] x_io (written)
 *   xn        [tokens][d_model] io (written), or NULL with w_pre
 * io BF16 with x_io BF16 or F32, or both F32.  d_model 4 to 8192.  eps >= 0.
 * Squares are summed as they are: a row whose sum of squares leaves fp32 (values
 * of 1e17 and more) has the norm 0, a row that holds NaN or infinity has NaN.  With
 * eps 0 a row of zeros has NaN, one whose squares vanish (values below 1e-22) infinities.
 */
naju_status_t naju_res_norm_fwd(int64_t tokens, int64_t d_model, int32_t io, int32_t x_io,
                                const void *x, const void *y, const void *z, const float *scale,
                                const float *w_post, const float *w_pre, float eps, void *x_new,
                                void *xn, void *stream);

/*
 * Its gradients, for the gradients dxn of xn and dx_new of x':
 *   dx     [tokens][d_model] g_io   of x' with what reached it through xn, which is
 *          the gradient of x too (written)
 *   dy, dz [tokens][d_model] io     (written; with y, z)
 *   dscale, dw_post, dw_pre  [d_model] fp32 (written), each may be NULL; sums over
 *          the tokens in a fixed order, zeros for no tokens
 *   dxn    [tokens][d_model] g_io, with w_pre;  dx_new  [tokens][d_model] g_io or
 *          NULL (= zeros), one of the two at least
 *   x_new  [tokens][d_model] x_io   x' (with w_pre)
 *   y, z, scale, w_post, w_pre, eps as in the forward call
 *   g_io   F32, or BF16 where io is BF16
 *   ws     naju_res_norm_bwd_workspace_bytes() bytes, 256-byte aligned (no initial
 *          contents needed; not used when tokens == 0)
 */
size_t naju_res_norm_bwd_workspace_bytes(int64_t tokens, int64_t d_model);
naju_status_t naju_res_norm_bwd(int64_t tokens, int64_t d_model, int32_t io, int32_t x_io,
                                int32_t g_io, const void *dxn, const void *dx_new,
                                const void *x_new, const void *y, const void *z,
                                const float *scale, const float *w_post, const float *w_pre,
                                float eps, void *dx, void *dy, void *dz, float *dscale,
                                float *dw_post, float *dw_pre, void *ws, size_t ws_bytes,
                                void *stream);

/*
 * Linear attention with a decay for each head, over sequences:
 *     S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
 *   q         [batch][seqlen][heads][d_key] io, k [..][kv_heads][d_key], v
 *             [..][kv_heads][d_value]; ldq, ldk, ldv: elements from one token to
 *             the next (parts of a joint projection), a multiple of 16 bytes, 2^20 at
 *             most; rows of the batch lie seqlen times as far apart (seqlen 1: up to
 *             2^40, the last token of longer rows).  Heads h of q read the key and
 *             value of head h / (heads / kv_heads)
 *   log_decay [heads] fp32, at most 0 (-inf: only the token itself); a constant of
 *             the head, to which there is no gradient
 *   state     [batch][heads][d_key][d_value] fp32 before the first token, or NULL
 *             (= zeros);  state_out  after the last (written), or NULL; may be state
 *   lengths   [batch] int32 (taken into [0, seqlen]) or NULL (= seqlen): tokens of a
 *             row; what lies behind them is not read, and o is zero there
 *   o         [batch][seqlen][heads][d_value] io (written)
 *   ws        naju_linattn_fwd_workspace_bytes() bytes, 256-byte aligned (no initial
 *             contents needed; 0 bytes: may be NULL)
 * d_key, d_value multiples of 8 from 8 to 256; q, k, v, o (and the gradients) 16-byte
 * aligned.  Sums and states are fp32; bf16 products with a state and with the scores of a
 * chunk's tokens take 16 bits of these (two bf16 parts).  A NaN or infinite input reaches
 * what the formula says, an infinity also as NaN.
 */
size_t naju_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                        int64_t kv_heads, int64_t d_key, int64_t d_value);
naju_status_t naju_linattn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                               int64_t d_key, int64_t d_value, int32_t io, const void *q,
                               int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                               const float *log_decay, const float *state, const int32_t *lengths,
                               float scale, void *o, float *state_out, void *ws, size_t ws_bytes,
                               void *stream);

/*
 * Its gradients, for the gradients dout of o and dstate_out of the last state (NULL:
 * zeros).  dout [batch][seqlen][heads][d_value] io; what lies behind a row's length
 * is not read.
 *   dq, dk, dv  [batch][seqlen][heads or kv_heads][d] io, contiguous (written, zero
 *             behind a row's length; those of a shared head are summed in fp32 over
 *             its readers)
 *   dstate    [batch][heads][d_key][d_value] fp32 (written), or NULL
 *   ws        naju_linattn_bwd_workspace_bytes() bytes, as for the forward
 * A NaN or infinite input reaches what the formulas say, an infinity also as NaN.
 */
size_t naju_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                        int64_t kv_heads, int64_t d_key, int64_t d_value);
naju_status_t naju_linattn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                               int64_t d_key, int64_t d_value, int32_t io, const void *q,
                               int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                               const float *log_decay, const float *state, const int32_t *lengths,
                               float scale, const void *dout, const float *dstate_out, void *dq,
                               void *dk, void *dv, float *dstate, void *ws, size_t ws_bytes,
                               void *stream);

/*
 * One token of it for every batch row: q [batch][heads][d_key], k, v
 * [batch][kv_heads][..], o [batch][heads][d_value], contiguous.
 *   state     as above, 16-byte aligned, read;  state_out  written, state itself for a
 *             step in place, or another buffer that keeps the state before the token
 * No workspace.
 */
naju_status_t naju_linattn_step(int64_t batch, int64_t heads, int64_t kv_heads, int64_t d_key,
                                int64_t d_value, int32_t io, const void *q, const void *k,
                                const void *v, const float *log_decay, const float *state,
                                float scale, void *o, float *state_out, void *stream);

/*
 * One AdamW step over a list of tensors.  Per element, with t the step's number:
 *     g = grad_scale g
 *     m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *     p = p - lr weight_decay p
 *           - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32.  state_bits 32: m, v fp32.  state_bits 8: m and the square root of v as
 * 8-bit floats (e4m3: 4 exponent bits of bias 7, 3 mantissa bits, no infinities),
 * each times the fp32 scale of its 256 consecutive elements (the tensor's last block
 * may be shorter).  A scale is its block's largest magnitude / 448 (0 below 2^-120,
 * and the block then holds zeros); a root that would be 0 beside a first moment that is
 * not is stored as the smallest code (2^-9 of its scale); p is formed from the unrounded m
 * and v.  Zeros (codes and scales) are the states of a first step.
 *   state_bits 8  rounds values to nearest even: each step's states are as near as 8 bits
 *             come, but a change of less than half a code (3 to 6 %) is lost at every step
 *             anew.  With beta2 = 0.999 a root falls by 0.05 % a step at most, so only
 *             its block's largest follows gradients that become smaller.
 *   state_bits 8 + NAJU_STOCHASTIC  rounds to one of the two neighbouring codes, with
 *             probabilities that make the stored value right in the mean, so that states
 *             follow their formulas over the steps: what training is to use.  The random
 *             numbers are functions of the step's number and the element's index: equal
 *             calls give equal bits (so replays of a captured call need step_dev).
 * A NaN gradient makes its element NaN, one that is infinite or has an infinite
 * square its block's states.
 *   tensors   host array, read during the call only
 *   step      number of this step, from 1; or step_dev, a device int32 that holds it
 *             (a captured graph then reads it at every replay; it is not advanced)
 *   lr_dev    device fp32 that holds the learning rate, or NULL (= lr)
 *   grad_scale  device fp32 (of a clipped norm, say), or NULL (= 1)
 *   g_io      type of every tensor's gradient
 * Two tensors whose p overlap are refused; the other outputs must not overlap.
 * An output may be its own input (NULL says so); otherwise outputs must not alias inputs.
 */
typedef struct {
    int64_t n;               /* elements; 0: the tensor is skipped */
    float *p;                /* [n] fp32 parameters */
    const void *g;           /* [n] g_io gradient */
    void *m, *v;             /* [n] fp32 or e4m3 states */
    float *m_scale, *v_scale; /* [ceil(n / 256)] with 8-bit states */
    float *p_out;            /* where results go; NULL: in place */
    void *m_out, *v_out;
    float *m_scale_out, *v_scale_out;
    void *copy;              /* [n] bf16: the new p rounded (written), or NULL */
} naju_adamw_tensor_t;
naju_status_t naju_adamw_step(int64_t n_tensors, const naju_adamw_tensor_t *tensors,
                              int32_t g_io, int32_t state_bits, double lr, double beta1,
                              double beta2, double eps, double weight_decay, int64_t step,
                              const int32_t *step_dev, const float *lr_dev,
                              const float *grad_scale, void *stream);

/* Thread-local description of the last non-OK status ("" if none). */
const char *naju_last_error(void);

/* Library version string. */
const char *naju_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NAJU_H */
