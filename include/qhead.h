/*
 * qhead.h -- C ABI of the GB300 fused quantized LM-head ("Flash Cut-Cross-
 * Entropy" over a frozen 4/8-bit affine-quantized head).
 *
 * The operation is the one described on the page "mlx-bun 0.0.4 -> 0.0.6"
 * (src/train/flash-cce.ts): for hidden states h[M,H] and a quantized head W
 * (FlashCceHead: packed uint32 codes, per-group scales and biases, bits,
 * group size, optional final-logit soft cap)
 *
 *     w[v,d]   = scale[v, d/group] * q[v,d] + bias[v, d/group]
 *     raw[m,v] = sum_d h[m,d] * w[v,d]
 *     z[m,v]   = cap * tanh(raw[m,v] / cap)      (z = raw when cap <= 0)
 *     lse[m]   = log sum_v exp(z[m,v])
 *     logp[m]  = z[m, target[m]] - lse[m]
 *
 * and, for the frozen head, the gradient of sum_m dlogp[m] * logp[m]:
 *
 *     dh[m,:]  = sum_v dlogp[m] * (1[v == target[m]] - exp(z[m,v] - lse[m]))
 *                              * sech2[m,v] * w[v,:]
 *     sech2    = 1 - tanh^2(raw / cap)           (1 when the cap is off)
 *
 * The vocab loop runs inside the kernels: neither the [M,V] logits nor a
 * dequantized [V,H] head is ever written to device memory.  The same call
 * with targets == NULL is the speculative-decode verify step of the page
 * "mlx-bun 0.0.8 -> 0.0.10" (src/spec/generate.ts, picksBatched): one head
 * pass over the gamma+1 window, then the argmax of every position (argmax of
 * the raw logits; the soft cap and the lse shift are monotone, so it is also
 * the argmax of z and of logp).
 *
 * Conventions shared by every entry point
 *   - All array arguments are DEVICE pointers unless stated otherwise.
 *   - The caller owns and allocates every input, output and workspace; the
 *     library allocates nothing and keeps no per-call state.
 *   - Calls are asynchronous and ordered on `stream` (a cudaStream_t passed as
 *     void*; NULL is the legacy default stream).  Nothing synchronizes.
 *   - Return value: QHEAD_OK or an error code; on error nothing was launched
 *     (argument errors) or a launch failed (QHEAD_ECUDA).  A message for the
 *     calling thread is available from qhead_last_error().
 *   - There is no fallback path: unsupported shapes are rejected.
 *   - Kernel time limits: every wait inside a pipelined kernel gives up after
 *     2 s (only a defect or a stalled device makes one that long).  The kernel
 *     then stops waiting, lets the copies and tensor-core operations it has
 *     issued complete, runs to its end and records the failure; qhead_fwd then
 *     writes logp = NaN, lse = NaN and argmax = -1 for every active row, and
 *     qhead_bwd writes NaN to every active row of dh (inactive rows keep their
 *     defined values).  The return value cannot report this, because the call
 *     returns before its kernels run.
 */
#ifndef QHEAD_H
#define QHEAD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define QHEAD_OK 0
#define QHEAD_EINVAL 1        /* null required pointer, misalignment, bad size, small workspace */
#define QHEAD_EUNSUPPORTED 2  /* bits / group / H / sb_dtype the library does not implement */
#define QHEAD_ECUDA 3         /* a CUDA launch or runtime call failed */

/* Element type of scales and biases. */
#define QHEAD_SB_F16 0
#define QHEAD_SB_BF16 1
#define QHEAD_SB_F32 2

/*
 * The frozen quantized head (FlashCceHead on the page "mlx-bun 0.0.4 ->
 * 0.0.6", src/train/flash-cce.ts).
 *   wq       device, uint32 [V, H*bits/32], row-major.  Word j of row v holds
 *            elements j*(32/bits) + k, k = 0 .. 32/bits - 1, element k in bits
 *            bits*k .. bits*k + bits - 1 (least-significant field first).
 *            16-byte aligned.
 *   scales   device, [V, H/group] row-major, of type sb_dtype.  16-byte aligned.
 *   biases   device, [V, H/group] row-major, of type sb_dtype.  16-byte aligned.
 *   V        vocab rows, 1 <= V < 2^31.
 *   H        hidden size: a multiple of 128, 128 <= H <= 8192.
 *   bits     4 or 8.
 *   group    64 (the only group size implemented).
 *   sb_dtype QHEAD_SB_F16, QHEAD_SB_BF16 or QHEAD_SB_F32: the element type of
 *            scales and biases (the page casts any float type to f32).  The
 *            exact fp32 parts of the path (the target logit, the argmax
 *            recheck, the backward's one-hot term) widen the given values
 *            exactly.  The tensor-core and weight-streaming kernels take fp16
 *            operands: for a bf16 or fp32 head each call first rounds scales
 *            and biases to fp16 (nearest) into its workspace -- exact for bf16
 *            values of magnitude in [2^-17, 65504] or zero, one rounding for
 *            fp32 -- which costs a pass over 2 * V * H/64 elements and
 *            2 * 2 * V * H/64 bytes of workspace.  Magnitudes above 65504
 *            become infinite there (results NaN).
 *   softcap  final-logit soft cap; <= 0 turns it off.
 */
typedef struct qhead_head {
    const uint32_t* wq;
    const void* scales;
    const void* biases;
    int64_t V;
    int32_t H;
    int32_t bits;
    int32_t group;
    int32_t sb_dtype;
    float softcap;
} qhead_head;

/*
 * Workspace bytes qhead_fwd / qhead_bwd need for M rows with this head on the
 * current device (the plan depends on M, the head's shape and the SM count).
 * Returns 0 for M == 0 and (size_t)-1 if the arguments are invalid (see
 * qhead_last_error()).  Host-only; launches nothing.
 */
size_t qhead_fwd_workspace(const qhead_head* head, int64_t M);
size_t qhead_bwd_workspace(const qhead_head* head, int64_t M);

/*
 * Forward: logp, lse and argmax for every row of h.
 * Definition: flashCceForward on the page "mlx-bun 0.0.4 -> 0.0.6"
 * (src/train/flash-cce.ts, per-vocab-block partials merged into lse and
 * logp = target logit - lse); argmax as in picksBatched on the page
 * "mlx-bun 0.0.8 -> 0.0.10" (src/spec/generate.ts).
 *   h         device, bf16 [M, H] row-major, 16-byte aligned.  Every |h|
 *             must be below 65504: the kernels stage h as fp16 operands, so a
 *             larger magnitude becomes infinite there and the row's lse, logp
 *             (and dh) come out inf or NaN; no error is returned.
 *   M         rows, >= 0 (M == 0 returns QHEAD_OK and launches nothing).
 *   targets   device, int32 [M], or NULL (verify: no logp).  Each active
 *             row's target must lie in [0, V); a row whose target does not
 *             gets logp = NaN (no out-of-range read happens).
 *   mask      device, uint8 [M], or NULL (all rows active).  mask[m] != 0
 *             means row m is active; inactive rows are skipped and written as
 *             logp = 0, lse = 0, argmax = -1.
 *   logp      device, float [M], or NULL.  Requires targets.
 *   lse       device, float [M], or NULL.
 *   argmax    device, int32 [M], or NULL.  The lowest vocab index attaining
 *             the row's maximum logit (ties within float rounding of each
 *             other may resolve to either index).
 *   workspace device, >= qhead_fwd_workspace(head, M) bytes, 256-byte
 *             aligned; contents on entry are ignored.
 * Outputs may not alias inputs or each other.
 */
int qhead_fwd(const qhead_head* head, const void* h, int64_t M, const int32_t* targets,
              const uint8_t* mask, float* logp, float* lse, int32_t* argmax, void* workspace,
              size_t workspace_bytes, void* stream);

/*
 * Speculative-decode verify with the accept step fused on the device.
 * Definition: page "mlx-bun 0.0.8 -> 0.0.10" (src/spec/generate.ts): one head
 * pass over the gamma + 1 window, the argmax of every position (picksBatched),
 * then the longest prefix of the draft that the argmax reproduces.
 *   h         device, bf16 [B * W, H]: B windows of W = gamma + 1 rows each.
 *   B, W      B >= 0 windows (B == 0 returns QHEAD_OK), W in [1, 2^20].
 *   draft     device, int32 [B, W - 1]: the drafted tokens; required if W > 1.
 *   mask      as for qhead_fwd ([B * W] or NULL); a masked row's argmax is -1,
 *             so a draft token never matches it.
 *   lse       device, float [B * W], or NULL.
 *   argmax    device, int32 [B * W] (required): as for qhead_fwd.
 *   n_accept  device, int32 [B] (required): for window b, the first k < W - 1
 *             with draft[b, k] != argmax[b, k], or W - 1 if every draft token
 *             is accepted.
 *   next_token device, int32 [B], or NULL: argmax[b, n_accept[b]], the token
 *             the target model emits after the accepted prefix.
 *   workspace as for qhead_fwd with M = B * W (qhead_fwd_workspace(head, B * W)).
 * Outputs may not alias inputs or each other.
 */
int qhead_verify(const qhead_head* head, const void* h, int64_t B, int64_t W,
                 const int32_t* draft, const uint8_t* mask, float* lse, int32_t* argmax,
                 int32_t* n_accept, int32_t* next_token, void* workspace, size_t workspace_bytes,
                 void* stream);

/*
 * Backward of the frozen head: dh = d(sum_m dlogp[m] * logp[m]) / dh.
 * Definition: flashCceBackward on the page "mlx-bun 0.0.4 -> 0.0.6"
 * (src/train/flash-cce.ts: logits recomputed per vocab tile, coefficient
 * dlogp * (onehot - softmax) * sech2, dh accumulated over all vocab blocks),
 * with the forward's lse reused.
 *   h, M, targets, mask  as for qhead_fwd (including |h| < 65504); targets
 *             is required.
 *   lse       device, float [M]: the lse qhead_fwd returned for the same
 *             h / head / mask.
 *   dlogp     device, float [M]: the cotangent of each row's logp.
 *   dh        device, float [M, H] row-major, 16-byte aligned.  Every row is
 *             written; inactive rows are exactly 0.
 *   workspace device, >= qhead_bwd_workspace(head, M) bytes, 256-byte aligned.
 * The result is deterministic: fixed-order reductions; where vocab chunks add
 * into a partial buffer, each element receives one addition per chunk, in
 * chunk order.
 */
int qhead_bwd(const qhead_head* head, const void* h, int64_t M, const int32_t* targets,
              const uint8_t* mask, const float* lse, const float* dlogp, float* dh,
              void* workspace, size_t workspace_bytes, void* stream);

/*
 * The blockMax early exit (an approximate backward; page "mlx-bun 0.0.4 ->
 * 0.0.6", src/train/flash-cce.ts: the forward hands per-block logit maxima to
 * the backward, which skips a (token block, vocab block) program when every
 * token has exp(blockMax - lse) < eps and no target lies in the block).
 *
 * qhead_fwd_blockmax: qhead_fwd plus
 *   block_max device, float [M, ceil(V / 256)] row-major, 4-byte aligned: the
 *             maximum capped logit z of each active row over each 256-row
 *             vocab tile (rows with mask 0 are not written).
 *   workspace >= qhead_fwd_blockmax_workspace(head, M) bytes (every M takes
 *             the tensor-core path).
 *
 * qhead_bwd_blockskip: qhead_bwd, except that the (128 consecutive active
 * rows, 256-row vocab tile) blocks in which every row has
 * exp(block_max - lse) < eps and no row's target lies are left out of both
 * backward phases (their coefficients count as 0): dh then differs from the
 * exact one by at most |dlogp| * eps * sum_v |w_v| per row, and the skipped
 * blocks cost nothing.
 *   block_max the forward's block_max for the same h / head / mask.
 *   eps       in [0, 1]; 0 skips nothing (the exact backward).
 *   workspace >= qhead_bwd_blockskip_workspace(head, M) bytes.
 */
size_t qhead_fwd_blockmax_workspace(const qhead_head* head, int64_t M);
int qhead_fwd_blockmax(const qhead_head* head, const void* h, int64_t M, const int32_t* targets,
                       const uint8_t* mask, float* logp, float* lse, int32_t* argmax,
                       float* block_max, void* workspace, size_t workspace_bytes, void* stream);
size_t qhead_bwd_blockskip_workspace(const qhead_head* head, int64_t M);
int qhead_bwd_blockskip(const qhead_head* head, const void* h, int64_t M,
                        const int32_t* targets, const uint8_t* mask, const float* lse,
                        const float* dlogp, const float* block_max, float eps, float* dh,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * The coefficient filter (an approximate backward; page "mlx-bun 0.0.4 ->
 * 0.0.6", src/train/flash-cce.ts: the backward's near-zero coefficient filter
 * skips the dh contraction of a coefficient tile whose largest |coeff| is
 * below eps, since the softmax mass concentrates on a few vocab rows).
 *
 * qhead_bwd_filter: qhead_bwd, except that the blocks of 32 consecutive
 * active rows x 32 vocab rows (rows 32k .. 32k + 31) in which no row's target
 * lies and every softmax term |dlogp[m]| * softmax[m, v] * sech2[m, v] is
 * below eps are cold: their coefficients count as 0, and a dh step whose
 * blocks are all cold is skipped.  Blocks holding a target always stay warm
 * (the one-hot term is added whole).  dh then differs from the exact one by at
 * most eps * sum_v |w_v| per row.  The decision is taken in fp32 on the
 * kernel's logits, so a block whose largest term lies within a small relative
 * distance of eps may go either way.
 *   eps       >= 0 (+inf allowed); 0 makes nothing cold (the exact backward).
 *             NaN or a negative value is rejected (QHEAD_EINVAL).
 *   cold      device, uint8 [ceil(M / 32), ceil(V / 32)] row-major, or NULL:
 *             1 where the block of active rows 32j .. 32j + 31 (ascending
 *             order of the active rows) and vocab rows 32k .. 32k + 31 is
 *             cold, else 0; row blocks past the active rows are 1.
 *   workspace >= qhead_bwd_filter_workspace(head, M) bytes (every M takes
 *             the tensor-core path).
 */
size_t qhead_bwd_filter_workspace(const qhead_head* head, int64_t M);
int qhead_bwd_filter(const qhead_head* head, const void* h, int64_t M, const int32_t* targets,
                     const uint8_t* mask, const float* lse, const float* dlogp, float eps,
                     float* dh, uint8_t* cold, void* workspace, size_t workspace_bytes,
                     void* stream);

/*
 * Workspace bytes qhead_bwd_dw needs for M rows with this head ((size_t)-1 on
 * invalid arguments).
 */
size_t qhead_bwd_dw_workspace(const qhead_head* head, int64_t M);

/*
 * Backward with the head gradient: dw = d(sum_m dlogp[m] * logp[m]) / dW with
 * respect to the dequantized head W[v, d] = scale * q + bias, and optionally
 * dh as qhead_bwd computes it, from one pass of logit recomputation.
 * Definition: the classifier gradient (dC) of the Apple CCE reference that
 * the page "mlx-bun 0.0.4 -> 0.0.6" (src/train/flash-cce.ts) cites; the pages
 * compute none because their head is frozen:
 *     dw[v, :] = sum_m dlogp[m] * (1[v == target_m] - softmax[m, v]) * sech2[m, v] * h[m, :].
 * From it, d/dscale[v, g] = sum_{d in g} q[v, d] * dw[v, d] and
 * d/dbias[v, g] = sum_{d in g} dw[v, d] (the codes are not differentiable).
 *   h, M, targets, mask, lse, dlogp  as for qhead_bwd.
 *   dh        device, float [M, H], 16-byte aligned, or NULL (not computed).
 *   dw        device, float [V, H] row-major, 32-byte aligned; every element is
 *             written (M == 0 or no active row: all zeros).
 *   workspace device, >= qhead_bwd_dw_workspace(head, M) bytes, 256-byte aligned.
 * Every M takes the tensor-core path (dw reuses its per-chunk coefficient
 * blocks).  A row whose target lies outside [0, V) contributes its softmax
 * term but no one-hot term.  If a kernel wait expires, every element of dw is
 * NaN.  The result is deterministic: each dw element is written once, and the
 * rows that share a target are summed in row order.
 */
int qhead_bwd_dw(const qhead_head* head, const void* h, int64_t M, const int32_t* targets,
                 const uint8_t* mask, const float* lse, const float* dlogp, float* dh, float* dw,
                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Forward without a workspace argument, for callers that cannot allocate
 * device memory (no counterpart on the pages: it is an addition for this
 * library's users).  Engines that run the verify step inside a pre-sized
 * memory arena, plugins hosted by frameworks that forbid allocation after
 * start-up, and latency-critical loops that must not enter the allocator
 * cannot call cudaMalloc to provide qhead_fwd's workspace.  This call takes
 * the same arguments as qhead_fwd minus the workspace and computes the same
 * outputs, bit for bit, using instead a fixed scratch array of 8 MiB
 * (8388608 bytes) that lives in the library on every device that loads it,
 * until the process exits.  It allocates nothing and calls no allocating
 * routine.
 *   - The first call with a given device current looks up the array's device
 *     address (cudaGetSymbolAddress) and caches it by device ordinal; make
 *     that first call before any stream capture on the device.  The cached
 *     address belongs to the device's primary context as it was then: after
 *     cudaDeviceReset on that device, or with a non-primary context current
 *     on it, the cached address is stale and this call must not be used.
 *   - M rows whose workspace (qhead_fwd_workspace) exceeds the scratch size
 *     are rejected with QHEAD_EINVAL and a message; nothing is launched.
 *     In practice the scratch holds up to about 200 rows at H = 2560,
 *     V = 262144 (the weight-streaming path up to 16 rows needs a few hundred
 *     KB; the tensor-core path from 17 rows 32 bytes per row and 256-row
 *     vocab tile of partials); a bf16 or fp32 head's fp16 copies of scales
 *     and biases (4 * V * H/64 bytes, 42 MB at that shape) do not fit, so
 *     such heads are rejected.
 *   - Every call shares the one array.  No byte of it needs to start at zero
 *     (a call writes all scratch it reads), but calls whose kernels may
 *     overlap on the GPU (e.g. issued on different streams without ordering)
 *     race on it: order them on one stream or with events.
 *   - A call rejected by the size check disarms the thread's one-shot hooks
 *     (qhead_time_next_head_kernel, qhead_test_stall_next_call) as a forward
 *     call would.
 */
int qhead_fwd_noalloc(const qhead_head* head, const void* h, int64_t M, const int32_t* targets,
                      const uint8_t* mask, float* logp, float* lse, int32_t* argmax,
                      void* stream);

/* Element types of the operators below (the values of QHEAD_SB_*). */
#define QHEAD_F16 0
#define QHEAD_BF16 1
#define QHEAD_F32 2

/*
 * Embedding lookup from the head's table (a tied table; no counterpart on the
 * pages):
 *     out[m, :] = scale * (s[t, d / 64] * q[t, d] + b[t, d / 64]),  t = tokens[m]
 * in fp32 from the scales and biases in their own type, rounded once.
 *   tokens    device, int32 [M].
 *   mask      device, uint8 [M], or NULL (all rows on); a row that is off is
 *             written as zeros, its token is not looked at.
 *   scale     finite.
 *   out       device, [M, H] of type out_dtype, 16-byte aligned.  A row whose
 *             token lies outside [0, V) is written as NaN (no read happens).
 * M == 0 returns QHEAD_OK and launches nothing.
 */
int qhead_embed(const qhead_head* head, const int32_t* tokens, int64_t M, const uint8_t* mask,
                float scale, void* out, int out_dtype, void* stream);

/*
 * The gradient of qhead_embed with respect to the dequantized table:
 *     dw[v, :] = (accumulate ? dw[v, :] : 0) + scale * sum_{m on, tokens[m] == v} dout[m, :]
 * summed in fp32, rows in ascending order in a fixed grouping (deterministic;
 * no atomic additions).  Only the head's V and H matter.
 *   dout      device, [M, H] of type dout_dtype, 16-byte aligned.
 *   dw        device, float [V, H], 32-byte aligned: the layout of
 *             qhead_bwd_dw's dw, so that a tied table's two gradients can be
 *             added into one buffer.  Rows whose token lies outside [0, V)
 *             contribute nothing.  Without accumulate every element is written.
 *   workspace device, >= qhead_embed_bwd_workspace(head, M) bytes, 256-byte aligned.
 */
size_t qhead_embed_bwd_workspace(const qhead_head* head, int64_t M);
int qhead_embed_bwd(const qhead_head* head, const int32_t* tokens, int64_t M, const uint8_t* mask,
                    float scale, const void* dout, int dout_dtype, float* dw, int accumulate,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Layer norm of the rows of x (no counterpart on the pages: the norm whose
 * output is the head's h), or with center == 0 its root-mean-square form:
 *     xc = x - mean(x)  (center == 0: x);  rstd = 1 / sqrt(mean(xc^2) + eps)
 *     y  = xc * rstd * weight + bias
 *   x         device, [M, H] of type x_dtype, row stride ldx >= H elements.
 *   H         1 <= H <= 8192 (any).
 *   weight    device, [H] of type w_dtype.
 *   bias      device, [H] of type w_dtype, or NULL (none).
 *   eps       >= 0 and finite.  A constant row with eps == 0 gives NaN.
 *   y         device, [M, H] contiguous, of type y_dtype.
 *   mean      device, float [M]; required with center, else must be NULL.
 *   rstd      device, float [M].
 * Every pointer is aligned to its element; x, y, weight and bias aligned to 16
 * bytes with H and ldx multiples of 8 take 16-byte accesses.
 */
int qhead_layer_norm(const void* x, int x_dtype, int64_t ldx, int64_t M, int64_t H,
                     const void* weight, const void* bias, int w_dtype, float eps, int center,
                     void* y, int y_dtype, float* mean, float* rstd, void* stream);

/*
 * The gradient of qhead_layer_norm: with xh = xc * rstd and g = dy * weight,
 *     dx = rstd * (g - mean(g) - xh * mean(g * xh))   (mean == NULL: no mean(g) term)
 *     dweight = sum_m dy * xh;  dbias = sum_m dy
 *   mean      the forward's, or NULL for the uncentred form.
 *   dy        device, [M, H] of type dy_dtype, row stride ldy >= H elements
 *             (qhead_bwd's float dh, for example).
 *   dx        device, [M, H] contiguous, of type x_dtype.
 *   dweight   device, float [H].
 *   dbias     device, float [H], or NULL.
 *   workspace device, >= qhead_layer_norm_bwd_workspace(M, H) bytes, 256-byte aligned.
 * M == 0 writes zeros to dweight and dbias.  Deterministic.
 */
size_t qhead_layer_norm_bwd_workspace(int64_t M, int64_t H);
int qhead_layer_norm_bwd(const void* x, int x_dtype, int64_t ldx, int64_t M, int64_t H,
                         const void* weight, int w_dtype, const float* mean, const float* rstd,
                         const void* dy, int dy_dtype, int64_t ldy, void* dx, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Distillation of the head against a teacher's top logits (no counterpart on
 * the pages, whose losses take one target per row).  Per active row, over its
 * valid entries k (ids[m, k] >= 0) and the whole vocabulary v, z as in
 * qhead_fwd:
 *     p_k  = softmax_k(tlogits[m, k] / temperature)
 *     lse  = log sum_v exp(z_v / temperature)
 *     loss = sum_k p_k * (log p_k - z_{ids[m, k]} / temperature + lse)
 *   h, M, mask  as for qhead_fwd (including |h| < 65504).
 *   ids       device, int32 [M, K]; a negative id is padding.  A token listed
 *             twice counts with the sum of its entries' p.
 *   tlogits   device, [M, K] of type t_dtype: logits or log-probabilities
 *             (only differences within a row matter); -inf is no mass.
 *   K         1 <= K <= 1024.
 *   temperature  > 0 and finite, a normal float (its reciprocal is one, too).
 *   loss, lse device, float [M]; inactive rows 0.  A row without a valid entry
 *             of finite logit has loss 0; one with an id >= V or a logit that
 *             is NaN or +inf has loss NaN.
 *   kept      device, float [M, qhead_distill_kept(head, M, K)], 32-byte
 *             aligned, for the backward: in the first K columns the exact fp32
 *             logits z of the valid entries (0 elsewhere), then the exact logits
 *             of the largest other vocab rows (those with a thousandth of the sum
 *             or more, up to 16, wherever they lie), and (as int32 bits, 0: none)
 *             those rows plus one; at M <= 16, or while M * V * 4 is at
 *             most 4 GiB, also the row's V logits, so that the backward need not
 *             form them again, with (q_v - p_v) * sech2 * 2^126 (-inf: 0) in
 *             place of those of the tokens whose exact ones are kept.  In a row
 *             without such others, +inf or -inf as the first's logit tells that
 *             its gradient is NaN or 0.
 *   workspace device, >= qhead_distill_fwd_workspace(head, M, K) bytes,
 *             256-byte aligned.
 * Up to 16 rows the weight-streaming kernel forms the logits, above them the
 * tensor-core kernel.  The listed tokens and the largest others enter lse with
 * their exact logits, the rest with the kernel's.
 */
int64_t qhead_distill_kept(const qhead_head* head, int64_t M, int64_t K); /* columns; -1: invalid */
size_t qhead_distill_fwd_workspace(const qhead_head* head, int64_t M, int64_t K);
int qhead_distill_fwd(const qhead_head* head, const void* h, int64_t M, const int32_t* ids,
                      const void* tlogits, int t_dtype, int64_t K, float temperature,
                      const uint8_t* mask, float* loss, float* lse, float* kept, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * The gradient of sum_m dloss[m] * loss[m] with respect to h, the head frozen:
 *     dh[m, :] = (dloss[m] / temperature) * sum_v (q_v - p_v) * sech2[m, v] * w[v, :]
 * with q_v = exp(z_v / temperature - lse).
 *   lse, kept the forward's, for the same arguments.
 *   dloss     device, float [M].
 *   dh        device, bf16 [M, H] (h's type; the contraction's operands carry
 *             fp16 precision), 16-byte aligned.  Inactive rows and rows with
 *             nothing to learn from are 0; rows of NaN loss are NaN.
 *   workspace device, >= qhead_distill_bwd_workspace(head, M, K) bytes,
 *             256-byte aligned.
 */
size_t qhead_distill_bwd_workspace(const qhead_head* head, int64_t M, int64_t K);
int qhead_distill_bwd(const qhead_head* head, const void* h, int64_t M, const int32_t* ids,
                      const void* tlogits, int t_dtype, int64_t K, float temperature,
                      const uint8_t* mask, const float* kept, const float* lse, const float* dloss,
                      void* dh, void* workspace, size_t workspace_bytes, void* stream);

/* 8-bit floats (e4m3: 4 exponent bits, 3 mantissa bits, finite up to 448), where a
 * call says that it takes them. */
#define QHEAD_E4M3 3

/* Activations of qhead_linear: z; max(z, 0); z / (1 + exp(-z)); z Phi(z) with the
 * normal distribution function; and its form with tanh,
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2. */
#define QHEAD_ACT_NONE 0
#define QHEAD_ACT_RELU 1
#define QHEAD_ACT_SILU 2
#define QHEAD_ACT_GELU 3
#define QHEAD_ACT_GELU_TANH 4

/*
 * Matrix product with bias, activation and residual in its epilogue (no
 * counterpart on the pages: the block between the norm and the head, such as a
 * draft head's h + silu(W h + b)):
 *     z[m, n] = x_scale[m] * w_scale[n] * sum_k x[m, k] * weight[n, k] + bias[n]
 *     y[m, n] = act(z[m, n]) + residual[m, n]
 * accumulated and finished in fp32, rounded once.  (The tensor cores' fp32 sums
 * truncate: a float32 y is off by 5e-7 of its norm, 3e-6 for positive fp16 operands; a
 * 16-bit one is formed in one sum, which stays far below its rounding up to some
 * 10^5 terms.)
 *   x         device, [M, K] of type dtype, row stride ldx >= K elements.
 *   weight    device, [N, K] of type dtype, row stride ldw >= K elements.
 *   dtype     QHEAD_BF16, QHEAD_F16, or QHEAD_E4M3 with x_scale and w_scale.
 *   K, N      >= 1 and at most 2^24.
 *   x_scale, w_scale  device, float [M] and [N] for QHEAD_E4M3, else NULL.
 *   bias      device, [N] of type bias_dtype, or NULL.
 *   residual  device, [M, N] of type res_dtype, row stride ldr >= N, or NULL.
 *   y         device, [M, N] contiguous, of type y_dtype (bias, residual and y:
 *             QHEAD_F16, QHEAD_BF16 or QHEAD_F32 each).
 *   pre       device, fp16 [M, N] contiguous, or NULL: z, for qhead_linear_bwd,
 *             saturated to the finite range (there act's derivative is what it
 *             is at the range's ends); where z is not 0 it keeps its sign, as the
 *             smallest fp16 at least (relu's derivative is that).
 *   workspace device, >= qhead_linear_workspace(...) bytes, 256-byte aligned
 *             (may be NULL when that is 0).
 * Every pointer is aligned to its elements.  x and weight with 16-byte aligned
 * starts and row strides of whole 16 bytes are read where they lie; others are
 * first copied to the workspace.  M == 0 returns QHEAD_OK.  A kernel wait that
 * expires (see above) makes the outputs that depend on it NaN.
 */
size_t qhead_linear_workspace(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K,
                              const void* weight, int64_t ldw, int64_t N);
int qhead_linear(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K, const void* weight,
                 int64_t ldw, int64_t N, const float* x_scale, const float* w_scale,
                 const void* bias, int bias_dtype, int act, const void* residual, int res_dtype,
                 int64_t ldr, void* y, int y_dtype, void* pre, void* workspace,
                 size_t workspace_bytes, void* stream);

/*
 * The gradient of qhead_linear (the residual's is dy itself):
 *     dz = dy * act'(z);  dx = dz * weight;  dweight = dz^T * x;  dbias = sum_m dz
 *   dtype     QHEAD_BF16 or QHEAD_F16: x, weight and the outputs.  dz is rounded
 *             to it as an operand of the two products (not for dbias), whatever dy's
 *             type: beside fp16 operands what is below 2^-25 is lost and what is
 *             above 65504 infinite, as in a dy of fp16.
 *   dy        device, [M, N] of type dy_dtype (any of the three), row stride ldy >= N.
 *   pre       the forward's; may be NULL when act is QHEAD_ACT_NONE.
 *   dx        device, [M, K] contiguous, or NULL (not wanted).
 *   dweight   device, [N, K] contiguous, or NULL.
 *   dbias     device, [N], or NULL.
 *   workspace device, >= qhead_linear_bwd_workspace(...) bytes, 256-byte aligned.
 * M == 0 writes zeros to dweight and dbias.  Deterministic.
 * qhead_linear_bwd_dbias: the same with a type of its own for dbias (QHEAD_F16,
 * QHEAD_BF16 or QHEAD_F32: the bias's, such as float32 beside 16-bit operands), to
 * which the fp32 sum is rounded.
 */
size_t qhead_linear_bwd_workspace(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K,
                                  const void* weight, int64_t ldw, int64_t N);
int qhead_linear_bwd(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K,
                     const void* weight, int64_t ldw, int64_t N, const void* dy, int dy_dtype,
                     int64_t ldy, const void* pre, int act, void* dx, void* dweight, void* dbias,
                     void* workspace, size_t workspace_bytes, void* stream);
int qhead_linear_bwd_dbias(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K,
                           const void* weight, int64_t ldw, int64_t N, const void* dy, int dy_dtype,
                           int64_t ldy, const void* pre, int act, void* dx, void* dweight,
                           void* dbias, int dbias_dtype, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * A residual's addition and the norm behind it (no counterpart on the pages):
 *     t = x + residual;  total = t, rounded;  y = norm(t)
 * with qhead_layer_norm's norm, taken of the unrounded fp32 t.
 *   x         device, [M, H] of type x_dtype, row stride ldx >= H.
 *   residual  device, [M, H] of type res_dtype, row stride ldr >= H.
 *   total     device, [M, H] contiguous, of type res_dtype.
 *   M, H, weight, bias, w_dtype, eps, center, y, y_dtype, mean, rstd  as for
 *             qhead_layer_norm.
 */
int qhead_add_norm(const void* x, int x_dtype, int64_t ldx, const void* residual, int res_dtype,
                   int64_t ldr, int64_t M, int64_t H, const void* weight, const void* bias,
                   int w_dtype, float eps, int center, void* total, void* y, int y_dtype,
                   float* mean, float* rstd, void* stream);

/*
 * The same with an output in 8 bits, for qhead_linear's 8-bit operands:
 *     scale[m] = max_d |y[m, d]| / 448;  codes[m, d] = e4m3(y[m, d] / scale[m])
 * rounded to nearest.  (The maximum counts as 1e-30 at least; where y is NaN, so is
 * the code.)
 *   residual  NULL: t = x, and total must be NULL.
 *   codes     device, e4m3 [M, H] contiguous.
 *   scale     device, float [M].
 */
int qhead_norm_8bit(const void* x, int x_dtype, int64_t ldx, const void* residual, int res_dtype,
                    int64_t ldr, int64_t M, int64_t H, const void* weight, const void* bias,
                    int w_dtype, float eps, int center, void* total, void* codes, float* scale,
                    void* stream);

/*
 * The gradient of qhead_add_norm: dx (of x and of the residual alike) is
 * qhead_layer_norm_bwd's at total, plus what arrives at total itself.
 *   total     the forward's, of type t_dtype (as rounded: the norm's gradient is
 *             taken there, with the forward's mean and rstd).
 *   dtotal    device, [M, H] of type t_dtype, row stride ldd >= H, or NULL (none).
 *   dx        device, [M, H] contiguous, of type t_dtype.
 *   workspace >= qhead_layer_norm_bwd_workspace(M, H) bytes; the rest as there.
 */
int qhead_add_norm_bwd(const void* total, int t_dtype, int64_t ldt, int64_t M, int64_t H,
                       const void* weight, int w_dtype, const float* mean, const float* rstd,
                       const void* dy, int dy_dtype, int64_t ldy, const void* dtotal, int64_t ldd,
                       void* dx, float* dweight, float* dbias, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * The global norm of many gradient tensors, and clipping (no counterpart on the
 * pages):
 *     norm = sqrt(sum over tensors and elements of g^2)
 *     out  = g * min(1, max_norm / (norm + 1e-6))
 *   tensors, sizes, dtypes  HOST arrays of count entries, read during the call:
 *             device address, elements (>= 0) and type of each (contiguous) tensor.
 *   count     >= 0 (0: the norm is 0).
 *   norm      device, float.
 *   max_norm  > 0 and finite.
 *   out, out_dtypes  HOST arrays: where each scaled tensor goes and its type; or
 *             both NULL: in place (then nothing is written if norm is within
 *             max_norm).  An entry of out may be its own tensor, with the same
 *             type; apart from that no output may overlap a tensor or another output.
 *   workspace device, >= qhead_grad_norm_workspace(count) bytes, 256-byte aligned.
 * A norm that is inf or NaN scales by 0 or NaN as the formula says: look at norm
 * before the step is taken.  Squares that fp32 cannot hold are summed in fp64.
 * Deterministic.
 */
size_t qhead_grad_norm_workspace(int64_t count);
int qhead_grad_norm(const void* const* tensors, const int64_t* sizes, const int* dtypes,
                    int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                    void* stream);
int qhead_clip_grads(void* const* tensors, const int64_t* sizes, const int* dtypes, int64_t count,
                     float max_norm, void* const* out, const int* out_dtypes, float* norm,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Message for the last error on the calling thread ("" if none).  The
 * pointer stays valid until the thread's next qhead_* call. */
const char* qhead_last_error(void);

/*
 * Instrumentation (no counterpart on the pages): arm a one-shot hook on the
 * calling thread.  The thread's next forward or backward call (qhead_fwd,
 * qhead_verify, qhead_fwd_noalloc, qhead_fwd_blockmax, qhead_distill_fwd,
 * qhead_bwd and the other backward entry points of the head) records the CUDA event `start` on its stream
 * immediately before its head kernel (the vocab-streaming contraction that
 * dominates the call; for a backward on the tensor-core path, the chain of
 * its per-chunk kernels) and `stop` immediately after it, then disarms the
 * hook.  A call rejected before it launches anything disarms it too.  start and stop are
 * cudaEvent_t handles passed as void*; passing NULL for both disarms.
 */
void qhead_time_next_head_kernel(void* start, void* stop);

/*
 * Test instrumentation (no counterpart on the pages): arm a one-shot switch
 * on the calling thread.  The thread's next forward or backward call (the
 * entry points listed for qhead_time_next_head_kernel, qhead_linear and
 * qhead_linear_bwd) launches its pipelined kernel with the TMA producer issuing no loads,
 * so the consumers' bounded waits expire and the call ends as described under
 * "Kernel time limits" (about 2 s later, without a fault).  armed = 0
 * disarms.  Exists so that the time-limit path can be
 * tested.
 */
void qhead_test_stall_next_call(int armed);

/* Library version string, e.g. "qhead 0.1.0 sm_103a". */
const char* qhead_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QHEAD_H */
