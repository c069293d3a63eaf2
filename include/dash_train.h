/*
 * dash_train.h -- C ABI of the operators around the attention in a training step whose
 * results are reproducible: token embedding and its gradient, the norm and rotation of
 * queries and keys, the cross entropy of a large vocabulary with its gradient, and gradient
 * clipping. Built into the same library as dash_attn.h, whose status codes they return.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every sum over tokens, rows or parameters is split and joined in an order that depends
 *   on the arguments alone (no floating-point atomics, no dependence on the SM count):
 *   equal arguments give equal bits, run to run and GPU to GPU of the same model.
 * - All device pointers are owned by the caller and stay valid until the work queued on
 *   `stream` has finished. Nothing is allocated, and nothing is kept between calls.
 * - Calls are asynchronous on `stream`, may be captured into a graph, and return argument
 *   errors synchronously with nothing queued. Workspaces are 256-byte aligned, need no
 *   initialisation, and must not be shared by calls that may overlap.
 * - Indexes read on the device (token ids, positions, targets) are checked there: one out
 *   of range is never used as an address. The call's status -- dash_attn_get_status on the
 *   workspace, or the optional `status` word of a call without one -- then reads
 *   DASH_ERR_BOUNDS, and what the row yields is said at the call.
 * - Index arrays are int32 or int64 (`id_bits` 32 or 64). Sums are held in fp32 (fp64 where
 *   said) and rounded once, to nearest even, when a result is stored.
 */
#ifndef DASH_TRAIN_H
#define DASH_TRAIN_H

#include "dash_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators that take more than bf16. */
typedef enum { DASH_BF16 = 0, DASH_FP16 = 1, DASH_FP32 = 2 } dash_dtype_t;

/* ---- Token embedding ------------------------------------------------------------------ */

/*
 * out[t] = scale * table[ids[t]], rounded once (copied when scale is 1).
 *   table : [V, D] of `dtype`, rows ld_table elements apart (read)
 *   ids   : [T] int32 or int64 (read)
 *   out   : [T, D] of `dtype`, rows ld_out elements apart (written)
 *   status: optional device int32 (NULL = none), cleared by the call; an id outside [0, V)
 *           makes its output row NaN and sets it to DASH_ERR_BOUNDS
 * T >= 0, V >= 1, 1 <= D <= 2^20, T and V below 2^31 - 256, leading dimensions not below D;
 * any element alignment (rows that are whole 16-byte pieces are moved as such).
 */
dash_status_t dash_embed_fwd(const void* table, const void* ids, void* out, int* status,
                             long long T, long long V, int D, long long ld_table, long long ld_out,
                             float scale, int dtype, int id_bits, cudaStream_t stream);

/*
 * dtable[v] = scale * sum over the tokens with ids[t] = v of dout[t]  (zero rows for ids that
 * do not occur); with accumulate != 0 the sum is added to what dtable holds, with one
 * rounding, and rows of other ids are left alone (several micro-batches; a table tied to the
 * output embedding).
 * The tokens are sorted by id, stably, and an id's rows are summed in fp32 in that order, in
 * runs of 32 sorted places that are then joined in order.
 *   dout  : [T, D] of dout_dtype, rows ld_dout elements apart (read)
 *   dtable: [V, D] contiguous, of dtable_dtype: dout's type or DASH_FP32 (written)
 *   padding_idx : an id whose tokens are left out, or -1
 *   workspace : dash_embed_bwd_workspace_size(T, V, D) bytes
 * An id outside [0, V) contributes nothing and sets the workspace's status to
 * DASH_ERR_BOUNDS. Sizes and alignment as above.
 */
size_t dash_embed_bwd_workspace_size(long long T, long long V, int D);
dash_status_t dash_embed_bwd(const void* dout, const void* ids, void* dtable, void* workspace,
                             size_t workspace_bytes, long long T, long long V, int D,
                             long long ld_dout, float scale, long long padding_idx, int accumulate,
                             int dout_dtype, int dtable_dtype, int id_bits, cudaStream_t stream);

/* ---- Norm and rotation of queries and keys -------------------------------------------- */

/*
 * Per token and head: y = x / sqrt(mean(x^2) + eps) * w over the head's D values, then the
 * rotation of y's first R values by the token's angles: pair (a, b) becomes
 * (a cos - b sin, b cos + a sin); pair i is (i, i + R/2), or (2i, 2i + 1) with interleaved
 * != 0. The other D - R values pass. Queries and keys in one launch, rounded once.
 *   q, k     : [B, S, Hq, D], [B, S, Hk, D] of `dtype`, D contiguous, with element strides
 *              {batch, token, head} in q_strides and k_strides: views of a fused projection
 *              or of [B, H, S, D] are read in place (multiples of 8)
 *   wq, wk   : fp32 [D], or NULL for ones
 *   cos, sin : fp32 [P, R / 2], contiguous; row p holds the angles of position p
 *   positions: [B, S] int32 or int64, batches pos_stride elements apart (0: one row for
 *              all), or NULL for 0 .. S - 1
 *   q_out, k_out : contiguous [B, S, Hq, D], [B, S, Hk, D], as dash_attn_fwd reads them
 *              (written; must not overlap the inputs)
 *   status   : as for dash_embed_fwd; a position outside [0, P) gives NaN rows
 * D a multiple of 8 up to 256; R even, 0 <= R <= D; eps >= 0; B, S >= 0; Hq, Hk >= 0;
 * B * S * (Hq + Hk) below 2^31 - 256. Pointers 16-byte aligned (positions: as elements).
 */
dash_status_t dash_qk_norm_rope_fwd(const void* q, const void* k, const float* wq, const float* wk,
                                    const float* cos, const float* sin, const void* positions,
                                    void* q_out, void* k_out, int* status, int B, int S, int Hq,
                                    int Hk, int D, int R, long long P, const long long* q_strides,
                                    const long long* k_strides, long long pos_stride, float eps,
                                    int interleaved, int dtype, int id_bits, cudaStream_t stream);

/*
 * Gradients of the above: with d = the rotation's transpose applied to d(out) and r =
 * 1 / sqrt(mean(x^2) + eps), dw = sum over rows of d x r and
 * dx = r (w d - x r mean(w d x r)). r is recomputed from x, nothing is saved by the forward.
 *   dq_out, dk_out : contiguous [B, S, Hq, D], [B, S, Hk, D] (read)
 *   dq, dk   : strided as dq_strides and dk_strides say (written), so that they may be the
 *              parts of a fused projection's gradient; a stride of zero over more than one
 *              element is refused here (inputs may have it: heads or batches that are shared)
 *   dwq, dwk : fp32 [D] (written; NULL: not wanted)
 *   workspace: dash_qk_norm_rope_bwd_workspace_size(B, S, Hq, Hk, D) bytes
 * A position out of range gives NaN rows in dq and dk (and NaN in dwq, dwk) and the status
 * DASH_ERR_BOUNDS.
 */
size_t dash_qk_norm_rope_bwd_workspace_size(int B, int S, int Hq, int Hk, int D);
dash_status_t dash_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q,
                                    const void* k, const float* wq, const float* wk,
                                    const float* cos, const float* sin, const void* positions,
                                    void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                                    size_t workspace_bytes, int B, int S, int Hq, int Hk, int D,
                                    int R, long long P, const long long* q_strides,
                                    const long long* k_strides, const long long* dq_strides,
                                    const long long* dk_strides, long long pos_stride, float eps,
                                    int interleaved, int dtype, int id_bits, cudaStream_t stream);

/* ---- Gradient norm and clipping --------------------------------------------------------- */

/* One tensor of a clipping plan: numel elements of `dtype` at `grad`; its clipped values go
 * to `out`, which is `grad` itself or a buffer that overlaps no tensor of the plan. */
typedef struct {
  const void* grad;
  void* out;
  long long numel;
  int dtype;                 /* dash_dtype_t */
} dash_clip_tensor_t;

/*
 * A plan holds the table of a list of tensors in a caller's device buffer, so that a step's
 * call moves no host memory. dash_grad_clip_plan copies the table (it waits for `stream`);
 * the plan stays valid while the tensors stay where they are. numel >= 0 each, n >= 1; the
 * elements need only their own alignment. The plan also holds the call's partial sums, so
 * calls on one plan must not overlap.
 */
size_t dash_grad_clip_plan_size(const dash_clip_tensor_t* tensors, int n);
dash_status_t dash_grad_clip_plan(const dash_clip_tensor_t* tensors, int n, void* plan,
                                  size_t plan_bytes, cudaStream_t stream);

/*
 * *norm = sqrt(sum of all elements squared), and out = grad * (max_norm / *norm) for every
 * tensor when *norm > max_norm, out = grad otherwise (nothing is written then where out is
 * grad). Squares are summed in fp32 over at most 64 elements of a tensor, these sums in fp64;
 * where squares would overflow or vanish in fp32 the elements are rescaled by a power of two
 * first. When the norm is not finite in fp32 *norm says so and the values are passed
 * unscaled.
 *   plan : from dash_grad_clip_plan, on this device, of plan_bytes (dash_grad_clip_plan_size);
 *          something else gives the norm NaN and touches no tensor
 *   norm : device fp32 (written)
 * max_norm >= 0 (may be infinite: the norm alone, with copies where out is not grad).
 */
dash_status_t dash_grad_clip(void* plan, size_t plan_bytes, float max_norm, float* norm,
                             cudaStream_t stream);

/* ---- Softmax cross entropy from hidden states --------------------------------------- */

/*
 * loss[t] = lse[t] - z[t][y_t],  lse[t] = log sum_v exp(z[t][v]),  z = scale * X W^T,
 * without storing the logits z. A row whose target is ignore_index has loss 0 (its lse is
 * computed all the same); a target outside [0, V) that is not ignore_index gives loss NaN
 * and the status DASH_ERR_BOUNDS.
 *   x       : bf16 [T, D], rows ldx elements apart (read)
 *   w       : bf16 [V, D], rows ldw elements apart (read)
 *   targets : [T] int32 or int64 (read)
 *   loss    : fp32 [T] (written)        lse : fp32 [T] (written)
 *   workspace : dash_linear_xent_workspace_size(T, V, D) bytes
 * T >= 0, V >= 1, D a positive multiple of 8, ldx and ldw multiples of 8 not below D,
 * scale > 0; x, w, dx and dw 16-byte aligned, the others as their elements. T * D, V * D up to
 * 2^40; T, V below 2^31 - 256.
 * Returns DASH_ERR_UNSUPPORTED for other sizes. bf16 only, as the attention: the gradient
 * passes G below through the tensor cores in the operands' type, and fp16 would lose its
 * small probabilities.
 */
size_t dash_linear_xent_workspace_size(long long T, long long V, int D);
dash_status_t dash_linear_xent_fwd(const void* x, const void* w, const void* targets, float* loss,
                                   float* lse, void* workspace, size_t workspace_bytes, long long T,
                                   long long V, int D, long long ldx, long long ldw, float scale,
                                   long long ignore_index, int id_bits, cudaStream_t stream);

/*
 * Gradient of sum_t dloss[t] * loss[t]:
 *   G[t][v] = scale * dloss[t] * (exp(z[t][v] - lse[t]) - [v = y_t])  (0 for ignored rows),
 *   dX = G W,   dW = G^T X.
 * The logits are recomputed piece by piece of the vocabulary; a piece of G is held in the
 * workspace in bf16, as the tensor cores need it, the products are summed in fp32. G is rounded
 * no more than the result that it goes into: by at most 2^-8 of each entry for dx and a bf16 dw;
 * by 2^-16 (two terms) for an fp32 dw, whose product takes twice as long for it, and for both
 * results up to 128 tokens.
 *   lse     : fp32 [T] from dash_linear_xent_fwd (read)
 *   dloss   : fp32 [T] (read)
 *   dx      : bf16 [T, D] contiguous (written)
 *   dw      : [V, D] contiguous, bf16 or fp32 by dw_dtype (written; with accumulate != 0
 *             the gradient is added to what it holds, with one rounding)
 *   workspace : the same size as the forward's
 * A target out of range is treated as ignored and sets the status DASH_ERR_BOUNDS.
 * Other arguments and errors as for the forward.
 */
dash_status_t dash_linear_xent_bwd(const void* x, const void* w, const void* targets,
                                   const float* lse, const float* dloss, void* dx, void* dw,
                                   void* workspace, size_t workspace_bytes, long long T,
                                   long long V, int D, long long ldx, long long ldw, float scale,
                                   long long ignore_index, int id_bits, int dw_dtype,
                                   int accumulate, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DASH_TRAIN_H */
