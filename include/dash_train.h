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
 * scale > 0; x, w, dx and dw 16-byte aligned, the others as their elements. T * D, V * D up to 2^40; T, V below 2^31 - 256.
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
 * workspace in bf16 (its one rounding: half a unit in 2^-8 of each entry, as the tensor
 * cores need it), the products are summed in fp32.
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
