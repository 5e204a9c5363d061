/*
 * littlebit_train.h -- C ABI of the operators around the LittleBit layers in
 * quantisation-aware training (B200, sm_100a).
 *
 * littlebit_backward.h carries gradients through a layer; a training step also
 * needs both ends of the model and an update of the latent factors:
 *   - the token embedding and its gradient,
 *   - the softmax cross entropy of the last hidden states against the
 *     vocabulary matrix, with the gradients of both,
 *   - the orthogonalised update of a latent factor (the Newton-Schulz form of
 *     the Muon optimiser) from its gradient dU or dV.
 *
 * Conventions are those of littlebit.h: device pointers unless stated, arrays
 * of pointers are HOST arrays of device pointers, row-major dense matrices,
 * `stream` is a cudaStream_t passed as void*, every check of the arguments is
 * made before anything is enqueued (LB_ERR_CUDA and LB_ERR_OOM can come later and
 * leave the outputs unspecified), nothing synchronises the host unless it says
 * so.  No call here allocates device memory or keeps anything between calls: scratch
 * is the `workspace` argument, 256-byte aligned and at least as large as the
 * matching *_workspace_bytes call says (host only; 0 also for sizes that the
 * operator refuses; NULL will do where 0 bytes are needed); its contents need
 * not be initialised and mean nothing afterwards.  Calls that use different
 * workspaces and outputs may overlap on the device (streams, captured graphs);
 * calls that share one must be ordered.  All calls can be captured into a CUDA
 * graph.
 * Outputs must not overlap inputs.  The same call gives the same bits every time.
 */
#ifndef LITTLEBIT_TRAIN_H
#define LITTLEBIT_TRAIN_H

#include "littlebit.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators that take more than one. */
typedef enum lb_dtype {
    LB_F32 = 0,   /* IEEE binary32 */
    LB_BF16 = 1   /* bfloat16      */
} lb_dtype;

/*
 * Token embedding: out[m] = scale * table[id_m], rounded once to the output type.
 *   ids    int64 [M]; an id outside 0 .. V-1 (such as a padding -1) gives a row of zeros
 *   table  table_dtype [V][D]        out  out_dtype [M][D]      (lb_dtype values)
 * Arrays need the alignment of their elements (16 bytes and D a multiple of 8
 * are fastest).  V, D >= 1; M = 0 is a valid empty call.
 * Errors: LB_ERR_INVALID_ARG, LB_ERR_UNSUPPORTED (M >= 2^31, D > 2^25), LB_ERR_CUDA.
 */
LB_API lb_status lb_embedding_forward(const int64_t *ids, int64_t M, const void *table, int table_dtype, int V, int D,
                                      float scale, void *out, int out_dtype, void *stream);

/*
 * Its gradient: dtable[v] = scale * (sum of dout[m] over the m with id_m = v),
 * zeros for a row that no id names; the whole of dtable is overwritten.  The
 * sums are float32, by increasing m within groups of the sorted tokens (a
 * fixed order: the same bits every time), times scale, rounded once.
 *   dout  dout_dtype [M][D]          dtable  dtable_dtype [V][D]
 * An id outside 0 .. V-1 adds nothing.  M = 0 writes zeros.
 * Errors: LB_ERR_INVALID_ARG, LB_ERR_UNSUPPORTED (M >= 2^31, D > 2^23), LB_ERR_CUDA.
 */
LB_API size_t lb_embedding_backward_workspace_bytes(int64_t M, int V, int D);
LB_API lb_status lb_embedding_backward(const int64_t *ids, int64_t M, const void *dout, int dout_dtype, int V, int D,
                                       float scale, void *dtable, int dtable_dtype, void *workspace,
                                       size_t workspace_bytes, void *stream);

/*
 * Softmax cross entropy against a vocabulary matrix, without the logits:
 *     z = H W^T [M x V],  lse_m = log sum_v exp z_mv,  loss_m = lse_m - z_m,label(m)
 *
 *   H       bfloat16 [M][D], hidden states        W       bfloat16 [V][D], vocabulary matrix
 *   labels  int64 [M]; a label outside 0 .. V-1 (such as -100) marks a row that does not count: its loss is 0
 *   loss    float32 [M]                           lse     float32 [M] (every row)
 * H and W 16-byte aligned, D a multiple of 8, D, V >= 1; M = 0 is a valid
 * empty call.  Products accumulate in float32 on the tensor cores; the maximum
 * and sum of the softmax are float32.  A row with a NaN or an infinite logit
 * has lse and loss NaN (an infinity below every other logit counts as weight 0).
 * Errors: LB_ERR_INVALID_ARG (null, misaligned, bad size, workspace too
 * small), LB_ERR_UNSUPPORTED (D not a multiple of 8; M or V above 2^28, D above
 * 2^20, or more than 2^28 tiles of 256 x 256 in a product), LB_ERR_CUDA.
 */
LB_API size_t lb_cross_entropy_forward_workspace_bytes(int M, int D, int V);
LB_API lb_status lb_cross_entropy_forward(const uint16_t *H, const uint16_t *W, const int64_t *labels, int M, int D,
                                          int V, float *loss, float *lse, void *workspace, size_t workspace_bytes,
                                          void *stream);

/*
 * The same loss together with its gradients, for row weights w (the derivative
 * of the training objective by each row's loss, 1 / count for a mean):
 *     G = diag(w) (softmax(z) - onehot(labels)),   dH = G W,   dW = G^T H
 * A row that does not count has G = 0, whatever its hidden state holds.
 *
 *   weight  float32 [M]       loss  float32 [M]
 *   dH      bfloat16 [M][D]   dW    bfloat16 [V][D], or NULL for a frozen vocabulary matrix; both are overwritten
 *   rows    rows taken at a time (0: 8192; more than 32768: 32768).  The scratch holds 16 bits per
 *           logit of one such piece, never of all M rows when M is larger;
 *           with more than one piece dW is summed over them in float32.
 * Softmax entries go through binary16 relative to the largest of their 128
 * neighbours (v / 128): right to 2^-11, but 0 below 2^-40 of that one.
 * G is rounded to bfloat16 once, as an operand of the two products (dH is made
 * good for the rounding of the label's entry); they accumulate in float32 and
 * dH, dW are rounded once.  All else as above; rows
 * must be >= 0; with M = 0 only dW is written (zeros).
 */
LB_API size_t lb_cross_entropy_gradient_workspace_bytes(int M, int D, int V, int with_dW, int rows);
LB_API lb_status lb_cross_entropy_gradient(const uint16_t *H, const uint16_t *W, const int64_t *labels,
                                           const float *weight, int M, int D, int V, int rows, float *loss,
                                           uint16_t *dH, uint16_t *dW, void *workspace, size_t workspace_bytes,
                                           void *stream);

/*
 * Orthogonalised updates, for the gradients of latent factors (dU, dV of
 * lb_layer_backward, or their running mean): for each matrix, by the
 * Newton-Schulz iteration of the Muon optimiser,
 *     X = G / (|G|_F + eps);   `steps` times:
 *     X <- a X + b (X X^T) X + c (X X^T)^2 X,   (a, b, c) = (3.4445, -4.7750, 2.0315)
 * which carries every singular value that is not tiny close to 1.
 *
 *   G      [n] pointers to dtype [rows_i][cols_i] (lb_dtype), aligned to their elements
 *   rows, cols   HOST int [n], >= 1; min(rows, cols) <= LB_MAX_RANK
 *   steps  1 .. 10 (5 is usual);  eps >= 0 (1e-7 is usual)
 *   O      [n] pointers to bfloat16 [rows_i][cols_i], overwritten
 * n = 0 is a valid empty call; all matrices of a call share its launches, so
 * pass a block's latents together.  (They also share the GPU: how the sum over a
 * long axis is cut follows from the whole set, so a matrix's last float32 bits
 * may depend on what else is in the call.)  Float32 in effect: products take operands
 * of 22 bits and accumulate in float32, the result is rounded once.  (The
 * iteration runs on G^T G / |G|_F^2: a singular value s |G|_F has there a
 * relative error of about 2^-22 / s^2, which shows for s < 1e-3 after more than
 * five steps, when such values too come close to 1.)  A matrix of zeros gives
 * zeros; one with a NaN or an infinity gives NaN throughout, and touches no
 * other matrix.
 * Errors: LB_ERR_INVALID_ARG, LB_ERR_UNSUPPORTED (steps > 10, min(rows, cols)
 * > LB_MAX_RANK, a side above 2^24), LB_ERR_OOM (host memory), LB_ERR_CUDA.
 */
LB_API size_t lb_orthogonalise_workspace_bytes(const int *rows, const int *cols, int n, int dtype);
LB_API lb_status lb_orthogonalise(const void *const *G, int dtype, const int *rows, const int *cols, int n, int steps,
                                  float eps, uint16_t *const *O, void *workspace, size_t workspace_bytes,
                                  void *stream);

/* Device-side status of the tensor-core kernels of this header on the current
 * device: synchronises `stream`, returns LB_ERR_TIMEOUT if a bounded wait gave
 * up since the last check (the outputs of that call are unspecified) and
 * clears it.  Not to be called while a stream is being captured. */
LB_API lb_status lb_train_status(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LITTLEBIT_TRAIN_H */
