/*
 * hqq_layers.h -- C ABI of libhqq_layers.so: the blocks around the quantized
 * Linear layer that a model is trained, evaluated and served with on MI355X
 * (gfx950): the gated feed-forward block, the softmax cross entropy of a
 * quantized output head, and the backward passes through frozen quantized
 * weights.  It stands beside hqq_linear (hqq.h), whose formats, conventions
 * and status codes it shares.
 *
 * Weights.  A weight W [N, K] is in the axis = 1 layout of hqq.h: packed codes
 * (nbits in {1, 2, 4, 8}), fp32 scale and zero [N, K / group_size], group_size
 * in {8, ..., 256} dividing K, K a multiple of 32.  Its value W_hat is exactly
 * what hqq_dequantize_ex writes for the call's dtype (the fp16 or bf16 rounding
 * of the fp32 quotient (code - zero) / scale).  The codes, scales and zeros are
 * constants here: gradients go to the activations.
 *
 * Numbers.  Activations and their gradients are fp16 or bf16 (dtype); products
 * of 16-bit values are exact and summed in fp32; what each call rounds to 16
 * bits besides its 16-bit outputs is said there.
 *
 * Conventions of hqq.h hold: device pointers, 16-byte aligned unless said
 * otherwise; all arguments are checked on the host before anything is enqueued;
 * calls only enqueue work on `stream` of the current device; nothing is
 * allocated and no state is kept.  Inputs and outputs are contiguous,
 * row-major; outputs and the bytes of workspace that the call uses must not overlap
 * its inputs, the weights' arrays among them, or one another (HQQ_EINVAL_PTR).
 * Scales are finite and not 0, as hqq_quantize writes them.
 *
 * Workspace.  Each call takes a device workspace of at least the bytes that its
 * *_workspace function returns for the same sizes (HQQ_EWORKSPACE if smaller; 0
 * bytes need no pointer).  Nothing in it has to be set before a call or kept
 * after it, so calls that follow each other on one stream may share one; calls
 * that may run at the same time (two streams, two captured graphs) may not.
 *
 * Routes.  Few rows are multiplied straight from the packed codes; for more,
 * W_hat is unpacked into the workspace and a tiled product runs on it.  The
 * choice goes by sizes and format, and both stay within the same bounds.  The
 * environment variable HQQ_LAYERS_PATH=codes or =tiled, read at each call and by
 * the *_workspace functions, forces one (the codes up to 256 rows).
 */
#ifndef HQQ_LAYERS_H
#define HQQ_LAYERS_H

#include "hqq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HQQ_EINVAL_ACT (-10)  /* act not one of HQQ_ACT_*                             */
#define HQQ_EWORKSPACE (-11)  /* workspace smaller than the *_workspace function says */

/* Activations of the gated block. */
#define HQQ_ACT_SILU 0      /* g / (1 + exp(-g))                                       */
#define HQQ_ACT_GELU 1      /* g * (1 + erf(g / sqrt 2)) / 2                           */
#define HQQ_ACT_GELU_TANH 2 /* g * (1 + tanh(sqrt(2 / pi) * (g + 0.044715 g^3))) / 2   */

/* A quantized weight's arrays (read only). */
typedef struct hqq_weight {
    const uint32_t *packed;
    const float *scale;
    const float *zero;
} hqq_weight;

/* Gated feed-forward block: Y = act(X . Wg_hat^T) * (X . Wu_hat^T).
 *   X     [M, K], gate and up: weights [N, K] of one format, Y [M, N]
 * Both projections stay in fp32; each output is rounded once.
 * Limits of all calls (HQQ_EINVAL_SHAPE): M, N >= 1; M <= 2^20; K <= 2^17;
 * N <= 2^22; M * N <= 2^40; the codes and the meta of a weight each below 2^31
 * bytes. */
HQQ_API int64_t hqq_linear_gated_workspace(int64_t M, int64_t K, int64_t N, int nbits, int group_size);
HQQ_API int hqq_linear_gated(const uint16_t *X, int64_t M, int64_t K, const hqq_weight *gate,
                             const hqq_weight *up, int64_t N, int nbits, int group_size, int dtype,
                             int act, uint16_t *Y, void *workspace, int64_t workspace_bytes,
                             void *stream);

/* The block's backward pass: with G = X . Wg_hat^T and U = X . Wu_hat^T
 * computed anew (they are not kept by the forward pass),
 *   dG = dY * U * act'(G),  dU = dY * act(G),  dX = dG . Wg_hat + dU . Wu_hat.
 *   dY [M, N] read, dX [M, K] written
 * dG and dU are formed in fp32 and rounded once to the dtype for the second
 * pair of products (fp16: times a power of two chosen per row from max |dY|,
 * sum |X| and the weights' largest |W_hat|, so that neither small gradients nor
 * small projections lose precision, and nothing overflows). */
HQQ_API int64_t hqq_linear_gated_backward_workspace(int64_t M, int64_t K, int64_t N, int nbits,
                                                    int group_size);
HQQ_API int hqq_linear_gated_backward(const uint16_t *dY, const uint16_t *X, int64_t M, int64_t K,
                                      const hqq_weight *gate, const hqq_weight *up, int64_t N,
                                      int nbits, int group_size, int dtype, int act, uint16_t *dX,
                                      void *workspace, int64_t workspace_bytes, void *stream);

/* One weight of hqq_linear_batch_backward: its arrays, its output width N and
 * the gradient dY [M, N] of its output (read only). */
typedef struct hqq_linear_grad {
    const uint32_t *packed;
    const float *scale;
    const float *zero;
    int64_t N;
    const uint16_t *dY;
} hqq_linear_grad;

/* The backward pass of hqq_linear_batch: dX = sum_i dY_i . W_hat_i for count
 * weights [N_i, K] of one format that read the same X [M, K] (count = 1: the
 * backward pass of hqq_linear).  The sum over all weights and outputs is one
 * fp32 sum, rounded once.
 *   ws  HOST array of count descriptors, 1 <= count <= HQQ_MAX_GRADS; their N,
 *       each rounded up to 64, add up to at most 2^23
 *   n   (workspace function) HOST array of the count widths N_i */
#define HQQ_MAX_GRADS 16
HQQ_API int64_t hqq_linear_batch_backward_workspace(int64_t M, int64_t K, const int64_t *n, int count,
                                                    int nbits, int group_size);
HQQ_API int hqq_linear_batch_backward(const hqq_linear_grad *ws, int count, int64_t M, int64_t K,
                                      int nbits, int group_size, int dtype, uint16_t *dX,
                                      void *workspace, int64_t workspace_bytes, void *stream);

/* Softmax cross entropy of a quantized output head W [N, K] over N classes:
 * with logits l = X . W_hat^T in fp32 (formed a piece of the vocabulary at a
 * time, never kept),
 *   lse[m]  = log sum_n exp(l[m][n])
 *   loss[m] = lse[m] - l[m][targets[m]], evaluated as log(1 + the others'
 *             share), so that a confident row's small loss keeps its precision
 * A row whose target lies outside [0, N) (-100, say) is ignored: loss 0; its
 * lse is still written.
 * Infinite and NaN logits (an input that is not finite) give what these formulas
 * give in IEEE arithmetic: lse +inf beside a +inf logit, -inf where all are -inf.
 *   targets int64 [M] (8-byte aligned), loss and lse fp32 [M] (4-byte aligned) */
HQQ_API int64_t hqq_linear_cross_entropy_workspace(int64_t M, int64_t K, int64_t N, int nbits,
                                                   int group_size);
HQQ_API int hqq_linear_cross_entropy(const uint16_t *X, int64_t M, int64_t K, const hqq_weight *head,
                                     int64_t N, int nbits, int group_size, int dtype,
                                     const int64_t *targets, float *loss, float *lse, void *workspace,
                                     int64_t workspace_bytes, void *stream);

/* Its backward pass: dX[m] = dloss[m] * sum_n (exp(l[m][n] - lse[m]) - [n =
 * targets[m]]) W_hat[n], with the logits computed anew and lse the forward
 * pass's.  Ignored rows get 0, whatever their dloss, lse and X hold.  The
 * differences are formed in fp32 and rounded once to the dtype (fp16: as
 * multiples of 2^-15 with fp16's own exponent below) for the second product.
 *   dloss and lse fp32 [M] (4-byte aligned), dX [M, K] written */
HQQ_API int64_t hqq_linear_cross_entropy_backward_workspace(int64_t M, int64_t K, int64_t N, int nbits,
                                                            int group_size);
HQQ_API int hqq_linear_cross_entropy_backward(const float *dloss, const uint16_t *X, int64_t M,
                                              int64_t K, const hqq_weight *head, int64_t N, int nbits,
                                              int group_size, int dtype, const int64_t *targets,
                                              const float *lse, uint16_t *dX, void *workspace,
                                              int64_t workspace_bytes, void *stream);

/* Static description of a status code of this header or of hqq.h. */
HQQ_API const char *hqq_layers_strerror(int status);

#ifdef __cplusplus
}
#endif
#endif /* HQQ_LAYERS_H */
