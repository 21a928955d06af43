/*
 * llm_int8_ffn.h - C ABI of the feed-forward operators of libllm_int8.so:
 * the int8 linear layer (llm_int8.h) with the work around it in its
 * epilogue, and the gradients that pass back through the frozen weight.
 *
 *   llm_int8_linear_epilogue  Y = act(Z + bias) + residual
 *   llm_int8_gated_linear     H = act(G) * U, [G | U] = Z + bias
 *   llm_int8_linear_backward  dX, and the gradient at the activation's input
 *   llm_int8_gated_backward   the same through the gated pair
 *
 * Z[t,n] = fl32(D * sW[n]) is what llm_int8_linear rounds to its fp16 Y; here it
 * stays fp32 through the epilogue, and each output is rounded to fp16 once.
 *
 * Gradients: outlier columns and codes are piecewise constant, so the
 * gradient is that of the dequantized product X . W'^T with
 * W'[n,k] = Wq[n,k] * sW[n] (the weight is frozen: it gets none).
 *
 * Conventions are those of llm_int8.h: dense row-major device memory, 16-byte
 * aligned, asynchronous and ordered on `stream` (of the current device, where all
 * memory lives), validated on the host before anything is launched, nothing
 * allocated, synchronized or read back, no mutable state in the library.
 * T, K, N as there; a gated pair has N = 2F rows.  Refused besides
 * (LI8_ERR_SHAPE): forward calls of ceil(T/256) * ceil(N/128) >= 2^23, backward
 * calls of N > 2^21 or T > 2^30.  T, N or F of 0 is an
 * empty call (dX is then zero where it has elements, and so is dbias).
 * Outputs and the workspace must not overlap inputs or one another, except for
 * a residual that is Y itself.  llm_int8_plan is about llm_int8_linear; the
 * calls here take its few-token paths for the same shapes
 * (llm_int8_ffn_plan.h says which kernels they run).
 * X and the weight must be finite.  A NaN of a bias or residual reaches the
 * outputs that it enters.  At Z = +inf (by its bias) every activation is +inf; at
 * -inf none keeps it, relu is 0 and the smooth ones are 0 times infinity, NaN.
 * A row of gradients that holds an infinity or NaN gives a dX row of infinities
 * and NaN (what a loss scaler looks for).  Results past fp16's range become
 * infinities.  Where pre holds such ones the slopes are those of its side (1 and
 * 0; none: 1); a pair's row may give infinities and NaN, as their products.
 */
#ifndef LLM_INT8_FFN_H
#define LLM_INT8_FFN_H

#include "llm_int8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum li8_act {
    LI8_ACT_NONE = 0,
    LI8_ACT_RELU = 1,
    LI8_ACT_SILU = 2,      /* z / (1 + exp(-z))                              */
    LI8_ACT_GELU = 3,      /* z P(z), P the normal distribution's integral   */
    LI8_ACT_GELU_TANH = 4  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
} li8_act;

/*
 * Y[T,N] = fp16(act(Z + bias) + residual).
 *   X, Wq, sW, threshold, workspace  as for llm_int8_linear (workspace of
 *              llm_int8_linear_workspace_bytes(T, K, N) bytes).
 *   bias       [N] fp16, or NULL.
 *   act        an li8_act.
 *   residual   [T,N] fp16, or NULL.  It may be Y itself (the sum is then
 *              formed in place), but must not overlap Y otherwise.
 *   Y          [T,N] fp16 out.
 *   pre        [T,N] fp16 out, or NULL: fp16(Z + bias), which
 *              llm_int8_linear_backward takes.
 */
li8_status llm_int8_linear_epilogue(const void *X, const int8_t *Wq, const float *sW,
                                    float threshold, int64_t T, int64_t K, int64_t N,
                                    const void *bias, int32_t act, const void *residual, void *Y,
                                    void *pre, void *workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/*
 * H[T,F] = fp16(act(G) * U), both projections in one product.
 *   Wq, sW     of the pair [2F,K]: the gate's F rows, then the up-projection's
 *              (int8_quantize_weight works row by row, so two quantized
 *              weights may simply be stored one after the other).
 *   bias       [2F] fp16, or NULL.
 *   H          [T,F] fp16 out.
 *   pre        [T,2F] fp16 out, or NULL: fp16 of [G | U], which
 *              llm_int8_gated_backward takes.
 *   workspace  llm_int8_linear_workspace_bytes(T, K, 2F) bytes.
 */
li8_status llm_int8_gated_linear(const void *X, const int8_t *Wq, const float *sW, float threshold,
                                 int64_t T, int64_t K, int64_t F, const void *bias, int32_t act,
                                 void *H, void *pre, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/*
 * Bytes of workspace for the gradients through a weight [N,K] (N = 2F for a
 * gated pair); 0 for an invalid or empty shape and where none is needed (NULL
 * is accepted then).
 */
size_t llm_int8_backward_workspace_bytes(int64_t T, int64_t K, int64_t N);

/*
 * dZ = dY * act'(pre),  dX[T,K] = fp16(dZ . W'),  dbias[n] = sum_t dZ[t,n].
 *   dY        [T,N] fp16 (the residual's gradient is dY itself).
 *   pre       [T,N] fp16, as llm_int8_linear_epilogue stored it; NULL with
 *             LI8_ACT_NONE, where it is not read.
 *   dX        [T,K] fp16 out.
 *   grad_pre  [T,N] fp16 out, or NULL: fp16(dZ), what the gradients of
 *             adapters beside the weight are made of.
 *   dbias     [N] fp32 out, or NULL.
 * The product's operand is fl16(dZ * sW) in units of a power of two of its
 * own for every row, chosen by the row's largest value, so that neither
 * large nor small gradients leave fp16's range; sums are fp32.  The same call
 * gives the same bits.
 */
li8_status llm_int8_linear_backward(const void *dY, const void *pre, int32_t act, const int8_t *Wq,
                                    const float *sW, int64_t T, int64_t K, int64_t N, void *dX,
                                    void *grad_pre, float *dbias, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/*
 * dG = dH * U * act'(G),  dU = dH * act(G),  dX = fp16([dG | dU] . W'),
 * dbias = sum_t [dG | dU].
 *   dH        [T,F] fp16;  pre [T,2F] fp16, as llm_int8_gated_linear stored it.
 *   dX        [T,K] fp16 out;  grad_pre [T,2F] fp16 out, or NULL;
 *   dbias     [2F] fp32 out, or NULL.
 *   workspace llm_int8_backward_workspace_bytes(T, K, 2F) bytes.
 */
li8_status llm_int8_gated_backward(const void *dH, const void *pre, int32_t act, const int8_t *Wq,
                                   const float *sW, int64_t T, int64_t K, int64_t F, void *dX,
                                   void *grad_pre, float *dbias, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LLM_INT8_FFN_H */
