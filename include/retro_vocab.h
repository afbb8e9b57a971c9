/*
 * retro_vocab.h - C ABI of the operators over a model's vocabulary: embedding
 * lookup, its gradient, and the softmax cross entropy through a resident head
 * with its gradients, of the MI355X (gfx950) OUT_PROD library.
 *
 * W is one table of N rows x K, a model's embedding or its output head (or both):
 * any weight type of retro_out_prod.h, row n at byte n * ldw, with ldw as in
 * retro_out_prod_strided (at least retro_row_bytes(type, K), and as aligned as the
 * type's blocks). Packed tables are read as they are: no decoded copy of the whole
 * table exists.
 *
 * Token ids and targets are T integers of RETRO_I32 or RETRO_I64 on the device.
 * One outside 0 .. N - 1 stands for no token, such as padding or a prompt that is
 * not learnt from: it is never an error and never read through.
 *
 * Float tensors are RETRO_F32, RETRO_F16 or RETRO_BF16 with contiguous rows a
 * given number of elements apart (ld at least the row's length, any alignment of
 * whole elements). W is 16-byte aligned.
 *
 * Execution and errors are those of retro_out_prod.h: asynchronous on the
 * stream, no allocation, no CPU fallback, negative codes, all checks made on the
 * host before any launch. Workspaces need no initial value, hold nothing between
 * calls, are 16-byte aligned and overlap no operand (RETRO_E_WORKSPACE); calls that
 * share one are ordered on a stream. Results are the same bits each time: no sum's
 * order depends on the run. Sizes: K < 2^22, N < 2^31, T < 2^31 (2^28 in the
 * embedding's gradient, 2^22 in the cross entropy), every array below 2^62 bytes
 * (RETRO_E_SHAPE).
 */
#ifndef RETRO_VOCAB_H
#define RETRO_VOCAB_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Types of ids and targets: the GGUF tensor-type ids. */
enum { RETRO_I32 = 26, RETRO_I64 = 27 };

/*
 * Y[t][k] = scale * W[ids[t]][k], zeros where ids[t] is no token: the decoded F32
 * value (retro_dequantize) times scale, rounded once to F32 and once to ytype.
 */
int retro_embedding(int type, const void *W, int64_t ldw, int idtype, const void *ids, float scale, int ytype, void *Y,
                    int64_t ldy, int64_t K, int64_t N, int64_t T, void *stream);

/*
 * The gradient of retro_embedding with respect to a float table:
 *     dW[n][k] = scale * sum_{t: ids[t] = n} dY[t][k]           accumulate == 0
 *     dW[n][k] = dW[n][k] + scale * sum ...                     accumulate != 0
 * dY is T x K of ytype; dW is N x K of wtype (RETRO_F32, RETRO_F16 or RETRO_BF16),
 * rows ldw elements apart. Without accumulate every row is written, zeros where no
 * token has it; with it only the rows that a token has are touched. The sum is
 * taken in F32 over rising t, in runs (the list sorted by id and t is cut into 16s, or into
 * 64s where ceil(T / 64) * ceil(K / 512) is 2048 and more) whose sums are then added in
 * their order; scale and dW's old value enter in F32, and the result is rounded to wtype once.
 * workspace: retro_embedding_backward_workspace_size bytes.
 */
int retro_embedding_backward(int idtype, const void *ids, int ytype, const void *dY, int64_t ldy, float scale, int wtype,
                             void *dW, int64_t ldw, int accumulate, int64_t K, int64_t N, int64_t T, void *workspace,
                             int64_t workspace_bytes, void *stream);
int64_t retro_embedding_backward_workspace_size(int64_t K, int64_t N, int64_t T);

/*
 * Softmax cross entropy through the head, without keeping the logits:
 *     l[t][n] = sum_k x[t][k] W[n][k]
 *     lse[t]  = log sum_n exp l[t][n]                           F32, of every token
 *     loss[t] = lse[t] - l[t][targets[t]]                       F32; 0 where the target is no token
 * (the loss is made of differences of logits: a small one has digits that lse, beside a
 * large logit, has not).
 * x is T x K of xtype, rows ldx elements apart. The operands enter the matrix cores
 * as they are where x and W are both F16 or both BF16; otherwise in one or two F16
 * parts scaled by powers of two (one a row of x, one for W): F16, BF16, MXFP4 and
 * NVFP4 in one, the others in two, which leaves at most 2^-22 of a value and
 * 2^-38 of the largest one of x's row, or of W's finite ones (or 2^-151). Up to 64 tokens through a
 * packed table of contiguous rows meet its codes as they are, x in the same parts; those
 * of Q2_K, Q3_K and NVFP4 meet its F32 values in F32. Sums are F32. An infinite or NaN
 * logit gives a NaN or infinite loss for its token, only -inf counts as a probability
 * of 0; an infinity in W makes the logits of an F32 x NaN where it meets x's two parts.
 * N == 0 gives lse = -inf.
 * workspace: retro_cross_entropy_workspace_size bytes.
 */
int retro_cross_entropy(int type, const void *W, int64_t ldw, int xtype, const void *X, int64_t ldx, int idtype,
                        const void *targets, float *loss, float *lse, int64_t K, int64_t N, int64_t T, void *workspace,
                        int64_t workspace_bytes, void *stream);
int64_t retro_cross_entropy_workspace_size(int type, int64_t ldw, int xtype, int64_t K, int64_t N, int64_t T);

/*
 * Its gradients, from lse as retro_cross_entropy gave it and the gradient dloss[t]
 * (F32) of each token's loss:
 *     d[t][n]  = exp(l[t][n] - lse[t]) - [n == targets[t]]
 *     dX[t][k] = dloss[t] * sum_n d[t][n] W[n][k]               of xtype
 *     dW[n][k] = sum_t dloss[t] * d[t][n] x[t][k]               of W's type; W of floats only
 * A token whose target is none has dX = 0 and no part in dW, whatever its x, lse and
 * dloss hold. dW may be NULL: the table is frozen; a packed table's is RETRO_E_TYPE.
 * dX may be NULL where dW is not. Both are overwritten. d and dloss * d (scaled by a
 * power of two) enter the products in as many bits as the result has: one part of
 * 11 bits (8 where x and W are BF16), two for F32 results. The logits are those of
 * retro_cross_entropy, so that d is off by their F32 sums and a step of lse alone. W enters dX's sum as it
 * does them, but where x is BF16 in one part of 11 bits (unless an F32 dW is wanted).
 * workspace: retro_cross_entropy_backward_workspace_size bytes.
 */
int retro_cross_entropy_backward(int type, const void *W, int64_t ldw, int xtype, const void *X, int64_t ldx, int idtype,
                                 const void *targets, const float *lse, const float *dloss, void *dX, int64_t lddx,
                                 void *dW, int64_t lddw, int64_t K, int64_t N, int64_t T, void *workspace,
                                 int64_t workspace_bytes, void *stream);
int64_t retro_cross_entropy_backward_workspace_size(int type, int64_t ldw, int xtype, int weight_grad, int64_t K,
                                                    int64_t N, int64_t T);

#ifdef __cplusplus
}
#endif
#endif
