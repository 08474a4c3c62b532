/*
 * vocab.h -- the vocabulary-head operators of libsgemm for MI355X (gfx950).
 *
 * Both are losses over the logits of T tokens against a vocabulary matrix,
 *
 *     z[t][v] = alpha * sum_h X[t][h] * W[v][h],      lse[t] = log(sum_v exp(z[t][v])),
 *
 * X a T x H and W a V x H row-major matrix, fp32 or bf16.  The T x V logits are never stored:
 *
 *   cross entropy   loss[t] = lse[t] - z[t][target[t]];
 *   distillation    loss[t] = sum_k q[t][k] * (log q[t][k] - (z[t][index[t][k]] - lse[t])),
 *                   q[t] the softmax of teacher_alpha * teacher[t][k] over the K entries with
 *                   index[t][k] >= 0: a teacher's top logits.
 *
 * The gradient entry points return those of sum_t dloss[t] * loss[t]:
 *
 *     D[t][v] = alpha * dloss[t] * (exp(z[t][v] - lse[t]) - y[t][v]),   dX = D W,   dW = D^T X,
 *
 * y the one-hot target, or the teacher's q added up per vocabulary row (an entry may be named
 * twice).  They recompute the logits in pieces of the vocabulary, from the forward call's lse.
 *
 * A piece's D is a workspace array of at most about 768 MB; one piece may be the whole vocabulary.
 *
 * Tokens that do not count -- target == ignore_index, or no index >= 0 -- have loss 0, lse 0 and
 * gradient 0, whatever X, dloss and teacher hold there (NaN and infinities included); among more
 * than 64 tokens they cost no product either.  A target or an index >= V (or a target < 0 that is
 * not ignore_index) cannot be refused without waiting for the device: nothing is read for it, and
 * the token's loss and the gradients that it enters are NaN.  Teacher entries of -infinity have
 * q = 0 and add nothing.
 *
 * Memory and streams: device pointers owned by the caller, work enqueued on `stream`, no wait, no
 * allocation, no memset; calls may be captured into a HIP graph.  `work` is scratch memory of at
 * least vocab_workspace(...) bytes, 16-byte aligned, whose contents before and after mean nothing.
 * dX and dW must not overlap X, W or each other.  Results do not depend on timing: the same call
 * gives the same bits.
 *
 * Precision: loss, lse, picked, dloss and teacher are fp32, as are all sums and softmax
 * statistics.  fp32 X and W of more than 64 tokens are multiplied as two fp16 parts each, scaled by
 * a power of two (a token's own for X; for W a row's own in the forward calls, one for the whole of W in
 * the gradients): values down to 2^-16 of the largest keep 23 bits, smaller ones are held to 2^-40 of the
 * largest.  Of D = s * (..), s = alpha * dloss, the part in brackets is held to 2^-40, in dX for every token
 * by itself; dW takes s * X in one power of two, held to 2^-40 of its largest value.  Values of W above
 * 2^90 may overflow.  Of 17 to 64 tokens the operands are three bf16 parts each, 24 bits; with up to 16 the
 * products are fp32's own.  An infinity in W may make NaN of every logit of its row, and a teacher's row of
 * -infinities alone makes its token NaN.  With bf16 X and W, D is rounded for the two gradient products: to
 * bf16 (cross entropy scales a token's row so that its target's entry is exact), or of up to 64 tokens to two
 * bf16 parts; dX and dW are rounded to bf16 at the end.
 *
 * A loss is a difference of lse and logits that were summed apart (of up to 64 tokens' cross entropy,
 * together), each off by a few roundings of its size: up to 3e-5 at a logit of 40, which is all of a confident
 * token's loss.  Cross entropy is not below 0.
 *
 * Return codes as in sgemm.h: 0, -i for argument i, +hipError_t from a launch.  T = 0 is a quick
 * return (dW, when wanted, is set to 0).
 */
#ifndef LIBSGEMM_VOCAB_H
#define LIBSGEMM_VOCAB_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { VOCAB_F32 = 0, VOCAB_BF16 = 1 }; /* the type of X, W, dX and dW */

/* Bytes of workspace of a call: grad 0 for the forward entry points, 1 for the gradients; K = 0 for
 * cross entropy, else the teacher's entries per token.  Of more than 64 tokens it holds about 768 MB at
 * most for a piece of the vocabulary, of 256 rows or more (packed W, also where bf16 W needs no packing, and D); X packed, in a gradient
 * twice, and dX in fp32 once for each part that its product is cut into; and T V / 8 bytes of
 * maxima and sums in a forward call.  A gradient from more than 8192 entries a token takes 8 T K bytes to
 * sort them.  Limits of every call: T <= 2^21,
 * V <= 2^31 - 1025, H <= 2^20, K * T < 2^31.  Negative: -i for argument i. */
SGEMM_API long long vocab_workspace(int dtype, int grad, int T, int V, int H, int K);

/* loss[T], lse[T] of cross entropy. */
SGEMM_API int vocab_ce(int dtype, int T, int V, int H, float alpha, const void *X, int ldx, const void *W, int ldw,
                       const long long *target, long long ignore_index, float *loss, float *lse, void *work,
                       long long work_bytes, hipStream_t stream);

/* dX (T x H) and dW (V x H) of cross entropy; either may be null (not wanted). */
SGEMM_API int vocab_ce_grad(int dtype, int T, int V, int H, float alpha, const void *X, int ldx, const void *W,
                            int ldw, const long long *target, long long ignore_index, const float *lse,
                            const float *dloss, void *dX, int lddx, void *dW, int lddw, void *work,
                            long long work_bytes, hipStream_t stream);

/* loss[T], lse[T] and picked (T x K, packed): the student's logits at the teacher's entries, 0
 * where there is none. */
SGEMM_API int vocab_distill(int dtype, int T, int V, int H, int K, float alpha, float teacher_alpha, const void *X,
                            int ldx, const void *W, int ldw, const long long *index, int ldi, const float *teacher,
                            int ldt, float *loss, float *lse, float *picked, void *work, long long work_bytes,
                            hipStream_t stream);

/* dX and dW of distillation, from the forward call's lse and picked; either may be null. */
SGEMM_API int vocab_distill_grad(int dtype, int T, int V, int H, int K, float alpha, float teacher_alpha,
                                 const void *X, int ldx, const void *W, int ldw, const long long *index, int ldi,
                                 const float *teacher, int ldt, const float *lse, const float *picked,
                                 const float *dloss, void *dX, int lddx, void *dW, int lddw, void *work,
                                 long long work_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_VOCAB_H */
