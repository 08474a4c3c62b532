/*
 * linear.h -- the linear layer with an epilogue of libsgemm for MI355X (gfx950), forward and gradient.
 *
 *     Z[t][n] = sum_h X[t][h] * W[n][h] + bias[n],      Y[t][n] = act(Z[t][n]) + residual[t][n],
 *
 * X a T x H, W an N x H row-major matrix, fp32 or bf16; bias and residual may be null.  The activations:
 *
 *   LINEAR_NONE       z
 *   LINEAR_RELU       max(z, 0)
 *   LINEAR_GELU       z * Phi(z), Phi the normal distribution function
 *   LINEAR_GELU_TANH  z / 2 * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3)))
 *   LINEAR_SILU       z / (1 + exp(-z))
 *
 * The gradient entry point takes dY and the kept Z (not needed without an activation) and returns
 *
 *     dZ = dY * act'(Z) (0 at z = 0 for RELU),   dX = dZ W,   dW = dZ^T X,   dbias[n] = sum_t dZ[t][n].
 *
 * The residual's gradient is dY itself.
 *
 * Types: all operands and results of a call have its dtype, but with out_dtype LINEAR_F32 beside bf16 operands Y
 * and the residual are fp32 (logits, say).  Everything is summed in fp32 and rounded once, when it is stored: Y is
 * computed from the unrounded Z, dX, dW and dbias from fp32 sums.  In bf16 the kept Z is rounded to bf16, and so is
 * dZ on its way into dX and dW (of up to 64 tokens it enters as two bf16 parts, 16 bits); dbias sums it before that.
 *
 * Products: bf16 operands on the bf16 matrix instructions.  fp32 operands on the fp32 ones; of 17 to 64 tokens as three
 * bf16 parts each, 24 bits, without what lies below 2^-126 (the last digits of values below 2^-110).  Infinities, NaN
 * and the largest values come out as in any fp32 sum, whatever the number of tokens, but in a gradient of up to 64:
 * there an infinity, and of 17 to 64 fp32 tokens a value from 2^127 on, may come out as NaN.  A row of X, dY or
 * residual reaches its own row of Y and dX alone.
 *
 * Memory and streams: device pointers owned by the caller, work enqueued on `stream`, no wait, no allocation, no
 * memset; calls may be captured into a HIP graph.  `work` is scratch memory of at least linear_workspace(...) bytes,
 * 16-byte aligned, whose contents before and after mean nothing; calls that may run at the same time need one each.
 * Results must not overlap an operand or each other (spans from the first to the last addressed byte).  The same call
 * gives the same bits.
 *
 * Return codes as in sgemm.h: 0, -i for argument i, +hipError_t from a launch.  T = 0 is a quick return (dW and
 * dbias, when wanted, are set to 0).
 */
#ifndef LIBSGEMM_LINEAR_H
#define LIBSGEMM_LINEAR_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { LINEAR_F32 = 0, LINEAR_BF16 = 1 };
enum { LINEAR_NONE = 0, LINEAR_RELU = 1, LINEAR_GELU = 2, LINEAR_GELU_TANH = 3, LINEAR_SILU = 4 };

/* Bytes of workspace of a call: grad 0 for linear_act, 1 for linear_act_grad.  It holds a copy of X and of W, in a
 * gradient also dZ, in rows of whole 128 bytes (for operands that are not 16-byte aligned, whose rows are no whole
 * 16 bytes), and the partial sums of a product that is cut along its long axis.  Limits of every call: T <= 2^24, N <= 2^21, H <= 2^20,
 * T * N <= 2^35, T * H <= 2^35.  Negative: -i for argument i. */
SGEMM_API long long linear_workspace(int dtype, int grad, int T, int N, int H);

/* Y (T x N) and, where Z is not null, the kept Z (T x N, in dtype). */
SGEMM_API int linear_act(int dtype, int out_dtype, int T, int N, int H, const void *X, int ldx, const void *W, int ldw,
                         const void *bias, const void *residual, int ldr, int activation, void *Y, int ldy, void *Z,
                         int ldz, void *work, long long work_bytes, hipStream_t stream);

/* dX (T x H), dW (N x H), dbias (N); each may be null (not wanted).  Z may be null without an activation. */
SGEMM_API int linear_act_grad(int dtype, int T, int N, int H, const void *X, int ldx, const void *W, int ldw,
                              const void *dY, int lddy, const void *Z, int ldz, int activation, void *dX, int lddx,
                              void *dW, int lddw, void *dbias, void *work, long long work_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_LINEAR_H */
