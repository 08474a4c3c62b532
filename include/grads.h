/*
 * grads.h -- the norm of many gradients and clipping by it, of libsgemm for MI355X (gfx950).
 *
 *     norm = sqrt(sum over all tensors and elements of x^2)
 *     out = x * min(1, max_norm / (norm + eps))      (x where norm + eps is 0)
 *
 * The tensors are row-major matrices, fp32 or bf16, mixed as they come; a contiguous tensor of any shape is one row.
 * Squares are summed in 64 bits, in an order that goes by the sizes alone: the same call gives the same bits, and
 * neither large nor small values leave the range.  norm is fp32, on the device; the factor is computed in 64 bits
 * from the sum, rounded to fp32, and each product rounded once to its tensor's type.  A NaN or an infinity in a
 * gradient makes norm what it makes of the sum, NaN or infinity, and the factor NaN or 0.
 *
 * Memory and streams: the array of GradTensor is host memory and read before the call returns; the tensors are device
 * memory owned by the caller.  Work is enqueued on `stream`, no wait, no allocation, no memset; calls may be captured
 * into a HIP graph.  `work` is scratch memory of at least grad_workspace(...) bytes, 16-byte aligned, whose contents
 * before and after mean nothing; calls that may run at the same time need one each.
 *
 * out may be the tensor itself (the same address, sizes and row stride), which is then left as it is where the factor
 * is 1; otherwise no out may overlap a tensor or another out (spans from the first to the last addressed byte).
 *
 * Return codes as in sgemm.h: 0, -i for argument i, +hipError_t from a launch.
 */
#ifndef LIBSGEMM_GRADS_H
#define LIBSGEMM_GRADS_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GRADS_F32 = 0, GRADS_BF16 = 1 };

/* One tensor: rows x cols elements, rows ld apart; out (rows ld_out apart) is looked at by clip_grad_norm alone.
 * rows < 2^31, ld < 2^31 where there are several rows; rows * cols <= 2^40. */
typedef struct {
    const void *x;
    void *out;
    long long rows, cols, ld, ld_out;
    long long dtype;
} GradTensor;

/* Bytes of workspace of a call with these tensors.  count <= 2^20.  Negative: -i for argument i. */
SGEMM_API long long grad_workspace(int count, const GradTensor *tensors);

/* norm[0]; 0 of no tensors. */
SGEMM_API int grad_norm(int count, const GradTensor *tensors, float *norm, void *work, long long work_bytes,
                        hipStream_t stream);

/* norm[0] of the tensors as they were, and every out. */
SGEMM_API int clip_grad_norm(int count, const GradTensor *tensors, float max_norm, float eps, float *norm, void *work,
                             long long work_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_GRADS_H */
