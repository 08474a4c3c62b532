/*
 * sample.h -- drawing tokens from rows of logits, of libsgemm for MI355X (gfx950).
 *
 * For each of T rows of V logits (fp32 or bf16, row-major) and the row's u in [0, 1):
 *
 *   1. z = logit / temperature; the row's tokens in the order of falling z, of equal ones the lower index first;
 *   2. the first top_k stay (top_k <= 0 or >= V: all);
 *   3. of those, each before which less than top_p of their probability lies; the first stays always
 *      (top_p >= 1: all);
 *   4. of those, each with at least min_p times the first one's probability (min_p <= 0: all; the first stays always);
 *   5. the token is the first, by index, up to which (itself included) more than u of the probability of what stays
 *      lies.  u >= 1 gives the last that stays, u < 0 the first.
 *
 * temperature 0 takes the largest logit, of equal ones the lowest index.  Logits of -infinity are never drawn.  A row
 * that holds NaN or +infinity, or no finite logit, gives -1, and so does a temperature that is negative, infinite or
 * NaN, or a NaN for u, top_p or min_p.
 *
 * Probabilities are added up as whole multiples of 2^-40 of the largest one, in 64 bits, so that a token does not
 * depend on timing or on how the work is cut.  exp(-x) of the distance x from the largest logit is off by up to
 * 2^-22 + 2^-23 x of itself.  A token whose probability is below 2^-41 of the largest one's is not drawn, nor is one
 * whose logit lies more than 3.4e38 below it, at any temperature; a temperature below 2^-119 counts as 2^-119.
 *
 * temperature, top_k, top_p and min_p are one value for all rows, or with a pointer (device memory) one for each.
 *
 * Memory and streams: device pointers owned by the caller, work enqueued on `stream`, no wait, no allocation, no
 * memset; calls may be captured into a HIP graph.  `work` is scratch memory of at least vocab_sample_workspace(...)
 * bytes, 16-byte aligned, whose contents before and after mean nothing; calls that may run at the same time need one each.
 *
 * Return codes as in sgemm.h: 0, -i for argument i, +hipError_t from a launch.  T = 0 is a quick return.
 */
#ifndef LIBSGEMM_SAMPLE_H
#define LIBSGEMM_SAMPLE_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SAMPLE_F32 = 0, SAMPLE_BF16 = 1 };

/* Bytes of workspace.  Limits of every call: T <= 2^21, 1 <= V <= 2^23.  Negative: -i for argument i. */
SGEMM_API long long vocab_sample_workspace(int dtype, int T, int V);

/* token[T].  Where temperatures, top_ks, top_ps or min_ps is not null it holds T values, and the one beside it is
 * not looked at. */
SGEMM_API int vocab_sample(int dtype, int T, int V, const void *logits, int ld, const float *u, float temperature,
                           const float *temperatures, long long top_k, const long long *top_ks, float top_p,
                           const float *top_ps, float min_p, const float *min_ps, long long *token, void *work,
                           long long work_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_SAMPLE_H */
