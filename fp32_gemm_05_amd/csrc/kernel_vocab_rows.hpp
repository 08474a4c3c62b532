// kernel_vocab_rows.hpp -- the per-token work around the products of kernel_vocab.hpp: which
// tokens count, their packed rows, the logits of their own entries, the statistics and the losses.
// All of it is a few reads of T x H and T x K values: bound by latency at small sizes and by HBM
// at large ones.
#pragma once

#include "kernel_vocab.hpp"

namespace libsgemm {
namespace vocab {

typedef long long i64;

// What a token is compared with.  Cross entropy: one entry, its target.  Distillation: the entries
// that a teacher gives, `index` < 0 where it gives none.
struct Entries {
    const i64* index;     // target (ld 1, k 1), or the teacher's entries
    long ld;
    int k;                // entries per token
    i64 ignore;           // cross entropy: the target that does not count
    const float* teacher; // null: cross entropy
    long ld_teacher;
    float teacher_alpha;
    __device__ bool counts(i64 v) const { return teacher ? v >= 0 : v != ignore; }
};

// rows[0 .. *count): the tokens that count, in order; pos: a token's place in rows, or -1.  One
// workgroup walks the tokens.  loss and lse (when given) of the others are 0.
__global__ void __launch_bounds__(1024) vocab_count_kernel(Entries e, int tokens, int* rows, int* pos, int* count,
                                                           float* loss, float* lse) {
    __shared__ int waves[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int done = 0;
    for (int t0 = 0; t0 < tokens; t0 += 1024) {
        const int t = t0 + threadIdx.x;
        bool live = false;
        if (t < tokens)
            for (int k = 0; k < e.k && !live; ++k) live = e.counts(e.index[(size_t)t * e.ld + k]);
        const unsigned long long m = __ballot(live);
        if (lane == 0) waves[wave] = __popcll(m);
        __syncthreads();
        int before = done, all = 0;
        for (int w = 0; w < 16; ++w) {
            before += w < wave ? waves[w] : 0;
            all += waves[w];
        }
        if (t < tokens) {
            const int at = before + __popcll(m & ((1ull << lane) - 1));
            pos[t] = live ? at : -1;
            if (live) rows[at] = t;
            if (!live && loss) loss[t] = 0.f;
            if (!live && lse) lse[t] = 0.f;
        }
        done += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) *count = done;
}

template <typename T>
__device__ inline float wave_dot(const T* x, const T* w, int n) {
    const int lane = threadIdx.x & 63;
    float s = 0.f;
    for (int i = lane; i < n; i += 64) s = __builtin_fmaf((float)x[i], (float)w[i], s);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    return s;
}
__device__ inline float wave_sum(float s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    return s;
}
__device__ inline float wave_max(float s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s = fmaxf(s, __shfl_xor(s, o));
    return s;
}

// Rows (through `map` when given) of a rows x cols matrix, packed: row i at dst + i * pitch, zero
// past cols up to kp, whole zero rows from the number of rows to its next multiple of 256.  scaled
// (when given) gets the rows times scale[i].
template <typename T, int P>
__global__ void __launch_bounds__(256) vocab_pack_kernel(const T* src, long ld, const int* map, const int* count,
                                                         int rows, int cols, char* dst, long pitch, int kp,
                                                         const float* scale, char* scaled) {
    const int i = blockIdx.x, n = count ? *count : rows;
    if (i >= (n + 255) / 256 * 256) return;
    const T* s = i < n ? src + (size_t)(map ? map[i] : i) * ld : nullptr;
    const float f = scaled && i < n ? scale[i] : 0.f;
    for (int k = threadIdx.x * 4; k < kp; k += 1024) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = s && k + q < cols ? (float)s[k + q] : 0.f;
        store4<P>(dst + (size_t)i * pitch, k, v);
        if (!scaled) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] *= f;
        store4<P>(scaled + (size_t)i * pitch, k, v);
    }
}

// z[t][k] = alpha * X[t] . W[index[t][k]], one wave each; 0 where there is no entry, NaN where an
// entry lies past the vocabulary.
template <typename T>
__global__ void __launch_bounds__(256) vocab_pick_kernel(Entries e, int tokens, int vocab, int hidden, float alpha,
                                                         const T* x, long ldx, const T* w, long ldw, float* z) {
    const long i = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= (long)tokens * e.k) return;
    const long t = i / e.k, k = i - t * e.k;
    const i64 v = e.index[t * e.ld + k];
    float s = 0.f;
    if (e.counts(v)) s = v >= 0 && v < vocab ? alpha * wave_dot(x + t * ldx, w + (size_t)v * ldw, hidden) : NAN;
    if ((threadIdx.x & 63) == 0) z[i] = s;
}

// The teacher's softmax over a token's entries, by one wave: maximum and log of the sum.
__device__ inline void teacher_stats(const Entries& e, long t, float& top, float& log_total) {
    const int lane = threadIdx.x & 63;
    const i64* index = e.index + t * e.ld;
    const float* teacher = e.teacher + t * e.ld_teacher;
    float m = -INFINITY;
    for (int k = lane; k < e.k; k += 64)
        if (index[k] >= 0) m = fmaxf(m, teacher[k] * e.teacher_alpha);
    top = wave_max(m);
    float s = 0.f;
    for (int k = lane; k < e.k; k += 64)
        if (index[k] >= 0) s += expf(teacher[k] * e.teacher_alpha - top);
    log_total = logf(wave_sum(s));
}

// lse of each counted token from its partial maxima and sums, then its loss.  A workgroup takes 32
// tokens, 8 threads each.
__global__ void __launch_bounds__(256) vocab_loss_kernel(Entries e, const int* rows, const int* count,
                                                         const float2* part, int parts, int tp, const float* z,
                                                         float* loss, float* lse) {
    __shared__ float tops[8][32], sums[8][32], lses[32];
    const int n = *count, tx = threadIdx.x & 31, ty = threadIdx.x >> 5, i0 = blockIdx.x * 32, i = i0 + tx;
    if (i0 >= n) return;
    float top = -INFINITY, sum = 0.f;
    if (i < n)
        for (int p = ty; p < parts; p += 8) {
            const float2 v = part[(size_t)p * tp + i];
            const float m = v.x > top || v.x != v.x ? v.x : top;
            if (m == -INFINITY) continue;
            sum = sum * expf(top - m) + v.y * expf(v.x - m);
            top = m;
        }
    tops[ty][tx] = top;
    sums[ty][tx] = sum;
    __syncthreads();
    if (ty == 0 && i < n) {
        float m = top;
        for (int y = 1; y < 8; ++y) m = tops[y][tx] > m || tops[y][tx] != tops[y][tx] ? tops[y][tx] : m;
        float s = 0.f;
        for (int y = 0; y < 8; ++y) s += m == -INFINITY ? 0.f : sums[y][tx] * expf(tops[y][tx] - m);
        const float l = m + logf(s);
        const int t = rows[i];
        lses[tx] = l;
        lse[t] = l;
        if (!e.teacher) loss[t] = l - z[t];
    }
    if (!e.teacher) return;
    __syncthreads();
    const int lane = threadIdx.x & 63;
    for (int y = threadIdx.x >> 6; y < 32; y += 4) {
        if (i0 + y >= n) break;
        const int t = rows[i0 + y];
        const float l = lses[y];
        float top_t, log_total, s = 0.f;
        teacher_stats(e, t, top_t, log_total);
        for (int k = lane; k < e.k; k += 64) {
            if (e.index[(size_t)t * e.ld + k] < 0) continue;
            const float lq = e.teacher[(size_t)t * e.ld_teacher + k] * e.teacher_alpha - top_t - log_total;
            const float q = expf(lq), zk = z[(size_t)t * e.k + k];
            // an entry without mass adds nothing, whatever its logarithm
            if (q != 0.f) s += q * (lq - zk + l);
            else if (zk != zk) s = NAN;
        }
        s = wave_sum(s);
        if (lane == 0) loss[t] = s;
    }
}

// Per counted token what its row of D needs; one wave per token.
//
// Cross entropy: with s = alpha * dloss, p the softmax and c = 1 - p[target], row i of D is p / c
// with -1 at the target, and X enters dW, and the product enters dX, times s * c.  The target's
// entry carries most of the gradient: as -1 it is exact in bf16, where alpha * dloss * (p - 1)
// would be rounded.  c comes from expm1, so a p close to 1 costs no digits; a c below 2^-25, where
// fp32 cannot tell p from 1, is raised to it.
//
// Distillation: row i of D is s * p, and s * (p - sum of q over the entries that name the same
// vocabulary row) at the entries; X and the product enter as they are.
__global__ void __launch_bounds__(256) vocab_rows_kernel(Entries e, int tokens, int vocab, float alpha,
                                                         const int* pos, const float* lse, const float* dloss,
                                                         const float* z, float* lse_c, float* scale, float* out_scale,
                                                         float* value) {
    const long t = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (t >= tokens) return;
    const int i = pos[t];
    if (i < 0) return;
    const float s = alpha * dloss[t], l = lse[t];
    float sc, os;
    if (!e.teacher) {
        const i64 v = e.index[t * e.ld];
        const float c = fmaxf(-expm1f(z[t] - l), 0x1p-25f);
        const bool good = v >= 0 && v < vocab;
        sc = good ? 1.f / c : NAN;
        os = good ? s * c : NAN;
        if (lane == 0) value[t] = -1.f;
    } else {
        bool good = true;
        float top, log_total;
        teacher_stats(e, t, top, log_total);
        const i64* index = e.index + t * e.ld;
        const float* teacher = e.teacher + t * e.ld_teacher;
        for (int k = lane; k < e.k; k += 64) {
            const i64 v = index[k];
            float d = 0.f;
            if (v >= 0) {
                good = good && v < vocab;
                float q = 0.f;
                for (int o = 0; o < e.k; ++o)
                    if (index[o] == v) q += expf(teacher[o] * e.teacher_alpha - top - log_total);
                d = s * (expf(z[t * e.k + k] - l) - q);
            }
            value[t * e.k + k] = d;
        }
        sc = __all(good) ? s : NAN;
        os = 1.f;
    }
    if (lane == 0) {
        lse_c[i] = l;
        scale[i] = sc;
        out_scale[i] = os;
    }
}

// Puts the entries' values into D where they fall into this piece.
template <int P>
__global__ void __launch_bounds__(256) vocab_patch_kernel(Entries e, int tokens, int v0, int vocab, const int* pos,
                                                          const float* value, char* d, long d_pitch) {
    const long j = (long)blockIdx.x * 256 + threadIdx.x;
    if (j >= (long)tokens * e.k) return;
    const long t = j / e.k, k = j - t * e.k;
    const int i = pos[t];
    const i64 v = e.index[t * e.ld + k];
    if (i < 0 || !e.counts(v) || v < v0 || v >= v0 + vocab) return;
    store1<P>(d + (size_t)i * d_pitch, v - v0, value[j]);
}

// dX of every token: the sum of its product's parts, or 0 where it does not count.
template <typename T>
__global__ void __launch_bounds__(256) vocab_dx_out_kernel(const int* pos, int hidden, const float* acc, int splits,
                                                           long tp, int hp, const float* scale, T* dx, long ld) {
    const int t = blockIdx.x, i = pos[t];
    const float s = i < 0 ? 0.f : scale[i];
    for (int h = threadIdx.x; h < hidden; h += 256) {
        float v = 0.f;
        if (i >= 0) {
            for (int z = 0; z < splits; ++z) v += acc[((size_t)z * tp + i) * hp + h];
            v *= s;
        }
        dx[(size_t)t * ld + h] = (T)v;
    }
}

}  // namespace vocab
}  // namespace libsgemm
