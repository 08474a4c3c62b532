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
// workgroup walks the tokens, 8192 at a time so that their entries are read together.  loss and lse
// (when given) of the others are 0.  Clears `zero` as well, the maxima that later kernels raise.
__global__ void __launch_bounds__(1024) vocab_count_kernel(Entries e, int tokens, int* rows, int* pos, int* count,
                                                           float* loss, float* lse, uint32_t* zero, int zeros) {
    constexpr int R = 8;
    __shared__ int waves[R][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < zeros; i += 1024) zero[i] = 0;
    int done = 0;
    for (int t0 = 0; t0 < tokens; t0 += 1024 * R) {
        bool live[R];
        unsigned long long m[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = t0 + r * 1024 + threadIdx.x;
            live[r] = t < tokens && e.counts(e.index[(size_t)t * e.ld]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = t0 + r * 1024 + threadIdx.x;
            if (t < tokens)
                for (int k = 1; k < e.k && !live[r]; ++k) live[r] = e.counts(e.index[(size_t)t * e.ld + k]);
            m[r] = __ballot(live[r]);
            if (lane == 0) waves[r][wave] = __popcll(m[r]);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int before = done;
            for (int w = 0; w < 16; ++w) {
                before += w < wave ? waves[r][w] : 0;
                done += waves[r][w];
            }
            const int t = t0 + r * 1024 + threadIdx.x;
            if (t >= tokens) continue;
            const int at = before + __popcll(m[r] & ((1ull << lane) - 1));
            pos[t] = live[r] ? at : -1;
            if (live[r]) rows[at] = t;
            if (!live[r] && loss) loss[t] = 0.f;
            if (!live[r] && lse) lse[t] = 0.f;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) *count = done;
}

// N consecutive values, at any alignment of their type (gfx950 loads unaligned vectors).
template <int N, typename T>
__device__ inline void load(const T* p, float (&v)[N]) {
    T t[N];
    __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)t[i];
}
template <typename T>
__device__ inline float wave_dot(const T* x, const T* w, int n) {
    constexpr int N = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    float s[N] = {};
    int i = lane * N;
#pragma unroll 4
    for (; i + N <= n; i += 64 * N) {
        float a[N], b[N];
        load(x + i, a);
        load(w + i, b);
#pragma unroll
        for (int q = 0; q < N; ++q) s[q] = __builtin_fmaf(a[q], b[q], s[q]);
    }
    for (; i < n; ++i) s[0] = __builtin_fmaf((float)x[i], (float)w[i], s[0]);  // the lane with the row's end
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < N; ++q) t += s[q];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o);
    return t;
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

// The largest finite |x|.
__device__ inline float finite_max(float m, float x) { return __builtin_isfinite(x) ? fmaxf(m, fabsf(x)) : m; }
template <int N>
__device__ inline float block_max(float m) {
    __shared__ float part[N / 64];
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < N / 64; ++w) m = fmaxf(m, part[w]);
    return m;
}

// The counted tokens' rows of X, packed: row i at dst + i * pitch, zero past the hidden size up to
// kp, whole zero rows from the number of tokens to its next multiple of 256.
//
// P = 1: `scaled` (when given) gets the rows times weight[i].  P = 2: each row in its own power of
// two, unit[i] what it is to be multiplied with; most (when given) the largest |weight| * unit.
template <typename T, int P>
__global__ void __launch_bounds__(256) vocab_pack_x_kernel(const T* src, long ld, const int* map, const int* count,
                                                           int cols, char* dst, long pitch, int kp,
                                                           const float* weight, char* scaled, float* unit,
                                                           uint32_t* most) {
    const int i = blockIdx.x, n = *count;
    if (i >= (n + 255) / 256 * 256) return;
    const T* s = i < n ? src + (size_t)map[i] * ld : nullptr;
    float f = 1.f;
    if constexpr (P == 2) {
        if (s) {
            float m = 0.f;
            for (int k = threadIdx.x * 4; k < cols; k += 1024)
                if (k + 4 <= cols) {
                    float v[4];
                    load(s + k, v);
#pragma unroll
                    for (int q = 0; q < 4; ++q) m = finite_max(m, v[q]);
                } else {
                    for (int q = k; q < cols; ++q) m = finite_max(m, (float)s[q]);
                }
            const int e = scale_exponent(block_max<256>(m));
            f = ldexpf(1.f, e);
            if (threadIdx.x == 0) {
                const float u = ldexpf(1.f, -e);
                unit[i] = u;
                const float w = most ? fabsf(weight[i] * u) : 0.f;
                if (w > 0.f) atomicMax(most, __float_as_uint(w));
            }
        }
    } else if (scaled && s) {
        f = weight[i];
    }
    for (int k = threadIdx.x * 4; k < kp; k += 1024) {
        float v[4] = {};
        if (s && k + 4 <= cols)
            load(s + k, v);
        else if (s)
            for (int q = 0; q < 4; ++q) v[q] = k + q < cols ? (float)s[k + q] : 0.f;
        if constexpr (P == 1) {
            store4<P>(dst + (size_t)i * pitch, k, v);
            if (!scaled) continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] *= f;
        store4<P>((P == 1 ? scaled : dst) + (size_t)i * pitch, k, v);
    }
}

// The largest finite magnitude of a piece of W, as the bits of a float.
template <typename T>
__global__ void __launch_bounds__(256) vocab_max_kernel(const T* src, long ld, int rows, int cols, uint32_t* most) {
    float m = 0.f;
    const int lane = threadIdx.x & 63;
    for (int r = blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += gridDim.x * 4) {
        const T* s = src + (size_t)r * ld;
        int k = lane * 4;
#pragma unroll 4
        for (; k + 4 <= cols; k += 256) {
            float v[4];
            load(s + k, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) m = finite_max(m, v[q]);
        }
        for (; k < cols; ++k) m = finite_max(m, (float)s[k]);
    }
    m = block_max<256>(m);
    if (threadIdx.x == 0 && m > 0.f) atomicMax(most, __float_as_uint(m));
}

// A piece of W packed, zero past the hidden size up to kp and from its rows to their next multiple
// of 256; P = 2: in the power of two of its largest value, *unit what a packed unit stands for.
template <typename T, int P>
__global__ void __launch_bounds__(256) vocab_pack_w_kernel(const T* src, long ld, int rows, int cols, char* dst,
                                                           long pitch, int kp, const uint32_t* most, float* unit) {
    const int i = blockIdx.x;
    const T* s = i < rows ? src + (size_t)i * ld : nullptr;
    float f = 1.f;
    if constexpr (P == 2) {
        const int e = scale_exponent(__uint_as_float(*most));
        f = ldexpf(1.f, e);
        if (i == 0 && threadIdx.x == 0) *unit = ldexpf(1.f, -e);
    }
    for (int k = threadIdx.x * 4; k < kp; k += 1024) {
        float v[4] = {};
        if (s && k + 4 <= cols)
            load(s + k, v);
        else if (s)
            for (int q = 0; q < 4; ++q) v[q] = k + q < cols ? (float)s[k + q] : 0.f;
        if constexpr (P == 2)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] *= f;
        store4<P>(dst + (size_t)i * pitch, k, v);
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

// lse of each counted token from its partial maxima and sums, then its loss.  A workgroup takes TX
// tokens, TY threads each: once through the maxima, once through the sums, so that no load waits
// for an exponential.
template <int TX>
__global__ void __launch_bounds__(1024) vocab_loss_kernel(Entries e, const int* rows, const int* count,
                                                          const float2* part, int parts, int tp, const float* z,
                                                          float* loss, float* lse) {
    constexpr int TY = 1024 / TX;
    __shared__ float slot[16][TX], lses[TX];
    const int n = *count, tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = blockIdx.x * TX, i = i0 + tx;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (i0 >= n) return;
    const auto larger = [](float a, float b) { return b > a || b != b ? b : a; };  // a NaN stays
    float top = -INFINITY;
    if (i < n)
#pragma unroll 8
        for (int p = ty; p < parts; p += TY) top = larger(top, part[(size_t)p * tp + i].x);
#pragma unroll
    for (int o = TX; o < 64; o *= 2) top = larger(top, __shfl_xor(top, o));
    if (lane < TX) slot[wave][tx] = top;
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 16; ++y) top = larger(top, slot[y][tx]);
    __syncthreads();
    float sum = 0.f;
    if (i < n && top != -INFINITY)
#pragma unroll 8
        for (int p = ty; p < parts; p += TY) {
            const float2 v = part[(size_t)p * tp + i];
            sum += v.y * expf(v.x - top);
        }
#pragma unroll
    for (int o = TX; o < 64; o *= 2) sum += __shfl_xor(sum, o);
    if (lane < TX) slot[wave][tx] = sum;
    __syncthreads();
    if (ty == 0 && i < n) {
        sum = 0.f;
#pragma unroll
        for (int y = 0; y < 16; ++y) sum += slot[y][tx];
        const float l = top + logf(sum);
        const int t = rows[i];
        lses[tx] = l;
        lse[t] = l;
        if (!e.teacher) loss[t] = l - z[t];
    }
    if (!e.teacher) return;
    __syncthreads();
    for (int y = wave; y < TX; y += 16) {
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

enum DForm { D_PACKED, D_APART, D_WHOLE };

// Per counted token what its row of D needs; one wave per token.
//
// Cross entropy: with s = alpha * dloss, p the softmax and c = 1 - p[target], row i of D is p / c
// with -1 at the target, and X enters dW, and the product enters dX, times s * c.  The target's
// entry carries most of the gradient: as -1 it is exact in bf16, where alpha * dloss * (p - 1)
// would be rounded.  c comes from expm1, so a p close to 1 costs no digits; a c below 2^-25, where
// fp32 cannot tell p from 1, is raised to it.
//
// Distillation: row i of D is p, and p - (sum of q over the entries that name the same vocabulary
// row) at the entries.  bf16: times s, with X and the product as they are, so that dW's factors are
// rounded once (D) and not twice; fp32 (D_APART): s enters with X and the product.
//
// D_WHOLE, for few tokens, whose D is kept wide: both operators' rows are s * (p - y), and X and the
// product enter as they are.
__global__ void __launch_bounds__(256) vocab_rows_kernel(Entries e, int tokens, int vocab, float alpha,
                                                         const int* pos, const float* lse, const float* dloss,
                                                         const float* z, float* lse_c, float* scale, float* out_scale,
                                                         float* value, DForm form) {
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
        sc = !good ? NAN : form == D_WHOLE ? s : 1.f / c;
        os = !good ? NAN : form == D_WHOLE ? 1.f : s * c;
        if (lane == 0) value[t] = form == D_WHOLE ? -s * c : -1.f;
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
                d = (form == D_APART ? 1.f : s) * (expf(z[t * e.k + k] - l) - q);
            }
            value[t * e.k + k] = d;
        }
        sc = __all(good) ? (form == D_APART ? 1.f : s) : NAN;
        os = form == D_APART ? s : 1.f;
    }
    if (lane == 0) {
        lse_c[i] = l;
        scale[i] = sc;
        out_scale[i] = os;
    }
}

// Puts the entries' values into D where they fall into this piece (P = 0: a D in fp32).
template <int P>
__global__ void __launch_bounds__(256) vocab_patch_kernel(Entries e, int tokens, int v0, int vocab, const int* pos,
                                                          const float* value, const float* weight,
                                                          const float* x_unit, const float* x_most, char* d,
                                                          long d_pitch) {
    const long j = (long)blockIdx.x * 256 + threadIdx.x;
    if (j >= (long)tokens * e.k) return;
    const long t = j / e.k, k = j - t * e.k;
    const int i = pos[t];
    const i64 v = e.index[t * e.ld + k];
    if (i < 0 || !e.counts(v) || v < v0 || v >= v0 + vocab) return;
    if constexpr (P == 0) {
        ((float*)(d + (size_t)i * d_pitch))[v - v0] = value[j];
        return;
    }
    const float f = P == 2 ? d_factor(weight[i], x_unit[i], *x_most) : 1.f;
    store1<P == 2 ? 2 : 1>(d + (size_t)i * d_pitch, v - v0, value[j] * f);
}

// dX of every token: the sum of its product's parts, or 0 where it does not count.
template <typename T, int P>
__global__ void __launch_bounds__(256) vocab_dx_out_kernel(const int* pos, const int* count, int hidden,
                                                           const float* acc, DxCut cut, int hp, const float* weight,
                                                           const float* x_unit, const float* x_most, T* dx, long ld) {
    const int t = blockIdx.x, i = pos[t], splits = cut.splits(*count);
    const size_t rows = cut.rows(*count);
    float s = 0.f;
    if (i >= 0) s = P == 1 ? weight[i] : *x_most / (x_unit[i] * kDScale);
    for (int h = threadIdx.x * 4; h < hidden; h += 1024) {
        f32x4 v = {};
        if (i >= 0)
            for (int z = 0; z < splits; ++z) v += *(const f32x4*)(acc + (z * rows + i) * hp + h);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (h + q < hidden) dx[(size_t)t * ld + h + q] = (T)(v[q] * s);
    }
}

}  // namespace vocab
}  // namespace libsgemm
