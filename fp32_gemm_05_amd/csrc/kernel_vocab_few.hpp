// kernel_vocab_few.hpp -- the products of the vocabulary-head operators for at most 64 tokens.
//
// With few tokens every product is one pass over W (or dW): 2 * tokens / sizeof(W) operations a
// byte.  So W goes from memory straight into the MFMA operands, whatever its alignment, with no
// packing pass; the tokens' side, a few hundred KB at most, comes from the caches in the order in
// which the lanes want it.  bf16 is multiplied with v_mfma_f32_16x16x32_bf16, fp32 with
// v_mfma_f32_16x16x4_f32: at 64 tokens the fp32 rate and the memory's are about even, below that
// memory bounds both.  D is kept in fp32, and with bf16 operands enters its products as the sum of
// two bf16 values (16 bits), which costs no time here.
//
// A "chunk" is 16 bytes: E consecutive elements that one lane loads.  A step is the 4 E elements
// along k that the four lane groups hold: one bf16 MFMA, or four fp32 MFMAs of which the s-th takes
// the s-th element of every lane's chunk (any order of k will do that both operands share).
#pragma once

#include "kernel_vocab_rows.hpp"

namespace libsgemm {
namespace vocab {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kFewTokens = 64;

template <typename T>
struct Chunk {
    static constexpr int E = 16 / sizeof(T), STEP = 4 * E;
    typedef T V __attribute__((ext_vector_type(E)));
    // E elements at p, at any alignment of T.
    static __device__ inline V load(const T* p) {
        V v;
        __builtin_memcpy(&v, p, 16);
        return v;
    }
    // The first n of them (n < E: the others are not read and are 0).
    static __device__ inline V load(const T* p, int n) {
        if (n >= E) return load(p);
        V v = {};
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n) v[i] = p[i];
        return v;
    }
    static __device__ inline f32x4 mma(V a, V b, f32x4 c) {
        if constexpr (sizeof(T) == 2) {
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
            return c;
        }
    }
};

// D's values as operands: fp32 as they are, or as bf16 high and low.
template <typename T>
struct Wide {
    typename Chunk<T>::V v[sizeof(T) == 2 ? 2 : 1];
    __device__ inline void set(int i, float x) {
        v[0][i] = (T)x;
        if constexpr (sizeof(T) == 2) v[1][i] = __builtin_isfinite(x) ? (T)(x - (float)v[0][i]) : (T)0.f;
    }
    static __device__ inline f32x4 mma(typename Chunk<T>::V a, const Wide& b, f32x4 c) {
        if constexpr (sizeof(T) == 2) c = Chunk<T>::mma(a, b.v[1], c);
        return Chunk<T>::mma(a, b.v[0], c);
    }
};

struct FewPrepArgs {
    Entries e;
    int tokens, nb, kt, hidden;
    int *rows, *pos, *count;
    float *loss, *lse;  // forward: 0 for the tokens that do not count
    char* xf;           // chunk (step * nb + b) * 64 + lane: token 16 b + lane % 16, hidden from step * STEP + lane / 16 * E
    char* xtf;          // chunk (hb * kt + j) * 64 + lane: hidden 16 hb + lane % 16, tokens from j * STEP + lane / 16 * E
    int xf_chunks, xtf_chunks;
};

// Which of at most 64 tokens count, and their rows of X in the two orders of chunks above.
template <typename T>
__global__ void __launch_bounds__(256) vocab_few_prep_kernel(FewPrepArgs a, const T* x, long ldx) {
    typedef Chunk<T> C;
    __shared__ int rows[kFewTokens], counted;
    if (threadIdx.x < 64) {
        const int t = threadIdx.x;
        bool live = false;
        for (int k = 0; k < a.e.k && t < a.tokens && !live; ++k) live = a.e.counts(a.e.index[(size_t)t * a.e.ld + k]);
        const unsigned long long m = __ballot(live);
        const int at = __popcll(m & ((1ull << t) - 1));
        if (live) rows[at] = t;
        if (t == 0) counted = __popcll(m);
        if (blockIdx.x == 0) {
            if (t < a.tokens) a.pos[t] = live ? at : -1;
            if (live) a.rows[at] = t;
            if (t == 0) *a.count = __popcll(m);
            if (a.loss && t < a.tokens && !live) a.loss[t] = a.lse[t] = 0.f;
        }
    }
    __syncthreads();
    const int n = counted;
    int i = blockIdx.x * 256 + threadIdx.x;
    typename C::V v = {};
    if (i < a.xf_chunks) {
        const int lane = i & 63, b = (i >> 6) % a.nb, step = (i >> 6) / a.nb;
        const int t = 16 * b + (lane & 15), k = step * C::STEP + (lane >> 4) * C::E;
        if (t < n && k < a.hidden) v = C::load(x + rows[t] * ldx + k, a.hidden - k);
        *(typename C::V*)(a.xf + 16L * i) = v;
    } else if ((i -= a.xf_chunks) < a.xtf_chunks) {
        const int lane = i & 63, j = (i >> 6) % a.kt, hb = (i >> 6) / a.kt;
        const int h = 16 * hb + (lane & 15), t = j * C::STEP + (lane >> 4) * C::E;
#pragma unroll
        for (int q = 0; q < C::E; ++q)
            if (t + q < n && h < a.hidden) v[q] = x[rows[t + q] * ldx + h];
        *(typename C::V*)(a.xtf + 16L * i) = v;
    }
}

struct FewArgs {
    const void* w;
    long ldw;
    int vocab, hidden;
    const char* xf;
    const int* count;
    float alpha;
    float2* part;        // forward: [workgroup][kFewTokens]
    const float* lse;    // gradient: per counted token
    const float* scale;
    float* d;            // gradient: [token][vp]
    long vp;
};

// z of 16 MR vocabulary rows and all tokens.  The four waves of a workgroup take every fourth U steps
// of the hidden size each, so that even a small vocabulary keeps many loads in flight, and add up in
// LDS; 16 B chunks of a row make 64-byte runs a step, U of them in a row.
template <typename T, int NB, bool GRAD>
__global__ void __launch_bounds__(256) vocab_few_logits_kernel(FewArgs a) {
    typedef Chunk<T> C;
    typedef typename C::V V;
    constexpr int MR = NB == 4 ? 4 : 2, U = NB == 4 ? 2 : 4;
    __shared__ f32x4 sums[4][MR * NB][64];
    const int count = *a.count;
    if (count == 0) return;
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int r0 = blockIdx.x * 16 * MR;
    const T* w[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) w[m] = (const T*)a.w + (size_t)imin(r0 + 16 * m + l, a.vocab - 1) * a.ldw + g * C::E;
    const V* xf = (const V*)a.xf + lane;
    f32x4 acc[MR][NB];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int full = a.hidden / C::STEP;  // steps without an end of the rows
    for (int s0 = wave * U; s0 < full; s0 += 4 * U) {
        if (s0 + U <= full) {
            V vw[U][MR], vx[U][NB];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int m = 0; m < MR; ++m) vw[u][m] = C::load(w[m] + (size_t)(s0 + u) * C::STEP);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int b = 0; b < NB; ++b) vx[u][b] = xf[((s0 + u) * NB + b) * 64];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int m = 0; m < MR; ++m)
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[m][b] = C::mma(vw[u][m], vx[u][b], acc[m][b]);
        } else {
            for (int s = s0; s < full; ++s) {
                V vw[MR];
#pragma unroll
                for (int m = 0; m < MR; ++m) vw[m] = C::load(w[m] + (size_t)s * C::STEP);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const V vx = xf[(s * NB + b) * 64];
#pragma unroll
                    for (int m = 0; m < MR; ++m) acc[m][b] = C::mma(vw[m], vx, acc[m][b]);
                }
            }
        }
    }
    if (full * C::STEP < a.hidden && wave == 3) {
        const int n = a.hidden - full * C::STEP - g * C::E;  // elements of this lane's chunk, maybe none
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const V vw = C::load(w[m] + (size_t)full * C::STEP, n);
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[m][b] = C::mma(vw, xf[(full * NB + b) * 64], acc[m][b]);
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[wave][m * NB + b][lane] = acc[m][b];
    __syncthreads();
    if (wave >= NB) return;
    // wave b: tokens 16 b + l, vocabulary rows r0 + 16 m + 4 g + i
    const int n = 16 * wave + l;
    f32x4 z[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        z[m] = sums[0][m * NB + wave][lane];
#pragma unroll
        for (int y = 1; y < 4; ++y) z[m] += sums[y][m * NB + wave][lane];
    }
    if constexpr (GRAD) {
        const bool live = n < count;
        const float lse = live ? a.lse[n] : 0.f, scale = live ? a.scale[n] : 0.f;
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const int v = r0 + 16 * m + 4 * g;
            f32x4 d;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[i] = live && v + i < a.vocab ? __expf(z[m][i] * a.alpha - lse) * scale : 0.f;
            *(f32x4*)(a.d + n * a.vp + v) = d;
        }
    } else {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = r0 + 16 * m + 4 * g + i < a.vocab ? z[m][i] * a.alpha : -INFINITY;
                z[m][i] = x;
                top = x > top || x != x ? x : top;  // a NaN stays
            }
#pragma unroll
        for (int o = 16; o < 64; o *= 2) {
            const float other = __shfl_xor(top, o);
            top = other > top || other != other ? other : top;
        }
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += __expf(z[m][i] - ref);
#pragma unroll
        for (int o = 16; o < 64; o *= 2) sum += __shfl_xor(sum, o);
        if (g == 0) a.part[(size_t)blockIdx.x * kFewTokens + n] = make_float2(top, sum);
    }
}

struct FewDwArgs {
    const char* xtf;
    const int* count;
    const float* d;
    long vp;
    int vocab, hidden, blocks;  // blocks of 16 hidden per workgroup
    void* out;
    long ld;
    int vec;
};

// dW of 256 vocabulary rows, 64 a wave, and `blocks` blocks of 16 hidden: a wave holds D of its rows
// and passes over the hidden blocks; bound by the stores.
template <typename T, int NB>
__global__ void __launch_bounds__(256) vocab_few_dw_kernel(FewDwArgs a) {
    typedef Chunk<T> C;
    typedef typename C::V V;
    typedef T T4 __attribute__((ext_vector_type(4)));
    constexpr int KT = (16 * NB + C::STEP - 1) / C::STEP;
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int v0 = blockIdx.x * 256 + (threadIdx.x >> 6) * 64;
    if (v0 >= a.vocab) return;
    const int count = *a.count;
    Wide<T> d[4][KT];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int q = 0; q < C::E; ++q) {
                const int t = j * C::STEP + g * C::E + q, v = v0 + 16 * b + l;
                d[b][j].set(q, t < count && v < a.vocab ? a.d[t * a.vp + v] : 0.f);
            }
    const int h_end = imin((int)(blockIdx.y + 1) * a.blocks, (a.hidden + 15) / 16);
    for (int hb = blockIdx.y * a.blocks; hb < h_end; ++hb) {
        V x[KT];
#pragma unroll
        for (int j = 0; j < KT; ++j) x[j] = ((const V*)a.xtf)[(hb * KT + j) * 64 + lane];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KT; ++j) c = Wide<T>::mma(x[j], d[b][j], c);
            const int v = v0 + 16 * b + l, h = 16 * hb + 4 * g;
            if (v >= a.vocab) continue;
            T* out = (T*)a.out + (size_t)v * a.ld + h;
            if (a.vec) {
                if (h < a.hidden) *(T4*)out = T4{(T)c[0], (T)c[1], (T)c[2], (T)c[3]};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (h + i < a.hidden) out[i] = (T)c[i];
            }
        }
    }
}

struct FewDxArgs {
    const void* w;
    long ldw;
    int vocab, hidden, splits;
    const int* count;
    const float* d;
    long vp;
    float* acc;  // [splits][16 NB][hp]
    int hp, add;
};

// dX of 16 E hidden over a part of the vocabulary.  A lane's chunks are E consecutive hidden of E
// rows of W; element e of the chunks makes the operand of the e-th 16 hidden, h0 + E * (lane % 16) + e.
// The four waves take every fourth step of the part and add up in LDS.
template <typename T, int NB>
__global__ void __launch_bounds__(256) vocab_few_dx_kernel(FewDxArgs a) {
    typedef Chunk<T> C;
    typedef typename C::V V;
    constexpr int E = C::E;
    __shared__ f32x4 sums[4][E][64];
    if (*a.count == 0) return;
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int h0 = blockIdx.x * 16 * E, h = h0 + l * E, n = a.hidden - h;
    const int steps = (a.vocab + C::STEP - 1) / C::STEP, z = blockIdx.y;
    const int first = (int)((long)steps * z / a.splits), last = (int)((long)steps * (z + 1) / a.splits);
    f32x4 acc[NB][E];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[b][e] = f32x4{0.f, 0.f, 0.f, 0.f};
    const T* w = (const T*)a.w + h;
    for (int s = first + wave; s < last; s += 4) {
        const int v = s * C::STEP + g * E;
        V rows[E];
#pragma unroll
        for (int q = 0; q < E; ++q) {
            // D is 0 past the vocabulary, where the last row stands in
            const T* p = w + (size_t)imin(v + q, a.vocab - 1) * a.ldw;
            rows[q] = n >= E ? C::load(p) : C::load(p, n);
        }
        Wide<T> d[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float* p = a.d + (16 * b + l) * a.vp + v;
#pragma unroll
            for (int q = 0; q < E; q += 4) {
                const f32x4 x = *(const f32x4*)(p + q);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[b].set(q + i, x[i]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            V x;
#pragma unroll
            for (int q = 0; q < E; ++q) x[q] = rows[q][e];
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[b][e] = Wide<T>::mma(x, d[b], acc[b][e]);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b > 0) __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) sums[wave][e][lane] = acc[b][e];
        __syncthreads();
        // element i of block e: token 16 b + l, hidden h0 + E * (4 g + i) + e
        float* out = a.acc + ((size_t)z * 16 * NB + 16 * b + l) * a.hp + h0 + E * 4 * g;
#pragma unroll
        for (int e = wave; e < E; e += 4) {
            f32x4 c = sums[0][e][lane];
#pragma unroll
            for (int y = 1; y < 4; ++y) c += sums[y][e][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float* p = out + E * i + e;
                *p = a.add ? *p + c[i] : c[i];
            }
        }
    }
}

}  // namespace vocab
}  // namespace libsgemm
