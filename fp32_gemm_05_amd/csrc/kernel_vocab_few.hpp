// kernel_vocab_few.hpp -- the products of the vocabulary-head operators for at most 64 tokens.
//
// With few tokens every product is one pass over W (or dW): 2 * tokens / sizeof(W) operations a
// byte.  So W goes from memory straight into the MFMA operands, whatever its alignment, with no
// packing pass; the tokens' side, a few hundred KB at most, comes from the caches.  Tokens that do not
// count keep their place: their columns are computed and left out at the end.  bf16 is multiplied with v_mfma_f32_16x16x32_bf16, fp32 with
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
    typedef T Row __attribute__((ext_vector_type(E), aligned(sizeof(T))));  // E values in memory, at any alignment
    // dW's hidden: rows 4 g + i of the F blocks of a group are hidden 16 F * group + 4 F g + 4 f + i, so
    // that a lane ends with E consecutive ones.
    static constexpr int F = E / 4;
    static __host__ __device__ constexpr int hidden_of(int hb, int row) {
        return 16 * F * (hb / F) + 4 * F * (row >> 2) + 4 * (hb % F) + (row & 3);
    }
    // c[m][b] += a[m] b[b] over a step; the products of one c stand apart, none waits for the one before.
    template <int M, int B>
    static __device__ inline void mma(const V (&a)[M], const V (&b)[B], f32x4 (&c)[M][B]) {
#pragma unroll
        for (int s = 0; s < (sizeof(T) == 2 ? 1 : 4); ++s)
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if constexpr (sizeof(T) == 2)
                        c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], c[i][j], 0, 0, 0);
                    else
                        c[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][s], b[j][s], c[i][j], 0, 0, 0);
    }
};

// D's values as operands: fp32 as they are (PARTS 1), or as bf16 low and high.
template <typename T>
struct Wide {
    static constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    // Element i of the parts.
    static __device__ inline void set(typename Chunk<T>::V (&v)[PARTS], int i, float x) {
        const T high = (T)x;
        v[PARTS - 1][i] = high;
        if constexpr (PARTS == 2) v[0][i] = __builtin_isfinite(x) ? (T)(x - (float)high) : (T)0.f;
    }
};

// Distillation's work on the entries, four waves a workgroup (token_wave).
template <typename T, bool GRAD>
__global__ void __launch_bounds__(256) vocab_few_token_kernel(TokenArgs a) {
    token_wave<T, GRAD>(a, (long)blockIdx.x * 4 + (threadIdx.x >> 6));
}

struct FewArgs {
    Entries e;
    int tokens;
    const void *x, *w;
    long ldx, ldw;
    int vocab, hidden, groups;  // of this piece; workgroups for its logits
    int whole_vocab;
    float alpha;
    i64 v0;                     // first vocabulary row of this piece
    float2* part;               // forward: [workgroup][kFewTokens]
    float* z;                   // forward, cross entropy: the target's logit
    // gradient, per token: D = exp(z - lse) * scale; cross entropy: scale = alpha * dloss
    const float *lse, *dloss, *scale;
    float* d;                   // [token][vp]
    long vp;
    // gradient, dW wanted, first piece: X in the order in which dW's product takes it, chunk
    // (hb * kt + j) * 64 + lane: hidden_of(hb, lane % 16), tokens from j * STEP + lane / 16 * E
    char* xtf;
    int kt, xtf_chunks;
};

// One chunk of xtf; the tokens that do not count are zeros.
template <typename T>
__device__ inline void few_transpose(const FewArgs& a, int i) {
    typedef Chunk<T> C;
    if (i >= a.xtf_chunks) return;
    const int lane = i & 63, j = (i >> 6) % a.kt, hb = (i >> 6) / a.kt;
    const int h = C::hidden_of(hb, lane & 15), t = j * C::STEP + (lane >> 4) * C::E;
    typename C::V v = {};
#pragma unroll
    for (int q = 0; q < C::E; ++q)
        if (t + q < a.tokens && h < a.hidden && any_entry(a.e, t + q, 0)) v[q] = ((const T*)a.x)[(t + q) * a.ldx + h];
    *(typename C::V*)(a.xtf + 16L * i) = v;
}

// z of 16 MR vocabulary rows and all tokens.  The four waves of a workgroup take every fourth U steps
// of the hidden size each, so that even a small vocabulary keeps many loads in flight, and add up in
// LDS; 16 B chunks of a row make 64-byte runs a step, U of them in a row.
template <typename T, int NB, bool GRAD>
__global__ void __launch_bounds__(256) vocab_few_logits_kernel(FewArgs a) {
    typedef Chunk<T> C;
    typedef typename C::V V;
    constexpr int MR = NB == 4 ? 4 : 2, U = NB == 4 ? 2 : 4;
    // all loads before the first MFMA, where the compiler would keep too few in flight; the long fp32 runs
    // of NB > 1 do better with loads between them
    constexpr bool HOLD = sizeof(T) == 2 || NB == 1;
    __shared__ f32x4 sums[4][NB][64];
    if (GRAD && (int)blockIdx.x >= a.groups)
        return few_transpose<T>(a, ((int)blockIdx.x - a.groups) * 256 + (int)threadIdx.x);
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int r0 = blockIdx.x * 16 * MR;
    const T* w[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) w[m] = (const T*)a.w + (size_t)imin(r0 + 16 * m + l, a.vocab - 1) * a.ldw + g * C::E;
    const T* x[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = (const T*)a.x + imin(16 * b + l, a.tokens - 1) * a.ldx + g * C::E;
    f32x4 acc[MR][NB];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int full = a.hidden / C::STEP;  // steps without an end of the rows
    const int groups = full / U;  // of U steps; this wave's are wave, wave + 4, ..
    for (int q = wave; q < groups; q += 4) {
        V vw[U][MR], vx[U][NB];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const T* p = w[m] + (size_t)q * U * C::STEP;
#pragma unroll
            for (int u = 0; u < U; ++u) vw[u][m] = C::load(p + u * C::STEP);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const T* p = x[b] + (size_t)q * U * C::STEP;
#pragma unroll
            for (int u = 0; u < U; ++u) vx[u][b] = C::load(p + u * C::STEP);
        }
        if (HOLD) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) C::mma(vw[u], vx[u], acc);
    }
    for (int s = groups * U + wave; s < full; s += 4) {
        V vw[MR], vx[NB];
#pragma unroll
        for (int m = 0; m < MR; ++m) vw[m] = C::load(w[m] + (size_t)s * C::STEP);
#pragma unroll
        for (int b = 0; b < NB; ++b) vx[b] = C::load(x[b] + (size_t)s * C::STEP);
        C::mma(vw, vx, acc);
    }
    if (full * C::STEP < a.hidden && wave == 3) {
        const int n = a.hidden - full * C::STEP - g * C::E;  // elements of this lane's chunk, maybe none
        V vw[MR], vx[NB];
#pragma unroll
        for (int m = 0; m < MR; ++m) vw[m] = C::load(w[m] + (size_t)full * C::STEP, n);
#pragma unroll
        for (int b = 0; b < NB; ++b) vx[b] = C::load(x[b] + (size_t)full * C::STEP, n);
        C::mma(vw, vx, acc);
    }
    // wave b gets the sums of tokens 16 b + l, vocabulary rows r0 + 16 m + 4 g + i
    f32x4 z[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        if (m > 0) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[wave][b][lane] = acc[m][b];
        __syncthreads();
        if (wave < NB) z[m] = sums[0][wave][lane] + sums[1][wave][lane] + sums[2][wave][lane] + sums[3][wave][lane];
    }
    if (wave >= NB) return;
    const int n = 16 * wave + l;
    if (n >= a.tokens && !GRAD) return;
    const bool live = n < a.tokens && any_entry(a.e, n, 0);
    // cross entropy: the target's row of this piece, or a row that none has
    i64 entry = -1;
    if (!a.e.teacher && live) {
        entry = a.e.index[n] - a.v0;
        if (entry < 0 || entry >= a.vocab) entry = -1;
    }
    if constexpr (GRAD) {
        float lse = 0.f, scale = 0.f;
        if (live) {
            lse = a.lse[n];
            scale = a.e.teacher ? a.scale[n] : a.alpha * a.dloss[n];
            // a target outside the vocabulary: NaN, as its loss is
            if (!a.e.teacher && (a.e.index[n] < 0 || a.e.index[n] >= a.whole_vocab)) scale = NAN;
        }
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const int v = r0 + 16 * m + 4 * g;
            f32x4 d;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = z[m][i] * a.alpha - lse;
                d[i] = live && v + i < a.vocab ? (v + i == entry ? expm1f(y) : __expf(y)) * scale : 0.f;
            }
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
                if (r0 + 16 * m + 4 * g + i == entry) a.z[n] = x;
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

struct FewGradArgs {
    const float* d;
    long vp;
    int tokens, vocab, hidden;
    // dX: `strips` of 16 E hidden, each in `splits` parts of the vocabulary
    const void* w;
    long ldw;
    int strips, splits;
    float* acc;  // [splits][16 NB][hp]
    int hp, add;
    // dW: workgroups of 256 vocabulary rows by `groups` groups of 128 bytes of them
    const char* xtf;
    int groups, row_groups;
    void* out;
    long ld;
};

// dW of 256 vocabulary rows, 64 a wave, and `groups` groups of 128 bytes along them: a wave holds D of
// its rows and passes over the groups.  Bound by the stores, which leave in whole lines at once: lines
// that stay open while the next operand is loaded are more than the L2 holds.
template <typename T, int NB>
__device__ inline void few_dw(const FewGradArgs& a, int block) {
    typedef Chunk<T> C;
    typedef typename C::V V;
    constexpr int KT = (16 * NB + C::STEP - 1) / C::STEP;
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int v0 = block % a.row_groups * 256 + (threadIdx.x >> 6) * 64;
    if (v0 >= a.vocab) return;
    constexpr int PARTS = Wide<T>::PARTS;
    V d[KT][4][PARTS];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int q = 0; q < C::E; ++q) {
                const int t = j * C::STEP + g * C::E + q, v = v0 + 16 * b + l;
                Wide<T>::set(d[j][b], q, t < a.tokens && v < a.vocab ? a.d[t * a.vp + v] : 0.f);
            }
    constexpr int F = C::F, HB = 2 * F;  // blocks of a group
    const int first = block / a.row_groups * a.groups, last = imin(first + a.groups, (a.hidden + 16 * HB - 1) / (16 * HB));
    for (int q = first; q < last; ++q) {
        V x[KT][HB];
        f32x4 c[HB][4] = {};
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int f = 0; f < HB; ++f) x[j][f] = ((const V*)a.xtf)[((q * HB + f) * KT + j) * 64 + lane];
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const V y[4] = {d[j][0][p], d[j][1][p], d[j][2][p], d[j][3][p]};
                C::mma(x[j], y, c);
            }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int v = v0 + 16 * b + l;
            if (v >= a.vocab) continue;
            T* out = (T*)a.out + (size_t)v * a.ld;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int h = 16 * F * (2 * q + s) + C::E * g;
                typename C::Row o;
#pragma unroll
                for (int i = 0; i < C::E; ++i) o[i] = (T)c[s * F + i / 4][b][i % 4];
                if (h + C::E <= a.hidden)
                    *(typename C::Row*)(out + h) = o;
                else
#pragma unroll
                    for (int i = 0; i < C::E; ++i)
                        if (h + i < a.hidden) out[h + i] = o[i];
            }
        }
    }
}

// dX of 16 E hidden over a part of the vocabulary.  A lane's chunks are E consecutive hidden of E
// rows of W; element e of the chunks makes the operand of the e-th 16 hidden, h0 + E * (lane % 16) + e.
// The four waves take every fourth step of the part and add up in LDS.
template <typename T, int NB>
__device__ inline void few_dx(const FewGradArgs& a, int block) {
    typedef Chunk<T> C;
    typedef typename C::V V;
    constexpr int E = C::E;
    __shared__ f32x4 sums[4][E][64];
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int h0 = block % a.strips * 16 * E, h = h0 + l * E, n = a.hidden - h;
    const int steps = (a.vocab + C::STEP - 1) / C::STEP, z = block / a.strips;
    const int first = (int)((long)steps * z / a.splits), last = (int)((long)steps * (z + 1) / a.splits);
    constexpr int PARTS = Wide<T>::PARTS, U = 8 / E;
    f32x4 acc[E][NB] = {};
    const T* w = (const T*)a.w + h;
    auto load = [&](int s0, V (&rows)[U][E], f32x4 (&x)[U][NB][E / 4]) {
        // D is 0 past the vocabulary, where the last row stands in, but not past this part
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = (s0 + u) * C::STEP + g * E;
#pragma unroll
            for (int q = 0; q < E; ++q) {
                const T* p = w + (size_t)imin(v + q, a.vocab - 1) * a.ldw;
                rows[u][q] = n >= E ? C::load(p) : C::load(p, n);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int q = 0; q < E / 4; ++q)
                    x[u][b][q] = s0 + u < last ? ((const f32x4*)(a.d + (16 * b + l) * a.vp + (s0 + u) * C::STEP + g * E))[q]
                                               : f32x4{0.f, 0.f, 0.f, 0.f};
        if (sizeof(T) == 2 || NB == 1) __builtin_amdgcn_sched_barrier(0);  // as above
    };
    auto multiply = [&](const V (&rows)[U][E], const f32x4 (&x)[U][NB][E / 4]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            V d[NB][PARTS], t[E];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int q = 0; q < E; ++q) Wide<T>::set(d[b], q, x[u][b][q / 4][q % 4]);
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int q = 0; q < E; ++q) t[e][q] = rows[u][q][e];
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                V y[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) y[b] = d[b][p];
                C::mma(t, y, acc);
            }
        }
    };
    for (int s = first + wave * U; s < last; s += 4 * U) {
        V rows[U][E];
        f32x4 x[U][NB][E / 4];
        load(s, rows, x);
        multiply(rows, x);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b > 0) __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) sums[wave][e][lane] = acc[e][b];
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

// Both gradients' products, in one launch: they need D alone.  strips = 0: no dX.
template <typename T, int NB>
__global__ void __launch_bounds__(256) vocab_few_grad_kernel(FewGradArgs a) {
    const int dx = a.strips * a.splits;
    if ((int)blockIdx.x < dx)
        few_dx<T, NB>(a, blockIdx.x);
    else
        few_dw<T, NB>(a, (int)blockIdx.x - dx);
}

}  // namespace vocab
}  // namespace libsgemm
