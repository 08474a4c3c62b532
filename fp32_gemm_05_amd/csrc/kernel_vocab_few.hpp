// kernel_vocab_few.hpp -- the products of the vocabulary-head operators for at most 64 tokens.
//
// With few tokens every product is one pass over W (or dW): 2 * tokens / sizeof(W) operations a
// byte.  So W goes from memory straight into the MFMA operands, whatever its alignment, with no
// packing pass; the tokens' side, a few hundred KB at most, comes from the caches.  Tokens that do not
// count keep their place: their columns are computed and left out at the end.
//
// Three ways to multiply.  Bf16: v_mfma_f32_16x16x32_bf16; D, kept in fp32, enters its products as two
// bf16 values (16 bits), which costs no time here.  Fp32: v_mfma_f32_16x16x4_f32, exact products; at
// more than 16 tokens its rate, not the memory's, would bound, so there Fp32Split cuts each value into
// three bf16 parts on the way (24 bits; of values from 2^-110 to 2^127, where the parts neither vanish nor
// round up to infinity) and takes the six products above 2^-24 of the whole: 384 cycles
// a 2 KB of W instead of 1024.
//
// A "chunk" is E consecutive elements along k in one lane.  A step is the 4 E elements that the four
// lane groups hold: one MFMA of 32 k, or four of 4 k of which the s-th takes the s-th element of every
// lane's chunk (any order of k will do that both operands share).
#pragma once

#include "kernel_vocab_rows.hpp"

namespace libsgemm {
namespace vocab {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kFewTokens = 64;

// What the three share.  T_: the type in memory, E_: elements of a chunk.
template <typename T_, int E_>
struct FewMode {
    typedef T_ T;
    static constexpr int E = E_, STEP = 4 * E, HE = 16 / sizeof(T);  // HE: elements of 16 bytes
    typedef T Raw __attribute__((ext_vector_type(E)));
    typedef T Quad __attribute__((ext_vector_type(HE)));
    typedef T Row __attribute__((ext_vector_type(HE), aligned(sizeof(T))));  // in memory, at any alignment
    // A V of elements at p, at any alignment of T.
    template <typename V>
    static __device__ inline V load(const T* p) {
        V v;
        __builtin_memcpy(&v, p, sizeof(V));
        return v;
    }
    // The first n of them (the others are not read and are 0).
    template <typename V>
    static __device__ inline V load(const T* p, int n) {
        constexpr int N = sizeof(V) / sizeof(T);
        if (n >= N) return load<V>(p);
        V v = {};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) v[i] = p[i];
        return v;
    }
    // dW's hidden: rows 4 g + i of the F blocks of a group are hidden 16 F * group + 4 F g + 4 f + i, so
    // that a lane ends with HE consecutive ones.
    static constexpr int F = HE / 4;
    static __host__ __device__ constexpr int hidden_of(int hb, int row) {
        return 16 * F * (hb / F) + 4 * F * (row >> 2) + 4 * (hb % F) + (row & 3);
    }
};
// Each has P parts of a chunk of X or W and DP of one of D, the most significant first.
struct Bf16 : FewMode<__bf16, 8> {
    typedef bf16x8 Part;
    static constexpr int P = 1, DP = 2;
    static __device__ inline void parts(Raw x, Part (&v)[1]) { v[0] = x; }
    static __device__ inline void parts(const float (&x)[8], Part (&v)[2]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[0][i] = (__bf16)x[i];
            v[1][i] = __builtin_isfinite(x[i]) ? (__bf16)(x[i] - (float)v[0][i]) : (__bf16)0.f;
        }
    }
    static __device__ inline f32x4 mma(Part a, Part b, f32x4 c, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static constexpr int MMAS = 1;
};
struct Fp32 : FewMode<float, 4> {
    typedef f32x4 Part;
    static constexpr int P = 1, DP = 1;
    static __device__ inline void parts(Raw x, Part (&v)[1]) { v[0] = x; }
    static __device__ inline void parts(const float (&x)[4], Part (&v)[1]) { v[0] = Part{x[0], x[1], x[2], x[3]}; }
    static __device__ inline f32x4 mma(Part a, Part b, f32x4 c, int s) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    }
    static constexpr int MMAS = 4;
};
struct Fp32Split : FewMode<float, 8> {
    typedef bf16x8 Part;
    static constexpr int P = 3, DP = 3;
    static __device__ inline void parts(const float (&x)[8], Part (&v)[3]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[0][i] = (__bf16)x[i];
            const float r = x[i] - (float)v[0][i];
            v[1][i] = (__bf16)r;
            v[2][i] = (__bf16)(r - (float)v[1][i]);
        }
    }
    static __device__ inline void parts(Raw x, Part (&v)[3]) {
        const float f[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
        parts(f, v);
    }
    static __device__ inline f32x4 mma(Part a, Part b, f32x4 c, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static constexpr int MMAS = 1;
};
// c[i] += a[i] b over a step, the smallest products first; those of one c stand apart.
template <class M, int PA, int PB, int N>
__device__ inline void few_mma(const typename M::Part (&a)[N][PA], const typename M::Part (&b)[PB], f32x4* const (&c)[N]) {
#pragma unroll
    for (int w = PA == 3 ? 2 : PA + PB - 2; w >= 0; --w)
#pragma unroll
        for (int p = 0; p < PA; ++p)
            if (w - p >= 0 && w - p < PB)
#pragma unroll
                for (int s = 0; s < M::MMAS; ++s)
#pragma unroll
                    for (int i = 0; i < N; ++i) *c[i] = M::mma(a[i][p], b[w - p], *c[i], s);
}

// c[i] += a b[i] the same way.
template <class M, int PA, int PB, int N>
__device__ inline void few_mma_t(const typename M::Part (&a)[PA], const typename M::Part (&b)[N][PB], f32x4* const (&c)[N]) {
#pragma unroll
    for (int w = PA == 3 ? 2 : PA + PB - 2; w >= 0; --w)
#pragma unroll
        for (int p = 0; p < PA; ++p)
            if (w - p >= 0 && w - p < PB)
#pragma unroll
                for (int s = 0; s < M::MMAS; ++s)
#pragma unroll
                    for (int i = 0; i < N; ++i) *c[i] = M::mma(a[p], b[i][w - p], *c[i], s);
}

// Distillation's work on the entries, four waves a workgroup (token_wave).
template <typename T, bool GRAD>
__global__ void __launch_bounds__(256) vocab_few_token_kernel(TokenArgs a) {
    for (long i = (long)blockIdx.x * 4 + (threadIdx.x >> 6); i < a.waves; i += (long)gridDim.x * 4) token_wave<T, GRAD>(a, i);
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
template <class C>
__device__ inline void few_transpose(const FewArgs& a, int i) {
    typedef typename C::T T;
    if (i >= a.xtf_chunks) return;
    const int lane = i & 63, j = (i >> 6) % a.kt, hb = (i >> 6) / a.kt;
    const int h = C::hidden_of(hb, lane & 15), t = j * C::STEP + (lane >> 4) * C::E;
    typename C::Raw v = {};
#pragma unroll
    for (int q = 0; q < C::E; ++q)
        if (t + q < a.tokens && h < a.hidden && any_entry(a.e, t + q, 0)) v[q] = ((const T*)a.x)[(t + q) * a.ldx + h];
    ((typename C::Raw*)a.xtf)[i] = v;
}

// z of 16 MR vocabulary rows and all tokens.  The four waves of a workgroup take every fourth U steps
// of the hidden size each, so that even a small vocabulary keeps many loads in flight, and add up in
// LDS; 16 B chunks of a row make 64-byte runs a step, U of them in a row.
template <class C, int NB, int MR, bool GRAD>
__global__ void __launch_bounds__(256) vocab_few_logits_kernel(FewArgs a) {
    typedef typename C::T T;
    typedef typename C::Raw Raw;
    typedef typename C::Part Part;
    // steps whose loads are held in registers at once
    constexpr int U = C::P == 3 ? (NB == 4 && MR == 2 ? 2 : 1) : MR == 4 ? 2 : 4;
    // all loads before the first MFMA, where the compiler would keep too few in flight; the long fp32 runs
    // of NB > 1 do better with loads between them
    constexpr bool HOLD = sizeof(T) == 2 || NB == 1;
    __shared__ f32x4 sums[4][NB][64];
    if (GRAD && (int)blockIdx.x >= a.groups)
        return few_transpose<C>(a, ((int)blockIdx.x - a.groups) * 256 + (int)threadIdx.x);
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int r0 = blockIdx.x * 16 * MR;
    const T *w[MR], *x[NB];
#pragma unroll
    for (int m = 0; m < MR; ++m) w[m] = (const T*)a.w + (size_t)imin(r0 + 16 * m + l, a.vocab - 1) * a.ldw + g * C::E;
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = (const T*)a.x + imin(16 * b + l, a.tokens - 1) * a.ldx + g * C::E;
    f32x4 acc[MR][NB];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Raw (&vw)[MR], const Raw (&vx)[NB]) {
        Part pw[MR][C::P];
#pragma unroll
        for (int m = 0; m < MR; ++m) C::parts(vw[m], pw[m]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            Part px[C::P];
            C::parts(vx[b], px);
            f32x4* c[MR];
#pragma unroll
            for (int m = 0; m < MR; ++m) c[m] = &acc[m][b];
            few_mma<C>(pw, px, c);
        }
    };
    const int full = a.hidden / C::STEP;  // steps without an end of the rows
    const int groups = full / U;          // of U steps; this wave's are wave, wave + 4, ..
    for (int q = wave; q < groups; q += 4) {
        Raw vw[U][MR], vx[U][NB];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const T* p = w[m] + (size_t)q * U * C::STEP;
#pragma unroll
            for (int u = 0; u < U; ++u) vw[u][m] = C::template load<Raw>(p + u * C::STEP);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const T* p = x[b] + (size_t)q * U * C::STEP;
#pragma unroll
            for (int u = 0; u < U; ++u) vx[u][b] = C::template load<Raw>(p + u * C::STEP);
        }
        if (HOLD) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(vw[u], vx[u]);
    }
    // the steps left over, and the last, partial one
    const int steps = (a.hidden + C::STEP - 1) / C::STEP;
    for (int s = groups * U + wave; s < steps; s += 4) {
        const int n = a.hidden - s * C::STEP - g * C::E;  // elements of this lane's chunk, maybe none
        Raw vw[MR], vx[NB];
#pragma unroll
        for (int m = 0; m < MR; ++m) vw[m] = C::template load<Raw>(w[m] + (size_t)s * C::STEP, n);
#pragma unroll
        for (int b = 0; b < NB; ++b) vx[b] = C::template load<Raw>(x[b] + (size_t)s * C::STEP, n);
        multiply(vw, vx);
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
    // dX: `strips` of 16 HE hidden, each in `splits` parts of the vocabulary
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
template <class C, int NB>
__device__ inline void few_dw(const FewGradArgs& a, int block) {
    typedef typename C::T T;
    typedef typename C::Raw Raw;
    typedef typename C::Part Part;
    constexpr int KT = (16 * NB + C::STEP - 1) / C::STEP, HE = C::HE;
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int v0 = block % a.row_groups * 256 + (threadIdx.x >> 6) * 64;
    if (v0 >= a.vocab) return;
    Part d[KT][4][C::DP];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            float f[C::E];
#pragma unroll
            for (int q = 0; q < C::E; ++q) {
                const int t = j * C::STEP + g * C::E + q, v = v0 + 16 * b + l;
                f[q] = t < a.tokens && v < a.vocab ? a.d[t * a.vp + v] : 0.f;
            }
            C::parts(f, d[j][b]);
        }
    constexpr int F = C::F, HB = 2 * F;  // blocks of a group
    const int first = block / a.row_groups * a.groups, last = imin(first + a.groups, (a.hidden + 16 * HB - 1) / (16 * HB));
    for (int q = first; q < last; ++q) {
        Raw x[KT][HB];
        f32x4 c[4][HB] = {};
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
            for (int f = 0; f < HB; ++f) x[j][f] = ((const Raw*)a.xtf)[((q * HB + f) * KT + j) * 64 + lane];
#pragma unroll
        for (int j = 0; j < KT; ++j) {
            Part px[HB][C::P];
#pragma unroll
            for (int f = 0; f < HB; ++f) C::parts(x[j][f], px[f]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                f32x4* o[HB];
#pragma unroll
                for (int f = 0; f < HB; ++f) o[f] = &c[b][f];
                few_mma<C>(px, d[j][b], o);
            }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int v = v0 + 16 * b + l;
            if (v >= a.vocab) continue;
            T* out = (T*)a.out + (size_t)v * a.ld;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int h = 16 * F * (2 * q + s) + HE * g;
                typename C::Row o;
#pragma unroll
                for (int i = 0; i < HE; ++i) o[i] = (T)c[b][s * F + i / 4][i % 4];
                if (h + HE <= a.hidden)
                    *(typename C::Row*)(out + h) = o;
                else
#pragma unroll
                    for (int i = 0; i < HE; ++i)
                        if (h + i < a.hidden) out[h + i] = o[i];
            }
        }
    }
}

// dX of 16 HE hidden over a part of the vocabulary.  A lane loads HE consecutive hidden of E rows of W;
// element e of them makes the operand of the e-th 16 hidden, h0 + HE * (lane % 16) + e.  The four waves
// take every fourth step of the part and add up in LDS.
template <class C, int NB>
__device__ inline void few_dx(const FewGradArgs& a, int block) {
    typedef typename C::T T;
    typedef typename C::Quad Quad;
    typedef typename C::Part Part;
    constexpr int E = C::E, HE = C::HE, U = 8 / E;
    __shared__ f32x4 sums[4][HE][64];
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int h0 = block % a.strips * 16 * HE, h = h0 + l * HE, n = a.hidden - h;
    const int steps = (a.vocab + C::STEP - 1) / C::STEP, z = block / a.strips;
    const int first = (int)((long)steps * z / a.splits), last = (int)((long)steps * (z + 1) / a.splits);
    f32x4 acc[HE][NB] = {};
    const T* w = (const T*)a.w + h;
    for (int s0 = first + wave * U; s0 < last; s0 += 4 * U) {
        Quad rows[U][E];
        f32x4 x[U][NB][E / 4];
        // D is 0 past the vocabulary, where the last row stands in, but not past this part
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = (s0 + u) * C::STEP + g * E;
#pragma unroll
            for (int q = 0; q < E; ++q) {
                const T* p = w + (size_t)imin(v + q, a.vocab - 1) * a.ldw;
                rows[u][q] = n >= HE ? C::template load<Quad>(p) : C::template load<Quad>(p, n);
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
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Part pd[NB][C::DP];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float f[E];
#pragma unroll
                for (int q = 0; q < E; ++q) f[q] = x[u][b][q / 4][q % 4];
                C::parts(f, pd[b]);
            }
#pragma unroll
            for (int e = 0; e < HE; ++e) {
                typename C::Raw t;
#pragma unroll
                for (int q = 0; q < E; ++q) t[q] = rows[u][q][e];
                Part pw[C::P];
                C::parts(t, pw);
                f32x4* o[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) o[b] = &acc[e][b];
                few_mma_t<C>(pw, pd, o);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b > 0) __syncthreads();
#pragma unroll
        for (int e = 0; e < HE; ++e) sums[wave][e][lane] = acc[e][b];
        __syncthreads();
        // element i of block e: token 16 b + l, hidden h0 + HE * (4 g + i) + e; wave i takes its HE in a row
        f32x4* out = (f32x4*)(a.acc + ((size_t)z * 16 * NB + 16 * b + l) * a.hp + h0 + HE * (4 * g + wave));
#pragma unroll
        for (int e = 0; e < HE; e += 4) {
            f32x4 c;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float* p = (const float*)&sums[0][e + q][lane] + wave;
                c[q] = p[0] + p[HE * 256] + p[2 * HE * 256] + p[3 * HE * 256];
            }
            out[e / 4] = a.add ? out[e / 4] + c : c;
        }
    }
}

// Both gradients' products, in one launch: they need D alone.  strips = 0: no dX.
template <class C, int NB>
__global__ void __launch_bounds__(256) vocab_few_grad_kernel(FewGradArgs a) {
    const int dx = a.strips * a.splits;
    if ((int)blockIdx.x < dx)
        few_dx<C, NB>(a, blockIdx.x);
    else
        few_dw<C, NB>(a, (int)blockIdx.x - dx);
}

}  // namespace vocab
}  // namespace libsgemm
