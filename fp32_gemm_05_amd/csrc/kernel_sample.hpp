// kernel_sample.hpp -- drawing tokens from rows of logits (gfx950).
//
// What stays of a row is a prefix of its order (falling logit, then rising index) whatever filters are set, so it
// is described by the key of the last logit that stays and how many of the logits equal to it do, from the lowest
// index on.  Keys are the fp32 values' bits in an order that compares as unsigned integers.
//
// Probabilities are whole multiples of 2^-40 of the largest, so their sums are exact in 64 bits and the same in any
// order: atomics and any cut of the row give one result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libsgemm {
namespace sample {

typedef unsigned long long u64;

struct Args {
    const void* logits;
    long ld;
    int vocab;
    const float *u, *temperatures;
    float temperature;
    const long long* top_ks;
    long long top_k;
    const float* top_ps;
    float top_p;
    const float* min_ps;
    float min_p;
    long long* token;
};

constexpr int kThreads = 1024, kWaves = kThreads / 64, kBins = 2048;

// Larger values have larger keys; -0 and 0 have one.
__device__ inline uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline float value_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// exp((x - top) / temperature) in units of 2^-40; c = log2(e) / temperature.  2^f by a polynomial on [-1/2, 1/2] of
// relative error 5e-11, in 64 bits, which cost gfx950 what 32 do.
__device__ inline u64 weight_of(float x, float top, double c) {
    const double t = ((double)x - (double)top) * c;
    if (!(t > -42.)) return 0;
    const double n = __builtin_rint(t), f = t - n;
    double p = 1.5201919728190897e-05;
    p = __builtin_fma(p, f, 0.0001546929113014313);
    p = __builtin_fma(p, f, 0.0013333922571744298);
    p = __builtin_fma(p, f, 0.009618027253716714);
    p = __builtin_fma(p, f, 0.05550410353437774);
    p = __builtin_fma(p, f, 0.24022651198157027);
    p = __builtin_fma(p, f, 0.69314718072845);
    p = __builtin_fma(p, f, 1.0);
    // the rounded value stands in the low bits of its sum with 2^52
    const double w = __builtin_amdgcn_ldexp(p, 40 + (int)n) + 0x1p52;
    return __builtin_bit_cast(u64, w) & ((1ull << 52) - 1);
}

template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
};

// f(index, value) for the elements [from, to) of a row, in pieces of 16 bytes a lane from lane `at` of `step`; a
// lane's own elements come in rising order.
template <typename T, class F>
__device__ inline void each(const T* row, int from, int to, int at, int step, F f) {
    constexpr int N = Vec<T>::N;
    for (int i = from + at * N; i < to; i += step * N) {
        if (i + N <= to) {
            T v[N];
            __builtin_memcpy(v, row + i, 16);
#pragma unroll
            for (int q = 0; q < N; ++q) f(i + q, (float)v[q]);
        } else {
            for (int q = 0; i + q < to; ++q) f(i + q, (float)row[i + q]);
        }
    }
}

__device__ inline u64 wave_scan(u64 v) {  // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const u64 w = __shfl_up(v, o);
        if (lane >= o) v += w;
    }
    return v;
}
// Exclusive sums over the workgroup; `all` gets the whole.  parts: kWaves in LDS.
__device__ inline u64 block_scan(u64 v, u64* parts, u64& all) {
    const int wave = threadIdx.x >> 6;
    const u64 own = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) parts[wave] = own;
    __syncthreads();
    u64 before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += parts[w];
        all += parts[w];
    }
    return before + own - v;
}

// The least that stays: keys above `key`, and the first `equal` (by index) of those with it.
struct Cut {
    uint32_t key;
    uint32_t equal;
};

struct Shared {
    uint32_t count[kBins];
    u64 mass[kBins];
    u64 parts[kWaves];
    u64 found[3];
    uint32_t keys[kWaves], bad[kWaves];
};

// Where the descending sum of counts (MASS: of masses) over the row's elements that stay under `cut` reaches
// `want` > 0, digit by digit of the keys.  MASS: how many of the last key are needed for it; else what is left.
template <bool MASS, typename T>
__device__ inline Cut descend(const Args& a, const T* row, float top, double c, Cut cut, u64 over, u64 want, Shared& s) {
    uint32_t prefix = 0, mask = 0;
    u64 in_bin = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
        __syncthreads();
        each(row, 0, a.vocab, threadIdx.x, kThreads, [&](int, float x) {
            const uint32_t k = key_of(x);
            if ((k & mask) != prefix || k < cut.key) return;
            const int bin = (k >> shift) & ((1 << bits) - 1);
            atomicAdd(&s.count[bin], 1u);
            if (MASS) atomicAdd(&s.mass[bin], weight_of(x, top, c));
        });
        __syncthreads();
        // of the elements with the cut's key only cut.equal count: `over` mass is too much
        if (MASS && threadIdx.x == 0 && (cut.key & mask) == prefix) s.mass[(cut.key >> shift) & ((1 << bits) - 1)] -= over;
        __syncthreads();
        // two bins a thread, from the largest keys down
        const int b1 = kBins - 1 - 2 * threadIdx.x, b0 = b1 - 1;
        const u64 v1 = MASS ? s.mass[b1] : s.count[b1], v0 = MASS ? s.mass[b0] : s.count[b0];
        u64 all;
        const u64 before = block_scan(v1 + v0, s.parts, all);
        if (before < want && want <= before + v1)
            s.found[0] = b1, s.found[1] = before, s.found[2] = s.count[b1];
        else if (before + v1 < want && want <= before + v1 + v0)
            s.found[0] = b0, s.found[1] = before + v1, s.found[2] = s.count[b0];
        __syncthreads();
        prefix |= (uint32_t)s.found[0] << shift;
        mask |= (uint32_t)((1u << bits) - 1) << shift;
        want -= s.found[1];
        in_bin = s.found[2];
    }
    if (!MASS) return {prefix, (uint32_t)want};
    const u64 w = weight_of(value_of(prefix), top, c);
    u64 need = w ? (want + w - 1) / w : in_bin;
    if (prefix == cut.key && need > cut.equal) need = cut.equal;
    return {prefix, (uint32_t)(need < in_bin ? need : in_bin)};
}

// One row a workgroup.
template <typename T>
__global__ void __launch_bounds__(kThreads) sample_row_kernel(Args a) {
    __shared__ Shared s;
    const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T* row = (const T*)a.logits + (size_t)r * a.ld;
    const float temperature = a.temperatures ? a.temperatures[r] : a.temperature;
    const float top_p = a.top_ps ? a.top_ps[r] : a.top_p, min_p = a.min_ps ? a.min_ps[r] : a.min_p, u = a.u[r];
    const long long top_k = a.top_ks ? a.top_ks[r] : a.top_k;
    const int V = a.vocab;

    uint32_t largest = 0;
    bool bad = false;
    each(row, 0, V, threadIdx.x, kThreads, [&](int, float x) {
        bad |= x != x;
        const uint32_t k = key_of(x);
        largest = k > largest ? k : largest;
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint32_t k = __shfl_xor(largest, o);
        largest = k > largest ? k : largest;
    }
    bad = __any(bad);
    if (lane == 0) s.keys[wave] = largest, s.bad[wave] = bad;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        largest = s.keys[w] > largest ? s.keys[w] : largest;
        bad |= s.bad[w] != 0;
    }
    const float top = value_of(largest);
    bad |= !__builtin_isfinite(top) || !(temperature >= 0.f && temperature < INFINITY) || u != u || top_p != top_p ||
           min_p != min_p;
    if (bad) {
        if (threadIdx.x == 0) a.token[r] = -1;
        return;
    }
    // temperature 0: the first of the largest
    Cut cut{key_of(-INFINITY) + 1, 0xffffffffu};
    double c = 0;
    if (temperature == 0.f) {
        cut = {largest, 1};
    } else {
        c = 1.4426950408889634 / (double)temperature;
        u64 over = 0;
        if (top_k > 0 && top_k < V) {
            // of fewer finite logits than top_k all stay
            const Cut k = descend<false>(a, row, top, c, Cut{0, 0}, 0, (u64)top_k, s);
            if (k.key >= cut.key) cut = k;
        }
        if (top_p < 1.f) {
            // the mass that stays so far, without the equal ones that do not
            u64 own = 0, same = 0, all, many;
            each(row, 0, V, threadIdx.x, kThreads, [&](int, float x) {
                const uint32_t k = key_of(x);
                if (k >= cut.key) own += weight_of(x, top, c);
                if (k == cut.key) ++same;
            });
            block_scan(own, s.parts, all);
            block_scan(same, s.parts, many);
            if (many > cut.equal) over = (many - cut.equal) * weight_of(value_of(cut.key), top, c);
            const double want = (double)top_p * (double)(all - over);
            const u64 least = want < 1. ? 1 : (u64)__builtin_ceil(want);
            cut = descend<true>(a, row, top, c, cut, over, least, s);
        }
        if (min_p > 0.f) {
            // the least logit of at least min_p times the largest one's probability
            const double least = (double)top + log((double)min_p) * (double)temperature;
            float x = (float)least;
            if ((double)x < least) x = value_of(key_of(x) + 1);
            if (min_p > 1.f)
                cut = {largest, 1};
            else if (key_of(x) > cut.key)
                cut = {key_of(x), 0xffffffffu};
        }
    }
    // tiles of `size` elements: what each holds of the mass, and how many of the cut's key
    const int size = V <= kBins * 1024 ? 1024 : (V + kBins - 1) / kBins, tiles = (V + size - 1) / size;
    __syncthreads();
    for (int t = wave; t < tiles; t += kWaves) {
        const int from = t * size, to = from + size < V ? from + size : V;
        u64 own = 0;
        uint32_t same = 0;
        each(row, from, to, lane, 64, [&](int, float x) {
            const uint32_t k = key_of(x);
            if (k > cut.key) own += temperature == 0.f ? 1 : weight_of(x, top, c);
            if (k == cut.key) ++same;
        });
        own = wave_scan(own);
        same = (uint32_t)wave_scan(same);
        if (lane == 63) s.mass[t] = own, s.count[t] = same;
    }
    __syncthreads();
    const u64 w = temperature == 0.f ? 1 : weight_of(value_of(cut.key), top, c);
    const int t0 = 2 * threadIdx.x, t1 = t0 + 1;
    const u64 n0 = t0 < tiles ? s.count[t0] : 0, n1 = t1 < tiles ? s.count[t1] : 0;
    u64 many, all;
    const u64 e0 = block_scan(n0 + n1, s.parts, many), e1 = e0 + n0;
    auto stay = [&](u64 before, u64 n) -> u64 { return before >= cut.equal ? 0 : n < cut.equal - before ? n : cut.equal - before; };
    const u64 m0 = (t0 < tiles ? s.mass[t0] : 0) + stay(e0, n0) * w, m1 = (t1 < tiles ? s.mass[t1] : 0) + stay(e1, n1) * w;
    const u64 before = block_scan(m0 + m1, s.parts, all);
    double at = (double)u * (double)all;
    at = at > 0. ? at : 0.;
    u64 target = at < (double)all ? (u64)at : all - 1;
    target = target < all ? target : all - 1;
    // the tile in which the sum passes the target
    if (before <= target && target < before + m0) s.found[0] = t0, s.found[1] = before, s.found[2] = e0;
    if (before + m0 <= target && target < before + m0 + m1) s.found[0] = t1, s.found[1] = before + m0, s.found[2] = e1;
    __syncthreads();
    const int from = (int)s.found[0] * size, to = from + size < V ? from + size : V;
    const u64 done = s.found[1], seen = s.found[2];
    const int per = (to - from + kThreads - 1) / kThreads, mine = from + threadIdx.x * per;
    const int end = mine + per < to ? mine + per : to;
    u64 same = 0;
    for (int i = mine; i < end; ++i) same += key_of((float)row[i]) == cut.key;
    const u64 first = seen + block_scan(same, s.parts, many);
    u64 own = stay(first, same) * w;
    auto weigh = [&](uint32_t k, float x) -> u64 { return k > cut.key ? temperature == 0.f ? 1 : weight_of(x, top, c) : 0; };
    for (int i = mine; i < end; ++i) own += weigh(key_of((float)row[i]), (float)row[i]);
    u64 sum = done + block_scan(own, s.parts, all);
    if (sum <= target && target < sum + own) {
        u64 eq = first;
        for (int i = mine; i < end; ++i) {
            const float x = (float)row[i];
            const uint32_t k = key_of(x);
            u64 v = weigh(k, x);
            if (k == cut.key) v = eq++ < cut.equal ? w : 0;
            sum += v;
            if (sum > target) {
                a.token[r] = i;
                return;
            }
        }
    }
}

}  // namespace sample
}  // namespace libsgemm
