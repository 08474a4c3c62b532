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

// exp((x - top) / temperature) as a multiple of 2^-40: log2(e) / temperature = c + c_low.  The exponent is kept in two
// parts, so that what is off is the exponential's own last place and x - top's rounding.
struct Scale {
    float top, c, c_low;
};
__device__ inline float exponent_of(float x, const Scale& s) { return (x - s.top) * s.c; }
__device__ inline float weight_of(float x, const Scale& s) {
    const float d = x - s.top, t = d * s.c;
    const float low = __builtin_fmaf(d, s.c_low, __builtin_fmaf(d, s.c, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    // (where t is -infinity, low is NaN)
    const float w = t > -42.f ? __builtin_fmaf(e * 0.693147181f, low, e) : 0.f;
    return (w + 0x1p-17f) - 0x1p-17f;
}
// In units; sums of up to 2^12 weights are exact in 64-bit floating point, and all of a row's as integers.
__device__ inline u64 units(double w) { return (u64)(w * 0x1p40); }

// A row's elements: V vectors of 16 bytes a thread in registers (V = 0: read from memory each time, U vectors on
// their way at once).  f(index, values) for each vector, of every thread together; past the row's end -infinity.
template <typename T, int V>
struct Row {
    static constexpr int N = 16 / sizeof(T), U = 4, HELD = V > 0 ? V : 1;
    const T* row;
    int size, used;  // used: vectors that hold something
    typedef uint32_t Vec __attribute__((ext_vector_type(4)));
    Vec held[HELD];

    __device__ inline Vec fetch(int v) const {
        const int i = (v * kThreads + (int)threadIdx.x) * N;
        Vec x;
        if (i + N <= size) {
            __builtin_memcpy(&x, row + i, 16);
        } else {
            T e[N];
#pragma unroll
            for (int q = 0; q < N; ++q) e[q] = i + q < size ? row[i + q] : (T)-INFINITY;
            __builtin_memcpy(&x, e, 16);
        }
        return x;
    }
    __device__ inline void init(const T* at, int n) {
        row = at, size = n, used = (n + kThreads * N - 1) / (kThreads * N);
        if (V > 0)
#pragma unroll
            for (int v = 0; v < HELD; ++v) held[v] = fetch(v);
    }
    template <class F>
    __device__ inline void use(int v, Vec x, F& f) const {
        // the values anew for each use, and a vector at a time: what one pass makes of them would otherwise be kept for
        // the next, for all vectors at once, and spill
        asm volatile("" : "+v"(x));
        T z[N];
        __builtin_memcpy(z, &x, 16);
        float y[N];
#pragma unroll
        for (int q = 0; q < N; ++q) y[q] = (float)z[q];
        int at = (v * kThreads + (int)threadIdx.x) * N;
        asm volatile("" : "+v"(at));
        f(at, y);
        __builtin_amdgcn_sched_barrier(0);
    }
    template <class F>
    __device__ inline void each(F f) const {
        if constexpr (V > 0) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v < used) use(v, held[v], f);
        } else {
            for (int v = 0; v < used; v += U) {
                Vec x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] = fetch(v + u);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v + u < used) use(v + u, x[u], f);
            }
        }
    }
};

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
#pragma unroll 2
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += parts[w];
        all += parts[w];
    }
    return before + own - v;
}

// What stays: keys above `key`, and the first `equal` (by index) of those with it.
struct Cut {
    uint32_t key, equal;
};
constexpr uint32_t kAll = 0xffffffffu;

constexpr int kList = 2048;
struct Shared {
    uint32_t count[kBins];
    u64 mass[kBins];
    u64 list[kList];
    u64 parts[kWaves], found[4];
    uint32_t keys[kWaves], bad[kWaves], listed;
};

// Bins of the exponent, from `from` below the top's on, `per` of them to a factor of two; those above it
// are bin -1, those below the last kBins.
struct Window {
    float from, per;
    __device__ int bin(float t) const {
        const float b = (-t - from) * per;
        return b < 0.f ? -1 : b < (float)kBins ? (int)b : kBins;
    }
};
// What the logits and the masses spread over: 2^-16, down to 2^-48, and far logits that only top_k counts.
__device__ inline Window window(int w) {
    return w == 0 ? Window{0.f, 128.f} : w == 1 ? Window{16.f, 64.f} : Window{48.f, 16.f};
}
constexpr int kWindows = 3;

// Counts, and where `weigh` the weights, of a window's bins.
template <class R>
__device__ inline void fill(const R& row, const Scale& sc, int w, bool weigh, Shared& s) {
    const Window win = window(w);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
    __syncthreads();
    row.each([&](int, const float (&x)[R::N]) {
#pragma unroll
        for (int q = 0; q < R::N; ++q) {
            const int bin = win.bin(exponent_of(x[q], sc));
            if (bin < 0 || bin >= kBins) continue;
            atomicAdd(&s.count[bin], 1u);
            if (weigh) atomicAdd(&s.mass[bin], units(weight_of(x[q], sc)));
        }
    });
    __syncthreads();
}

// The row's order is walked to where the sum of counts (by_mass: of masses) reaches `want` > 0: the cut there, and in
// `left` the mass that stays, where it is wanted (`weigh`).  False: it is not reached within the windows, or too many
// logits share a bin.  filled: the window that the bins hold.
template <class R>
__device__ inline bool find(const R& row, const Scale& sc, bool by_mass, u64 want, bool weigh, int& filled, Cut& cut, u64& left, Shared& s) {
    u64 before = 0, mass_before = 0;
    for (int w = 0; w < kWindows; ++w) {
        if (filled != w) {
            fill(row, sc, w, weigh, s);
            filled = w;
        }
        const int b0 = 2 * threadIdx.x, b1 = b0 + 1;
        const u64 c0 = s.count[b0], c1 = s.count[b1], m0 = s.mass[b0], m1 = s.mass[b1];
        u64 all, all_mass;
        const u64 mass = mass_before + block_scan(m0 + m1, s.parts, all_mass);
        u64 sum = before + block_scan(c0 + c1, s.parts, all);
        if (by_mass) sum = mass, all = all_mass;
        const u64 v0 = by_mass ? m0 : c0, v1 = by_mass ? m1 : c1;
        if (sum < want && want <= sum + v0) s.found[0] = b0, s.found[1] = sum, s.found[2] = mass;
        if (sum + v0 < want && want <= sum + v0 + v1) s.found[0] = b1, s.found[1] = sum + v0, s.found[2] = mass + m0;
        __syncthreads();
        if (before + all < want) {
            before += all;
            mass_before += all_mass;
            continue;
        }
        const int bin = (int)s.found[0];
        before = s.found[1];
        mass_before = s.found[2];
        const uint32_t n = s.count[bin];
        if (n > kList) return false;
        // the bin's logits in order: by key, then from the lowest index on
        if (threadIdx.x == 0) s.listed = 0;
        uint32_t size = 64;
        while (size < n) size *= 2;
        for (uint32_t i = threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
        __syncthreads();
        const Window win = window(w);
        row.each([&](int i, const float (&x)[R::N]) {
#pragma unroll
            for (int q = 0; q < R::N; ++q)
                if (win.bin(exponent_of(x[q], sc)) == bin)
                    s.list[atomicAdd(&s.listed, 1u)] = (u64)key_of(x[q]) << 32 | ~(uint32_t)(i + q);
        });
        __syncthreads();
        for (uint32_t k = 2; k <= size; k *= 2)
            for (uint32_t j = k / 2; j > 0; j /= 2) {
                for (uint32_t i = threadIdx.x; i < size / 2; i += kThreads) {
                    const uint32_t a = 2 * i - (i & (j - 1)), b = a + j;
                    const u64 x = s.list[a], y = s.list[b];
                    if ((x < y) == ((a & k) == 0)) s.list[a] = y, s.list[b] = x;
                }
                __syncthreads();
            }
        const u64 e0 = (uint32_t)b0 < n ? s.list[b0] : 0, e1 = (uint32_t)b1 < n ? s.list[b1] : 0;
        const uint32_t k0 = (uint32_t)(e0 >> 32), k1 = (uint32_t)(e1 >> 32);
        const u64 w0 = (uint32_t)b0 < n && weigh ? units(weight_of(value_of(k0), sc)) : 0;
        const u64 w1 = (uint32_t)b1 < n && weigh ? units(weight_of(value_of(k1), sc)) : 0;
        const u64 at = mass_before + block_scan(w0 + w1, s.parts, all);
        // the first of them that reaches it is the last that stays
        if ((uint32_t)b0 < n && (by_mass ? at < want && want <= at + w0 : before + b0 + 1 == want))
            s.found[0] = b0, s.found[1] = at + w0;
        if ((uint32_t)b1 < n && (by_mass ? at + w0 < want && want <= at + w0 + w1 : before + b1 + 1 == want))
            s.found[0] = b1, s.found[1] = at + w0 + w1;
        __syncthreads();
        const uint32_t last = (uint32_t)s.found[0];
        left = s.found[1];
        cut.key = (uint32_t)(s.list[last] >> 32);
        u64 same = 0, equal;
        for (uint32_t i = threadIdx.x; i <= last; i += kThreads) same += (uint32_t)(s.list[i] >> 32) == cut.key;
        block_scan(same, s.parts, equal);
        cut.equal = (uint32_t)equal;
        __syncthreads();
        return true;
    }
    return false;
}

// The same digit by digit of the keys, for any logits (all equal, or too far below the top for the windows).
template <class R>
__device__ inline void descend(const R& row, const Scale& sc, bool by_mass, u64 want, Cut& cut, Shared& s) {
    uint32_t prefix = 0, mask = 0;
    u64 in_bin = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
        __syncthreads();
        row.each([&](int, const float (&x)[R::N]) {
#pragma unroll
            for (int q = 0; q < R::N; ++q) {
                const uint32_t k = key_of(x[q]);
                if ((k & mask) != prefix || x[q] == -INFINITY) continue;
                const int bin = (k >> shift) & ((1 << bits) - 1);
                atomicAdd(&s.count[bin], 1u);
                if (by_mass) atomicAdd(&s.mass[bin], units(weight_of(x[q], sc)));
            }
        });
        __syncthreads();
        // two bins a thread, from the largest keys down
        const int b1 = kBins - 1 - 2 * threadIdx.x, b0 = b1 - 1;
        const u64 v1 = by_mass ? s.mass[b1] : s.count[b1], v0 = by_mass ? s.mass[b0] : s.count[b0];
        u64 all;
        const u64 before = block_scan(v1 + v0, s.parts, all);
        if (before < want && want <= before + v1) s.found[0] = b1, s.found[1] = before, s.found[2] = s.count[b1];
        if (before + v1 < want && want <= before + v1 + v0)
            s.found[0] = b0, s.found[1] = before + v1, s.found[2] = s.count[b0];
        __syncthreads();
        prefix |= (uint32_t)s.found[0] << shift;
        mask |= (uint32_t)((1u << bits) - 1) << shift;
        want -= s.found[1];
        in_bin = s.found[2];
    }
    u64 need = want;
    if (by_mass) {
        const u64 w = units(weight_of(value_of(prefix), sc));  // above 0: a mass was reached here
        need = (want + w - 1) / w;
    }
    cut = {prefix, (uint32_t)(need < in_bin ? need : in_bin)};
}

// The mass that stays.
template <class R>
__device__ inline u64 mass_of(const R& row, const Scale& sc, Cut cut, Shared& s) {
    u64 own = 0, same = 0, all, many;
    row.each([&](int, const float (&x)[R::N]) {
        double sum = 0;
#pragma unroll
        for (int q = 0; q < R::N; ++q) {
            const uint32_t k = key_of(x[q]);
            sum += k > cut.key ? (double)weight_of(x[q], sc) : 0.;
            same += k == cut.key;
        }
        own += units(sum);
    });
    block_scan(own, s.parts, all);
    block_scan(same, s.parts, many);
    return all + (many < cut.equal ? many : cut.equal) * units(weight_of(value_of(cut.key), sc));
}

template <class R>
__device__ inline u64 finite_of(const R& row, Shared& s) {
    u64 own = 0, all;
    row.each([&](int, const float (&x)[R::N]) {
#pragma unroll
        for (int q = 0; q < R::N; ++q) own += x[q] > -INFINITY;
    });
    block_scan(own, s.parts, all);
    return all;
}

// One row a workgroup.  V: vectors of the row in a thread's registers, 0 for longer ones.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sample_row_kernel(Args a) {
    __shared__ Shared s;
    const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, size = a.vocab;
    Row<T, V> row;
    row.init((const T*)a.logits + (size_t)r * a.ld, size);
    const float temperature = a.temperatures ? a.temperatures[r] : a.temperature;
    const float top_p = a.top_ps ? a.top_ps[r] : a.top_p, min_p = a.min_ps ? a.min_ps[r] : a.min_p, u = a.u[r];
    const long long top_k = a.top_ks ? a.top_ks[r] : a.top_k;

    float top = -INFINITY;
    bool bad = false;
    row.each([&](int, const float (&x)[Row<T, V>::N]) {
#pragma unroll
        for (int q = 0; q < Row<T, V>::N; ++q) {
            bad |= x[q] != x[q];
            top = fmaxf(top, x[q]);
        }
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    bad = __any(bad);
    if (lane == 0) s.keys[wave] = __builtin_bit_cast(uint32_t, top), s.bad[wave] = bad;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        top = fmaxf(top, __builtin_bit_cast(float, s.keys[w]));
        bad |= s.bad[w] != 0;
    }
    bad |= !__builtin_isfinite(top) || !(temperature >= 0.f && temperature < INFINITY) || u != u || top_p != top_p ||
           min_p != min_p;
    if (bad) {
        if (threadIdx.x == 0) a.token[r] = -1;
        return;
    }
    const double c = 1.4426950408889634 / (double)temperature;
    const Scale sc{top, (float)c, (float)(c - (double)(float)c)};
    Cut cut{key_of(-INFINITY) + 1, kAll};
    if (temperature == 0.f) {
        cut = {key_of(top), 1};  // the first of the largest
    } else {
        const bool weigh = top_p < 1.f;
        const bool ranked = top_k > 0 && top_k < size && (u64)top_k < finite_of(row, s);  // else all stay
        int filled = -1;
        u64 left = 0;
        bool weighed = false;
        for (int by_mass = ranked ? 0 : 1; by_mass < (weigh ? 2 : 1); ++by_mass) {
            u64 want = (u64)top_k;
            if (by_mass) {
                if (!weighed) left = mass_of(row, sc, cut, s);
                // less than `want` lies before the last that stays
                const double p = (double)top_p * (double)left;
                want = p < 1. ? 1 : (u64)__builtin_ceil(p);
            }
            weighed = find(row, sc, by_mass != 0, want, weigh, filled, cut, left, s);
            if (!weighed) {
                descend(row, sc, by_mass != 0, want, cut, s);
                filled = -1;
            }
        }
        if (min_p > 0.f) {
            // the least logit of at least min_p times the largest one's probability
            const double least = (double)top + log((double)min_p) * (double)temperature;
            float x = (float)least;
            if ((double)x < least) x = value_of(key_of(x) + 1);
            if (min_p > 1.f)
                cut = {key_of(top), 1};
            else if (key_of(x) > cut.key)
                cut = {key_of(x), kAll};
        }
    }

    // Blocks of a wave's vector, 2^k of them to a tile: what each tile holds of the mass, and how many of the cut's key
    constexpr int BLOCK = 64 * Row<T, V>::N;
    int k = 0;
    while ((((size - 1) / BLOCK + 1) - 1) >> k >= kBins) ++k;
    const bool limited = cut.equal != kAll;
    const bool greedy = temperature == 0.f;
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
    __syncthreads();
    row.each([&](int i, const float (&x)[Row<T, V>::N]) {
        double sum = 0;
        uint32_t same = 0;
#pragma unroll
        for (int q = 0; q < Row<T, V>::N; ++q) {
            const uint32_t key = key_of(x[q]);
            if (!greedy) sum += key > cut.key || (key == cut.key && !limited) ? (double)weight_of(x[q], sc) : 0.;
            if (limited) same += __popcll(__ballot(key == cut.key));
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
        if (lane == 0 && i < size) {
            const int tile = i / BLOCK >> k;
            if (sum > 0.) atomicAdd(&s.mass[tile], units(sum));
            if (same > 0) atomicAdd(&s.count[tile], same);
        }
    });
    __syncthreads();
    const u64 w = greedy ? 1 : limited ? units(weight_of(value_of(cut.key), sc)) : 0;
    const int t0 = 2 * threadIdx.x, t1 = t0 + 1;
    u64 many = 0, all, e0 = 0;
    auto stay = [&](u64 before, u64 n) -> u64 { return before >= cut.equal ? 0 : n < cut.equal - before ? n : cut.equal - before; };
    u64 m0 = s.mass[t0], m1 = s.mass[t1];
    const u64 n0 = s.count[t0], n1 = s.count[t1];
    if (limited) {
        e0 = block_scan(n0 + n1, s.parts, many);
        m0 += stay(e0, n0) * w;
        m1 += stay(e0 + n0, n1) * w;
    }
    const u64 before = block_scan(m0 + m1, s.parts, all);
    double at = (double)u * (double)all;
    at = at > 0. ? at : 0.;
    u64 target = at < (double)all ? (u64)at : all - 1;
    target = target < all ? target : all - 1;
    // the tile in which the sum passes the target
    if (before <= target && target < before + m0) s.found[0] = t0, s.found[1] = before, s.found[2] = e0;
    if (before + m0 <= target && target < before + m0 + m1) s.found[0] = t1, s.found[1] = before + m0, s.found[2] = e0 + n0;
    __syncthreads();
    const int from = (int)s.found[0] * (BLOCK << k), to = from + (BLOCK << k) < size ? from + (BLOCK << k) : size;
    const u64 done = s.found[1], seen = s.found[2];
    const int per = (to - from + kThreads - 1) / kThreads, mine = from + threadIdx.x * per;
    const int end = mine + per < to ? mine + per : to;
    auto weigh = [&](float x) -> u64 {
        const uint32_t key = key_of(x);
        return key > cut.key || (key == cut.key && !limited) ? greedy ? 0 : units(weight_of(x, sc)) : 0;
    };
    u64 first = seen, own = 0, same = 0;
    for (int i = mine; i < end; ++i) {
        own += weigh((float)row.row[i]);
        same += key_of((float)row.row[i]) == cut.key;
    }
    if (limited) {
        first += block_scan(same, s.parts, many);
        own += stay(first, same) * w;
    }
    u64 sum = done + block_scan(own, s.parts, all);
    if (sum <= target && target < sum + own) {
        for (int i = mine; i < end; ++i) {
            const float x = (float)row.row[i];
            if (limited && key_of(x) == cut.key)
                sum += first++ < cut.equal ? w : 0;
            else
                sum += weigh(x);
            if (sum > target) {
                a.token[r] = i;
                return;
            }
        }
    }
}

}  // namespace sample
}  // namespace libsgemm
