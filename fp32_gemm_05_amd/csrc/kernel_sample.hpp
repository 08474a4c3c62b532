// kernel_sample.hpp -- drawing tokens from rows of logits (gfx950).
//
// What stays of a row is a prefix of its order (falling logit, then rising index) whatever filters are set, so it
// is described by the last logit that stays and the index up to which logits equal to it do.
//
// Probabilities are whole multiples of 2^-40 of the largest, so their sums are exact in 64 bits and the same in any
// order: atomics and any cut of the row give one result.
//
// A workgroup has a row, part of it in registers.  What bounds it is its own passes over the row (131072 bf16 logits:
// 3.8 us for the largest, 19 for a pass of exponentials, 21 for one that counts bins as well, bound by the LDS's additions) and a
// dozen steps of all threads together (0.3 - 1 us each).  So it avoids passes: top_p and a large top_k look for
// the cut in counts of bins of the exponent, from which masses follow to 1 % of what lies on the lighter side, and order
// only the few logits at the border; a small top_k needs no counts (1024 threads' own largest bound it); what
// stays is listed where it is short, and only the listed weighed.  Few long rows are shared by several workgroups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libsgemm {
namespace sample {

typedef unsigned long long u64;

// A value that all lanes have, in a scalar register.
__device__ inline float uniform(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
__device__ inline int uniform(int x) {
    x = __builtin_amdgcn_readfirstlane(x);
    asm volatile("" : "+s"(x));
    return x;
}

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

// exp((x - top) / temperature) as a multiple of 2^-40: log2(e) / temperature = c + c_low, both kept, as an error of c
// is one of all exponents in one direction.  What is left is the rounding of x - top, of the exponent and of the
// exponential.  c is rounded down, so that both parts take -infinity to -infinity and not to NaN.
struct Scale {
    float top, c, c_low, bins;
    __device__ Scale(float top_, float temperature) : top(top_) {
        const double exact = fmin(1.4426950408889634 / (double)temperature, 0x1p120);  // no product with 0 is NaN
        c = (float)exact;
        if ((double)c > exact) c = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, c) - 1);
        c_low = fmaxf((float)(exact - (double)c), c * 0x1p-40f);
        c_low = uniform(c_low > 0.f ? c_low : 0x1p-149f);
        bins = uniform(c * -64.f);
        c = uniform(c);
    }
};
__device__ inline float weight_of(float x, const Scale& s) {
    const float d = x - s.top;
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(d, s.c, d * s.c_low));
    return (e + 0x1p-17f) - 0x1p-17f;
}
// In units of 2^-40.  Below 2^12 sums of weights are exact in 64-bit floating point, and as integers all of a row's
// are.
__device__ inline u64 units(double w) { return __builtin_bit_cast(u64, w + 0x1p12) & ((1ull << 52) - 1); }

// A row's elements: the first V vectors of 16 bytes a thread in registers, the others read from memory (the caches, after
// the first time) in each pass, U on their way at once.  32 registers are what a thread keeps beside its work: with 64
// the compiler spilled, and each pass read the spilled ones again (131072 bf16 logits: 5.3 us for the largest, against 3.8).
// f(index, values) for each vector, of every thread together; past the row's end -infinity.
template <typename T, int V>
struct Row {
    static constexpr int N = 16 / sizeof(T), U = 2;
    const T* row;
    int size, used;  // used: vectors that hold something
    typedef uint32_t Vec __attribute__((ext_vector_type(4)));
    Vec held[V];

    // Of a thread's v-th vector, computed anew each time: kept for all vectors they spill.
    static __device__ inline int index_of(int v) {
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));
        return (v * kThreads + t) * N;
    }
    __device__ inline Vec fetch(int v) const {
        const int i = index_of(v);
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
#pragma unroll
        for (int v = 0; v < V; ++v) held[v] = fetch(v);
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
        f(index_of(v), y);
        __builtin_amdgcn_sched_barrier(0);
    }
    template <class F>
    __device__ inline void each(F f) const {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < uniform(used)) use(v, held[v], f);
        if (used <= V) return;
        Vec x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = fetch(V + u);
#pragma unroll 1
        for (int v = V; v < used; v += U)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Vec y = x[u];
                x[u] = fetch(v + u + U);  // (past the end nothing is read)
                if (v + u < used) use(v + u, y, f);
            }
    }
};

// v plus that of the lane that CTRL names, in the rows of ROWS.
template <int CTRL, int ROWS>
__device__ inline u64 plus_lane(u64 v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
    return v + ((u64)hi << 32 | lo);
}
// Inclusive sums over rows of 16 lanes, and over the wave.
__device__ inline u64 row_scan(u64 v) {
    v = plus_lane<0x111, 0xf>(v);  // row_shr: 1, 2, 4, 8
    v = plus_lane<0x112, 0xf>(v);
    v = plus_lane<0x114, 0xf>(v);
    return plus_lane<0x118, 0xf>(v);
}
__device__ inline u64 wave_scan(u64 v) {
    v = plus_lane<0x142, 0xa>(row_scan(v));  // row_bcast: 15 into rows 1 and 3, 31 into rows 2 and 3
    return plus_lane<0x143, 0xc>(v);
}
__device__ inline u64 of_lane(u64 v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 | lo;
}
// Exclusive sums over the workgroup; `all` gets the whole.  parts: kWaves in LDS.
__device__ inline u64 block_scan(u64 v, u64* parts, u64& all) {
    static_assert(kWaves == 16, "a row of lanes");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const u64 own = wave_scan(v);
    __syncthreads();
    if (lane == 63) parts[wave] = own;
    __syncthreads();
    const u64 waves = row_scan(parts[lane & 15]);
    all = of_lane(waves, 15);
    return (wave > 0 ? of_lane(waves, wave - 1) : 0) + own - v;
}

// The largest value of a smaller key (that of -0 is no value's).
__device__ inline float below(uint32_t key) { return value_of(key - (key == 0x80000000u ? 2 : 1)); }

// What stays: logits above `edge`, and those equal to it up to index `last`.
struct Cut {
    float edge;
    int last;
    __device__ bool keeps(float x, int i) const { return x > edge || (x == edge && i <= last); }
};

constexpr int kList = 2048, kRanked = 256;
struct Shared {
    uint32_t count[kBins + 63];  // while they are counted the last bin has a place for each lane
    u64 mass[kBins], bins[kBins];
    u64 list[kList], range[2];
    uint32_t rank[kRanked];
    u64 parts[kWaves], found[4];
    float tops[kWaves];
    uint32_t front, back, token;
};

// Bins of the exponent, 64 of them to a factor of two from the largest logit down; the last holds all below 2^-32.
constexpr float kPerOctave = 64.f;
__device__ inline uint32_t bin_of(float x, const Scale& s) {
    return (uint32_t)fminf((x - s.top) * s.bins, (float)(kBins - 1));
}
// The least finite value of the bins up to `bin`: the lanes of a wave try 64 keys at once.
__device__ inline float least_of(uint32_t bin, const Scale& s) {
    const uint32_t first = key_of(-INFINITY) + 1, last = key_of(s.top), lane = threadIdx.x & 63;
    if (bin >= kBins - 1) return value_of(first);
    uint32_t base = first - 1;  // lies below
#pragma unroll
    for (int shift = 26; shift >= -4; shift -= 6) {
        const int sh = shift > 0 ? shift : 0;
        const uint64_t at = (uint64_t)base + ((uint64_t)(lane + 1) << sh);
        const bool below = at < last && bin_of(value_of((uint32_t)at), s) > bin;
        base += (uint32_t)__popcll(__ballot(below)) << sh;
    }
    return value_of(base + 1);
}

__device__ inline void clear(Shared& s) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
    if (threadIdx.x < 63) s.count[kBins + threadIdx.x] = 0;
    __syncthreads();
}

// Counts of the bins, -infinities in the last; where `weigh`, a thread's mass.  Most of a row may lie in the last
// bin, and lanes that add to one place wait for each other (131072 bf16 logits: 96 us, so 15): each has its own.
template <class R>
__device__ inline u64 fill(const R& row, const Scale& sc, bool weigh, Shared& s) {
    clear(s);
    u64 mass = 0;
    const float most = (float)(kBins - 1 + (threadIdx.x & 63));
    auto add = [&](float x) { atomicAdd(&s.count[(uint32_t)fminf((x - sc.top) * sc.bins, most)], 1u); };
    if (weigh)
        row.each([&](int, const float (&x)[R::N]) {
            double sum = 0;
#pragma unroll
            for (int q = 0; q < R::N; ++q) {
                add(x[q]);
                sum += (double)weight_of(x[q], sc);
            }
            mass += units(sum);
        });
    else
        row.each([&](int, const float (&x)[R::N]) {
#pragma unroll
            for (int q = 0; q < R::N; ++q) add(x[q]);
        });
    __syncthreads();
    if (threadIdx.x < 63) atomicAdd(&s.count[kBins - 1], s.count[kBins + threadIdx.x]);
    __syncthreads();
    return mass;
}

// The row's mass; a thread's share.
template <class R>
__device__ inline u64 mass_of(const R& row, const Scale& sc) {
    u64 mass = 0;
    row.each([&](int, const float (&x)[R::N]) {
        double sum = 0;
#pragma unroll
        for (int q = 0; q < R::N; ++q) sum += (double)weight_of(x[q], sc);
        mass += units(sum);
    });
    return mass;
}

// f(bin) of the first bin for which `is` turns true along the two bins of each thread, or -1 in none.  was: before
// the thread's first bin.
template <class F>
__device__ inline int first_bin(bool was, bool is0, bool is1, int slot, F note, Shared& s) {
    const int b0 = 2 * threadIdx.x;
    if (threadIdx.x == 0) s.found[slot] = (u64)-1;
    __syncthreads();
    if (!was && is0)
        s.found[slot] = b0, note(0);
    else if (!is0 && is1)
        s.found[slot] = b0 + 1, note(1);
    __syncthreads();
    return (int)s.found[slot];
}

// The bin in which the sum of counts from the top on reaches want > 0, and the sum before it, or -1.
__device__ inline int reach(u64 want, u64& before, Shared& s) {
    const int b0 = 2 * threadIdx.x, b1 = b0 + 1;
    const u64 v0 = s.count[b0], v1 = s.count[b1];
    u64 all;
    const u64 at = block_scan(v0 + v1, s.parts, all);
    const int bin = first_bin(at >= want, at + v0 >= want, at + v0 + v1 >= want, 0,
                              [&](int second) { s.found[1] = second ? at + v0 : at; }, s);
    before = s.found[1];
    return bin;
}

// The bins [lo, hi] in one of which the sum of masses from the top on reaches want <= total, from the counts.  A bin's
// mass lies between its count times the weights at its ends, 2^(1/64) apart; and so does what lies below a bin,
// which is the row's mass less the sum up to it.  counted: of the bins before lo, between: of lo to hi.
__device__ inline void reach_mass(u64 want, u64 total, int& lo, int& hi, u64& counted, u64& between, Shared& s) {
    const int b0 = 2 * threadIdx.x, b1 = b0 + 1;
    const u64 c0 = s.count[b0], c1 = s.count[b1];
    // 2^-16 more and less than the ends: an exponent's own rounding, and a weight's to units
    auto least = [&](int b, u64 c) -> u64 {
        const double w = (double)__builtin_amdgcn_exp2f(-(float)(b + 1) / kPerOctave) * (0x1p40 * (1 - 0x1p-16)) - 1.;
        return b < kBins - 1 && w > 0. ? (u64)(w * (double)c) : 0;
    };
    auto most = [&](int b, u64 c) -> u64 {
        return (u64)(((double)__builtin_amdgcn_exp2f(-(float)b / kPerOctave) * (0x1p40 * (1 + 0x1p-16)) + 2.) * (double)c);
    };
    const u64 l0 = least(b0, c0), l1 = least(b1, c1), m0 = most(b0, c0), m1 = most(b1, c1);
    u64 all_l, all_m, all_c;
    const u64 low = block_scan(l0 + l1, s.parts, all_l), high = block_scan(m0 + m1, s.parts, all_m);
    const u64 count = block_scan(c0 + c1, s.parts, all_c);
    auto at_least = [&](u64 l, u64 m) {
        const u64 below = all_m - m, rest = total > below ? total - below : 0;
        return l > rest ? l : rest;
    };
    auto at_most = [&](u64 l, u64 m) {
        const u64 below = all_l - l, rest = total > below ? total - below : 0;
        return m < rest ? m : rest;
    };
    lo = first_bin(at_most(low, high) >= want && b0 > 0, at_most(low + l0, high + m0) >= want,
                   at_most(low + l0 + l1, high + m0 + m1) >= want, 0, [&](int second) { s.found[1] = second ? count + c0 : count; }, s);
    hi = first_bin(at_least(low, high) >= want && b0 > 0, at_least(low + l0, high + m0) >= want,
                   at_least(low + l0 + l1, high + m0 + m1) >= want, 2,
                   [&](int second) { s.found[3] = count + c0 + (second ? c1 : 0); }, s);
    // (past the last bin nothing lies below: both are reached)
    counted = s.found[1];
    between = s.found[3] - counted;
}

// s.list[0, n) in falling order, n <= kRanked: each entry's rank is the number of larger ones (they are all different),
// counted by several threads each.
__device__ inline void sort(uint32_t n, Shared& s) {
    uint32_t places = 64;  // whole waves
    while (places < n) places *= 2;
    const uint32_t i = threadIdx.x & (places - 1), part = threadIdx.x / places, parts = kThreads / places;
    const uint32_t per = (n + parts - 1) / parts, from = part * per, to = from + per < n ? from + per : n;
    if (threadIdx.x < kRanked) s.rank[threadIdx.x] = 0;
    __syncthreads();
    const u64 own = i < n ? s.list[i] : 0;
    uint32_t larger = 0;
#pragma unroll 8
    for (uint32_t j = from; j < to; ++j) larger += s.list[j] > own;
    if (i < n && larger > 0) atomicAdd(&s.rank[i], larger);
    __syncthreads();
    if (threadIdx.x < n) s.list[s.rank[threadIdx.x]] = own;
    __syncthreads();
}

// A place behind what is listed already for each lane that `has` one: one addition a wave.
__device__ inline uint32_t place_of(bool has, uint32_t* listed) {
    const uint64_t mask = __ballot(has);
    if (mask == 0) return 0;
    const uint32_t lane = threadIdx.x & 63;
    uint32_t at = 0;
    if (lane == 0) at = atomicAdd(listed, (uint32_t)__popcll(mask));
    at = (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
    return at + (uint32_t)__popcll(mask & ((1ull << lane) - 1));
}

// The logits from `from` on: those below `sure` from the front of s.list on, the others from its back, where
// `certain`.  false: they are too many.
template <class R>
__device__ inline bool gather(const R& row, float from, float sure, bool certain, Shared& s) {
    __syncthreads();
    if (threadIdx.x == 0) s.front = s.back = 0;
    __syncthreads();
    row.each([&](int i, const float (&x)[R::N]) {
        uint32_t mine = 0, rest = 0;
#pragma unroll
        for (int q = 0; q < R::N; ++q) mine |= (uint32_t)(x[q] >= from && x[q] < sure) << q;
        if (certain)
#pragma unroll
            for (int q = 0; q < R::N; ++q) rest |= (uint32_t)(x[q] >= sure) << q;
        if (!__any((mine | rest) != 0)) return;
        if (*(volatile uint32_t*)&s.front + *(volatile uint32_t*)&s.back > kList) return;
        // few in a vector: a place at a time
#pragma unroll
        for (int q = 0; q < R::N; ++q) {
            const u64 entry = (u64)key_of(x[q]) << 32 | ~(uint32_t)(i + q);
            if (mine >> q & 1) {
                const uint32_t at = atomicAdd(&s.front, 1u);
                if (at < kList) s.list[at] = entry;
            }
            if (rest >> q & 1) {
                const uint32_t at = atomicAdd(&s.back, 1u);
                if (at < kList) s.list[kList - 1 - at] = entry;
            }
        }
    });
    __syncthreads();
    return s.front + s.back <= kList;
}
__device__ inline float value_at(uint32_t i, const Shared& s) { return value_of((uint32_t)(s.list[i] >> 32)); }
__device__ inline int index_at(uint32_t i, const Shared& s) { return (int)~(uint32_t)s.list[i]; }

// Tiles of the row for the sum by index: blocks of a wave's vector, 2^k of them each.
template <class R>
struct Tiles {
    static constexpr int BLOCK = 64 * R::N;
    int k, size;
    __device__ Tiles(int n) : k(0), size(n) {
        while (((n - 1) / BLOCK) >> k >= kBins) ++k;
    }
    __device__ int of(int i) const { return i / BLOCK >> k; }
};
// Each tile's mass that stays, in s.mass; EQUAL: some of those equal to the edge do.  first: the index of row's first.
template <bool EQUAL, class R>
__device__ inline void weigh_tiles(const R& row, const Scale& sc, const Tiles<R>& tiles, Cut cut, Shared& s, int first = 0) {
    clear(s);
    row.each([&](int i, const float (&x)[R::N]) {
        float most = x[0];
#pragma unroll
        for (int q = 1; q < R::N; ++q) most = fmaxf(most, x[q]);
        if (!__any(EQUAL ? most >= cut.edge : most > cut.edge)) return;
        double sum = 0;
#pragma unroll
        for (int q = 0; q < R::N; ++q)
            sum += (double)((EQUAL ? cut.keeps(x[q], i + q) : x[q] > cut.edge) ? weight_of(x[q], sc) : 0.f);
        const u64 whole = wave_scan(units(sum));
        if ((threadIdx.x & 63) == 63 && whole > 0) atomicAdd(&s.mass[tiles.of(first + i)], whole);
    });
    __syncthreads();
}
__device__ inline u64 sum_of_tiles(Shared& s) {
    u64 all;
    block_scan(s.mass[2 * threadIdx.x] + s.mass[2 * threadIdx.x + 1], s.parts, all);
    return all;
}
// What is listed: the first `front` of s.list and the last `back`.
struct Listed {
    uint32_t front, back;
    __device__ uint32_t size() const { return front + back; }
    __device__ uint32_t place(uint32_t i) const { return i < front ? i : kList - 1 - (i - front); }
};
// Adds those of them that stay to the tiles' masses.
template <class R>
__device__ inline void add_listed(Listed l, Cut cut, const Scale& sc, const Tiles<R>& tiles, Shared& s) {
    for (uint32_t i = threadIdx.x; i < l.size(); i += kThreads) {
        const uint32_t at = l.place(i);
        const float x = value_at(at, s);
        if (cut.keeps(x, index_at(at, s))) atomicAdd(&s.mass[tiles.of(index_at(at, s))], units(weight_of(x, sc)));
    }
}
__device__ inline u64 mass_listed(Listed l, const Scale& sc, Shared& s) {
    u64 own = 0, all;
    for (uint32_t i = threadIdx.x; i < l.size(); i += kThreads) own += units(weight_of(value_at(l.place(i), s), sc));
    block_scan(own, s.parts, all);
    return all;
}

// The cut digit by digit of the keys, for any logits (many equal, or far below the top): where the sum of counts
// (masses) reaches want > 0.
template <class R>
__device__ inline Cut descend(const R& row, const Scale& sc, const Tiles<R>& tiles, bool by_mass, u64 want, Shared& s) {
    uint32_t prefix = 0, mask = 0;
    u64 in_bin = 0;
    const int b0 = 2 * threadIdx.x, b1 = b0 + 1;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        clear(s);
        row.each([&](int, const float (&x)[R::N]) {
#pragma unroll
            for (int q = 0; q < R::N; ++q) {
                const uint32_t k = key_of(x[q]);
                if ((k & mask) != prefix || x[q] == -INFINITY) continue;
                const int bin = kBins - 1 - ((k >> shift) & ((1 << bits) - 1));  // the largest keys first
                atomicAdd(&s.count[bin], 1u);
                if (by_mass) atomicAdd(&s.mass[bin], units(weight_of(x[q], sc)));
            }
        });
        __syncthreads();
        const u64 v0 = by_mass ? s.mass[b0] : s.count[b0], v1 = by_mass ? s.mass[b1] : s.count[b1];
        u64 all;
        const u64 at = block_scan(v0 + v1, s.parts, all);
        const int bin = first_bin(at >= want, at + v0 >= want, at + v0 + v1 >= want, 0,
                                  [&](int second) { s.found[1] = second ? at + v0 : at; }, s);
        prefix |= (uint32_t)(kBins - 1 - bin) << shift;
        mask |= (uint32_t)((1u << bits) - 1) << shift;
        want -= s.found[1];
        in_bin = s.count[bin];
    }
    const float edge = value_of(prefix);
    u64 need = want;
    if (by_mass) {
        const u64 w = units(weight_of(edge, sc));  // above 0: a mass was reached here
        need = (want + w - 1) / w;
    }
    if (need >= in_bin) return {below(prefix), -1};
    // the index of the `need`-th of the equal ones: its tile, then its place there
    clear(s);
    row.each([&](int i, const float (&x)[R::N]) {
        uint32_t same = 0;
#pragma unroll
        for (int q = 0; q < R::N; ++q) same += __popcll(__ballot(x[q] == edge));
        if ((threadIdx.x & 63) == 63 && same > 0) atomicAdd(&s.count[tiles.of(i)], same);
    });
    __syncthreads();
    u64 before = 0;
    const int tile = reach(need, before, s);
    const int step = Tiles<R>::BLOCK << tiles.k, from = tile * step, to = from + step < tiles.size ? from + step : tiles.size;
    const int per = (to - from + kThreads - 1) / kThreads, mine = from + threadIdx.x * per, end = mine + per < to ? mine + per : to;
    u64 own = 0, all;
    for (int i = mine; i < end; ++i) own += (float)row.row[i] == edge;
    u64 at = before + block_scan(own, s.parts, all);
    if (at < need && need <= at + own)
        for (int i = mine; i < end; ++i)
            if ((float)row.row[i] == edge && ++at == need) s.found[0] = i;
    __syncthreads();
    return {edge, (int)s.found[0]};
}

// Less than this lies before the last that stays of `mass`.
__device__ inline u64 least_mass(float top_p, u64 mass) {
    const double p = (double)top_p * (double)mass;
    return p < 1. ? 1 : (u64)__builtin_ceil(p);
}

// Of the sorted list's first n the number up to which the sum of weights, with `before`, reaches want, or n;
// `all`: the sum of all n.
__device__ inline uint32_t listed_mass(uint32_t n, u64 before, u64 want, const Scale& sc, u64& all, Shared& s) {
    const uint32_t i0 = 2 * threadIdx.x, i1 = i0 + 1;
    const u64 w0 = i0 < n ? units(weight_of(value_at(i0, s), sc)) : 0, w1 = i1 < n ? units(weight_of(value_at(i1, s), sc)) : 0;
    const u64 at = before + block_scan(w0 + w1, s.parts, all);
    const int last = first_bin(at >= want && i0 > 0, at + w0 >= want && i0 < n, at + w0 + w1 >= want && i1 < n, 0, [](int) {}, s);
    return last < 0 ? n : (uint32_t)last + 1;
}
// The cut within the list's front, where the sum of counts (masses), with `before`, reaches want; those past it are
// dropped.  whole: within all that is listed.  A long list is narrowed first, by 2048 bins of what is left of its range
// (value and index in one number, so equal logits too come apart), what lies before the bin going to the back: merging it
// in LDS took 17 us for 2048.
__device__ inline Cut cut_listed(Listed& l, bool whole, bool by_mass, u64 want, u64 before, const Scale& sc, Shared& s) {
    u64 all;
    uint32_t n = whole ? l.size() : l.front;
    bool merge = whole && l.back > 0;
    while (n > kRanked || merge) {
        const uint32_t i0 = threadIdx.x, i1 = i0 + kThreads;
        if (threadIdx.x == 0) s.range[0] = ~0ull, s.range[1] = 0;
        s.bins[i0] = s.bins[i1] = 0;
        __syncthreads();
        const u64 e0 = i0 < n ? s.list[l.place(i0)] : 0, e1 = i1 < n ? s.list[l.place(i1)] : 0;
        u64 low = i0 < n ? e0 : ~0ull, high = e0 > e1 ? e0 : e1;
        if (i1 < n && e1 < low) low = e1;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const u64 a = __shfl_xor(low, o), b = __shfl_xor(high, o);
            low = a < low ? a : low;
            high = b > high ? b : high;
        }
        if ((threadIdx.x & 63) == 0 && i0 < n) atomicMin(&s.range[0], low), atomicMax(&s.range[1], high);
        __syncthreads();
        const u64 least = s.range[0], most = s.range[1];
        const int bits = 64 - __builtin_clzll((most - least) | 1), shift = bits > 11 ? bits - 11 : 0;
        auto bin_at = [&](u64 e) { return (uint32_t)((most - e) >> shift); };
        auto amount = [&](u64 e) { return by_mass ? units(weight_of(value_of((uint32_t)(e >> 32)), sc)) : 1ull; };
        if (i0 < n) atomicAdd(&s.bins[bin_at(e0)], amount(e0));
        if (i1 < n) atomicAdd(&s.bins[bin_at(e1)], amount(e1));
        __syncthreads();
        const u64 v0 = s.bins[2 * threadIdx.x], v1 = s.bins[2 * threadIdx.x + 1];
        const u64 at = before + block_scan(v0 + v1, s.parts, all);
        const uint32_t bin = first_bin(at >= want, at + v0 >= want, at + v0 + v1 >= want, 0,
                                       [&](int second) { s.found[1] = second ? at + v0 : at; }, s);
        before = s.found[1];
        if (threadIdx.x == 0) s.front = 0, s.back = merge ? 0 : l.back;
        __syncthreads();
        auto put = [&](u64 e, bool is) {
            const bool front = is && bin_at(e) == bin, back = is && bin_at(e) < bin;
            const uint32_t f = place_of(front, &s.front), b = place_of(back, &s.back);
            if (front) s.list[f] = e;
            if (back) s.list[kList - 1 - b] = e;
        };
        put(e0, i0 < n);
        put(e1, i1 < n);
        __syncthreads();
        l = {s.front, s.back};
        n = l.front;
        merge = false;
        __syncthreads();
    }
    sort(n, s);
    const uint32_t last = by_mass ? listed_mass(n, before, want, sc, all, s) - 1 : (uint32_t)(want - before) - 1;
    l.front = last + 1;
    return {value_at(last, s), index_at(last, s)};
}

// A row's settings.
struct Settings {
    float temperature, top_p, min_p, u;
    long long top_k;
    __device__ Settings(const Args& a, int r)
        : temperature(a.temperatures ? a.temperatures[r] : a.temperature), top_p(a.top_ps ? a.top_ps[r] : a.top_p),
          min_p(a.min_ps ? a.min_ps[r] : a.min_p), u(a.u[r]), top_k(a.top_ks ? a.top_ks[r] : a.top_k) {}
    __device__ bool valid(float top) const {
        return __builtin_isfinite(top) && temperature >= 0.f && temperature < INFINITY && u == u && top_p == top_p && min_p == min_p;
    }
    __device__ bool first_alone() const { return temperature == 0.f || min_p > 1.f; }
    __device__ bool weigh() const { return top_p < 1.f; }
    __device__ bool ranked(int size) const { return top_k > 0 && top_k < size; }
    static __device__ float lowest() { return value_of(key_of(-INFINITY) + 1); }  // of the finite values
    // The least logit of at least min_p times the largest one's probability.
    __device__ float least(float top) const {
        if (!(min_p > 0.f)) return lowest();
        const double x = (double)top + log((double)min_p) * (double)temperature;
        if (!(x > (double)lowest())) return lowest();
        const float y = (float)x;
        return (double)y < x ? value_of(key_of(y) + 1) : y;
    }
};

// The largest value, NaN where there is one; of a thread's own, and in every thread of the row's part.
template <class R>
__device__ inline float top_of(const R& row, float& own, Shared& s) {
    own = -INFINITY;
    row.each([&](int, const float (&x)[R::N]) {
#pragma unroll
        for (int q = 0; q < R::N; ++q) own = __builtin_elementwise_maximum(own, x[q]);
    });
    float top = own;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = __builtin_elementwise_maximum(top, __shfl_xor(top, o));
    if ((threadIdx.x & 63) == 0) s.tops[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) top = __builtin_elementwise_maximum(top, s.tops[w]);
    return uniform(top);
}
// The lowest index of a value, in s.token.
template <class R>
__device__ inline void first_of(const R& row, float value, Shared& s) {
    uint32_t first = 0xffffffffu;
    if (threadIdx.x == 0) s.token = first;
    row.each([&](int i, const float (&x)[R::N]) {
#pragma unroll
        for (int q = R::N - 1; q >= 0; --q)
            if (x[q] == value && (uint32_t)(i + q) < first) first = i + q;
    });
    __syncthreads();
    if (first != 0xffffffffu) atomicMin(&s.token, first);
    __syncthreads();
}

// The token by the tiles' masses in s.mass: the tile in which the sum passes u's share, and the place in it.
template <typename T, class R>
__device__ inline void pick(const T* row, const Tiles<R>& tiles, const Scale& sc, Cut cut, float u, long long* token, Shared& s) {
    const int t0 = 2 * threadIdx.x;
    const u64 m0 = s.mass[t0], m1 = s.mass[t0 + 1];
    u64 all;
    const u64 at = block_scan(m0 + m1, s.parts, all);
    double share = (double)u * (double)all;
    share = share > 0. ? share : 0.;
    u64 target = share < (double)all ? (u64)share : all - 1;
    target = target < all ? target : all - 1;
    const int tile = first_bin(at > target, at + m0 > target, at + m0 + m1 > target, 0,
                               [&](int second) { s.found[1] = second ? at + m0 : at; }, s);
    const int step = Tiles<R>::BLOCK << tiles.k, from = tile * step, to = from + step < tiles.size ? from + step : tiles.size;
    const int per = (to - from + kThreads - 1) / kThreads, mine = from + threadIdx.x * per, end = mine + per < to ? mine + per : to;
    const u64 done = s.found[1];
    auto mass = [&](int i) -> u64 {
        const float x = (float)row[i];
        return cut.keeps(x, i) ? units(weight_of(x, sc)) : 0;
    };
    u64 own = 0;
    for (int i = mine; i < end; ++i) own += mass(i);
    u64 sum = done + block_scan(own, s.parts, all);
    if (sum <= target && target < sum + own)
        for (int i = mine; i < end; ++i) {
            sum += mass(i);
            if (sum > target) {
                *token = i;
                return;
            }
        }
}

// One row.  V: vectors of the row in a thread's registers.
template <typename T, int V>
__device__ inline void draw_row(const Args& a, int r, Shared& s) {
    typedef Row<T, V> R;
    constexpr int N = R::N;
    const int size = a.vocab;
    R row;
    row.init((const T*)a.logits + (size_t)r * a.ld, size);
    const Settings set(a, r);
    const float top_p = set.top_p;
    const long long top_k = set.top_k;
    float own_top;
    const float top = top_of(row, own_top, s);
    if (!set.valid(top)) {
        if (threadIdx.x == 0) a.token[r] = -1;
        return;
    }
    if (set.first_alone()) {
        first_of(row, top, s);
        if (threadIdx.x == 0) a.token[r] = s.token;
        return;
    }
    const Scale sc(top, set.temperature);
    const Tiles<R> tiles(size);
    const float lowest = Settings::lowest(), least = set.least(top);
    const Cut at_least{below(key_of(least)), -1};
    const bool weigh = set.weigh(), ranked = set.ranked(size);

    // From one stage to the next until what stays is known: all of it as `cut`, or up to a border in a list.
    enum { QUICK, COUNT, LEAST, MASS, REST, WHOLE, BORDER, LISTED };
    int stage = ranked ? (top_k <= kThreads / 2 ? QUICK : COUNT) : !weigh ? REST : least > lowest ? LEAST : MASS;
    Cut cut{below(key_of(lowest)), -1};  // what top_k leaves, then all
    bool certain = false;                // what lies before the border is listed too
    u64 want = 0, total = 0;
    bool filled = false;
    float border = INFINITY;             // what lies from it on stays
    while (stage < WHOLE) {
        int lo = 0, hi = -1, next = stage;
        u64 before = 0;
        float from = lowest, sure = INFINITY;
        certain = false;
        if (stage == QUICK) {
            // top_k of the threads' own largest logits are as large as the least of those: where no more than the list holds
            // are, the counts of all are not needed.  Up to half of the threads': with more, the least of them leaves more
            // than the list holds (us, so / by counts: 300 rows of 131072 fp32, top_k 50 69 / 96, 512 94 / 117, 700 100 /
            // 120, 900 179 / 124; 64 of 32768 bf16 25 / 26, 29 / 30, 30 / 30, 40 / 31)
            clear(s);
            if (own_top > -INFINITY) atomicAdd(&s.count[bin_of(own_top, sc)], 1u);
            __syncthreads();
            hi = reach((u64)top_k, before, s);
            if (hi >= 0) from = weigh ? least_of(hi, sc) : fmaxf(least_of(hi, sc), least);
            next = WHOLE;
        } else if (stage == LEAST) {
            // min_p's cut first: where what it leaves is short, top_p's lies in that list or past it, and the counts
            // of all are not needed for it, only their mass
            hi = 0;
            from = least;
            next = WHOLE;
        } else if (stage == COUNT || stage == MASS) {
            if (!filled || (stage == MASS && total == 0)) {
                const u64 own = fill(row, sc, stage == MASS, s);
                if (stage == MASS) block_scan(own, s.parts, total);
                filled = true;
            }
            if (stage == COUNT) {
                lo = hi = reach((u64)top_k, before, s);
                next = weigh ? MASS : REST;
                if (before + s.count[hi] <= kList) {
                    next = WHOLE;
                    lo = 0;
                }
                from = least_of(hi, sc);
                if (next == WHOLE && !weigh) from = fmaxf(from, least);
                if (lo > 0) sure = least_of(lo - 1, sc);
            } else {
                if (want == 0) want = least_mass(top_p, total);
                u64 counted, between;
                reach_mass(want, total, lo, hi, counted, between, s);
                next = BORDER;
                if (lo > 0) sure = least_of(lo - 1, sc);
                from = least_of(hi, sc);
                if (least >= sure) {
                    stage = REST;  // min_p's cut lies before top_p's
                    continue;
                }
                certain = counted + between <= kList;
                border = sure;
                if (between > kList) hi = -1;
            }
        } else {
            if (!(least > lowest && least > cut.edge)) break;
            // min_p's cut: all that is as large, if it is short
            cut = at_least;
            hi = 0;
            from = least;
            next = LISTED;
        }
        const bool got = hi >= 0 && gather(row, from, sure, certain, s);
        if (got && (next == WHOLE || next == BORDER || next == LISTED)) {
            stage = next;
            break;
        }
        if (stage == QUICK || stage == LEAST) {
            stage = stage == QUICK ? COUNT : MASS;
            continue;
        }
        if (stage == REST) break;
        // the cut of top_k, or that of top_p where too many lie at its border
        bool stays = false;
        if (stage == COUNT && hi == kBins - 1) {  // of fewer finite logits than top_k all stay
            u64 own = 0, finite;
            row.each([&](int, const float (&x)[N]) {
#pragma unroll
                for (int q = 0; q < N; ++q) own += x[q] > -INFINITY;
            });
            block_scan(own, s.parts, finite);
            stays = finite <= (u64)top_k;
        }
        if (!stays) {
            if (got) {
                Listed border{s.front, 0};
                cut = cut_listed(border, false, false, (u64)top_k, before, sc, s);
            } else {
                cut = descend(row, sc, tiles, stage == MASS, stage == MASS ? want : (u64)top_k, s);
                filled = false;
            }
        }
        stage = stage == COUNT && weigh ? MASS : REST;
        if (stage == MASS && !stays) {
            weigh_tiles<true>(row, sc, tiles, cut, s);
            want = least_mass(top_p, sum_of_tiles(s));
            filled = false;
        }
    }

    // the tiles' masses
    Listed l{stage == REST ? 0 : s.front, stage == BORDER && certain ? s.back : 0};
    if (stage == WHOLE) {
        if (ranked && (u64)top_k <= l.front) cut = cut_listed(l, true, false, (u64)top_k, 0, sc, s);
        if (weigh) {
            const u64 listed = mass_listed(l, sc, s);
            if (ranked)
                total = listed;
            else
                block_scan(mass_of(row, sc), s.parts, total);
            want = least_mass(top_p, total);
            if (want <= listed) cut = cut_listed(l, true, true, want, 0, sc, s);
        }
    }
    if (stage == REST && cut.last >= 0) {
        weigh_tiles<true>(row, sc, tiles, cut, s);
    } else if (stage == REST || (stage == BORDER && !certain)) {
        if (stage == BORDER) cut = {below(key_of(border)), -1};
        weigh_tiles<false>(row, sc, tiles, cut, s);
    }
    if (stage == BORDER)
        cut = cut_listed(l, false, true, want, certain ? mass_listed(Listed{0, l.back}, sc, s) : sum_of_tiles(s), sc, s);
    if (least > cut.edge) cut = at_least;
    if (stage != REST) {
        if (stage != BORDER || certain) clear(s);
        add_listed(l, cut, sc, tiles, s);
        __syncthreads();
    }

    pick(row.row, tiles, sc, cut, set.u, a.token + r, s);
}

// One row a workgroup.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sample_row_kernel(Args a) {
    __shared__ Shared s;
    draw_row<T, V>(a, blockIdx.x, s);
}

// ---- few long rows: several workgroups each ------------------------------------------------------------
//
// With fewer rows than compute units a row's passes are shared by `splits` workgroups, each with `vectors` vectors of it a
// thread, in four launches: the largest; counts of the bins and the mass; what lies at the border and the
// tiles' masses; the token, by one workgroup again.  What the row kernel does in further passes (a border that many share,
// top_k beyond the list with top_p) it does here too, alone.

constexpr int kMostSplits = 16;
enum Mode { NO_ROW, FIRST, TILES, LIST, BORDER_LISTED, BORDER_TILES, BORDER_COUNTED, ALONE };
struct State {
    float tops[kMostSplits];
    u64 total, want;
    uint32_t front, back, first, mode;
};
struct SplitArgs {
    Args a;
    int splits, vectors;
    State* state;    // of each row, as the following
    uint32_t* count; // [kBins]
    u64* mass;       // [kBins]: of the tiles
    u64* list;       // [kList]
};

// This workgroup's part of its row: `at` its first element.
template <typename T, int V>
struct Part {
    typedef Row<T, V> R;
    int r, split, at, size;
    R row;
    __device__ Part(const SplitArgs& p) {
        r = blockIdx.x / p.splits, split = blockIdx.x - r * p.splits;
        const int step = p.vectors * kThreads * R::N;
        at = split * step;
        size = p.a.vocab - at < step ? p.a.vocab - at : step;
        row.init((const T*)p.a.logits + (size_t)r * p.a.ld + at, size);
    }
};
__device__ inline float top_of(const State& st, int splits) {
    float top = st.tops[0];
    for (int i = 1; i < splits; ++i) top = __builtin_elementwise_maximum(top, st.tops[i]);
    return uniform(top);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sample_top_kernel(SplitArgs p) {
    __shared__ Shared s;
    Part<T, V> part(p);
    State& st = p.state[part.r];
    for (int i = part.split * kThreads + threadIdx.x; i < kBins; i += p.splits * kThreads) {
        p.count[(size_t)part.r * kBins + i] = 0;
        p.mass[(size_t)part.r * kBins + i] = 0;
    }
    float own;
    const float top = top_of(part.row, own, s);
    if (threadIdx.x == 0) st.tops[part.split] = top;
    if (part.split == 0 && threadIdx.x == 0) st.total = 0, st.front = st.back = 0, st.first = 0xffffffffu;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sample_count_kernel(SplitArgs p) {
    __shared__ Shared s;
    const int r = blockIdx.x / p.splits;
    State& st = p.state[r];
    const Settings set(p.a, r);
    const float top = top_of(st, p.splits);
    const bool ranked = set.ranked(p.a.vocab), weigh = set.weigh() && !ranked;
    if (!set.valid(top) || set.first_alone() || !(ranked || weigh)) return;
    Part<T, V> part(p);
    const Scale sc(top, set.temperature);
    const u64 own = fill(part.row, sc, weigh, s);
    u64 all;
    block_scan(own, s.parts, all);
    if (weigh && threadIdx.x == 0) atomicAdd(&st.total, all);
    for (int i = threadIdx.x; i < kBins; i += kThreads)
        if (s.count[i] > 0) atomicAdd(&p.count[(size_t)r * kBins + i], s.count[i]);
}

// What the border's list and the tiles are made of: listed from `from` on, below `sure` at the border; in the tiles
// what is above `edge`.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sample_border_kernel(SplitArgs p) {
    __shared__ Shared s;
    Part<T, V> part(p);
    State& st = p.state[part.r];
    const Settings set(p.a, part.r);
    const float top = top_of(st, p.splits);
    if (!set.valid(top)) {
        if (part.split == 0 && threadIdx.x == 0) st.mode = NO_ROW;
        return;
    }
    if (set.first_alone()) {
        first_of(part.row, top, s);
        if (threadIdx.x == 0 && s.token != 0xffffffffu) atomicMin(&st.first, s.token + part.at);
        if (part.split == 0 && threadIdx.x == 0) st.mode = FIRST;
        return;
    }
    const Scale sc(top, set.temperature);
    const float least = set.least(top);
    const bool ranked = set.ranked(p.a.vocab), weigh = set.weigh();
    float from = INFINITY, sure = INFINITY, edge = below(key_of(least));
    Mode mode = TILES;
    u64 want = 0;
    if (ranked || weigh) {
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = p.count[(size_t)part.r * kBins + i];
        __syncthreads();
        int lo = 0, hi = 0;
        u64 before = 0, counted = 0, between = 0;
        if (ranked) {
            lo = hi = reach((u64)set.top_k, before, s);
            between = s.count[hi];
            counted = before;
            want = (u64)set.top_k - before;
            mode = counted + between <= kList ? LIST : weigh || hi == kBins - 1 || between > kList ? ALONE : BORDER_COUNTED;
            if (mode == LIST) lo = 0;
        } else {
            want = least_mass(set.top_p, st.total);
            reach_mass(want, st.total, lo, hi, counted, between, s);
            mode = between > kList ? ALONE : counted + between <= kList ? BORDER_LISTED : BORDER_TILES;
        }
        if (lo > 0) sure = least_of(lo - 1, sc);
        from = least_of(hi, sc);
        if (mode == LIST && !weigh) from = fmaxf(from, least);
        if (mode == BORDER_COUNTED || mode == BORDER_TILES) edge = below(key_of(sure));
        if (mode != LIST && mode != ALONE && least >= sure) {  // min_p's cut lies before theirs
            mode = TILES;
            from = INFINITY;
            edge = below(key_of(least));
        }
    }
    if (part.split == 0 && threadIdx.x == 0) st.mode = mode, st.want = want;
    if (mode == ALONE) return;
    if (from < INFINITY) {
        // (all of it fits the row's list, as the counts say)
        gather(part.row, from, sure, mode == BORDER_LISTED, s);
        if (threadIdx.x == 0) {
            s.found[0] = s.front > 0 ? atomicAdd(&st.front, s.front) : 0;
            s.found[1] = s.back > 0 ? atomicAdd(&st.back, s.back) : 0;
        }
        __syncthreads();
        u64* const list = p.list + (size_t)part.r * kList;
        const uint32_t f = (uint32_t)s.found[0], b = (uint32_t)s.found[1];
        for (uint32_t i = threadIdx.x; i < s.front + s.back; i += kThreads) {
            const bool front = i < s.front;
            const uint32_t place = front ? f + i : kList - 1 - (b + i - s.front);
            // the index counts from the row's start: its complement is in the low half
            if (place < kList) list[place] = s.list[front ? i : kList - 1 - (i - s.front)] - (u64)part.at;
        }
    }
    if (mode == TILES || mode == BORDER_TILES || mode == BORDER_COUNTED) {
        const Tiles<Row<T, V>> tiles(p.a.vocab);
        weigh_tiles<false>(part.row, sc, tiles, Cut{edge, -1}, s, part.at);
        // (a part is whole tiles)
        for (int i = threadIdx.x; i < kBins; i += kThreads)
            if (s.mass[i] > 0) p.mass[(size_t)part.r * kBins + i] = s.mass[i];
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sample_token_kernel(SplitArgs p) {
    __shared__ Shared s;
    const int r = blockIdx.x;
    const State& st = p.state[r];
    const int mode = st.mode;
    if (mode == NO_ROW || mode == FIRST) {
        if (threadIdx.x == 0) p.a.token[r] = mode == FIRST ? (long long)st.first : -1;
        return;
    }
    if (mode == ALONE) return draw_row<T, V>(p.a, r, s);
    const Settings set(p.a, r);
    const float top = top_of(st, p.splits), least = set.least(top);
    const Scale sc(top, set.temperature);
    const Tiles<Row<T, V>> tiles(p.a.vocab);
    Listed l{st.front, st.back};
    for (uint32_t i = threadIdx.x; i < l.size(); i += kThreads) s.list[l.place(i)] = p.list[(size_t)r * kList + l.place(i)];
    const bool tiled = mode == TILES || mode == BORDER_TILES || mode == BORDER_COUNTED;
    clear(s);
    if (tiled)
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.mass[i] = p.mass[(size_t)r * kBins + i];
    __syncthreads();
    const Cut at_least{below(key_of(least)), -1};
    Cut cut = at_least;
    if (mode == LIST) {
        if ((u64)set.top_k <= l.front) cut = cut_listed(l, true, false, (u64)set.top_k, 0, sc, s);
        if (set.weigh()) cut = cut_listed(l, true, true, least_mass(set.top_p, mass_listed(l, sc, s)), 0, sc, s);
    } else if (mode == BORDER_COUNTED) {
        cut = cut_listed(l, false, false, st.want, 0, sc, s);
    } else if (mode != TILES) {
        const u64 before = mode == BORDER_LISTED ? mass_listed(Listed{0, l.back}, sc, s) : sum_of_tiles(s);
        cut = cut_listed(l, false, true, st.want, before, sc, s);
    }
    if (least > cut.edge) cut = at_least;
    if (!tiled) clear(s);
    add_listed(l, cut, sc, tiles, s);
    __syncthreads();
    pick((const T*)p.a.logits + (size_t)r * p.a.ld, tiles, sc, cut, set.u, p.a.token + r, s);
}

}  // namespace sample
}  // namespace libsgemm
