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

// Whether a token has an entry among its from-th and later ones; eight are looked at at once.
__device__ inline bool any_entry(const Entries& e, long t, int from) {
    bool any = false;
    for (int k = from; k < e.k && !any; k += 8)
#pragma unroll
        for (int q = 0; q < 8; ++q) any |= e.counts(e.index[t * e.ld + imin(k + q, e.k - 1)]);
    return any;
}

// rows[0 .. *count): the tokens that count, in order; pos: a token's place in rows, or -1; loss and
// lse (when given) of the others 0.  By one workgroup of 256, 4096 tokens at a time so that their
// entries are read together.
struct Counted {
    int *rows, *pos, *count;
    float *loss, *lse;
};
__device__ inline void count_tokens(const Entries& e, int tokens, const Counted& c) {
    constexpr int R = 16;
    __shared__ int waves[R][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int done = 0;
    for (int t0 = 0; t0 < tokens; t0 += 256 * R) {
        bool live[R];
        unsigned long long m[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // past the end the last token again, so that no load stands behind a branch
            const int t = t0 + r * 256 + threadIdx.x;
            live[r] = e.counts(e.index[(size_t)imin(t, tokens - 1) * e.ld]) && t < tokens;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = t0 + r * 256 + threadIdx.x;
            if (t < tokens && !live[r]) live[r] = any_entry(e, t, 1);
            m[r] = __ballot(live[r]);
            if (lane == 0) waves[r][wave] = __popcll(m[r]);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int before = done;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                before += w < wave ? waves[r][w] : 0;
                done += waves[r][w];
            }
            const int t = t0 + r * 256 + threadIdx.x;
            if (t >= tokens) continue;
            const int at = before + __popcll(m[r] & ((1ull << lane) - 1));
            c.pos[t] = live[r] ? at : -1;
            if (live[r]) c.rows[at] = t;
            if (!live[r] && c.loss) c.loss[t] = c.lse[t] = 0.f;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) *c.count = done;
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

// Each entry's share of the teacher: the sum of q over the entries of its token that name the same row.  Up
// to kPairs entries a wave compares each with each (token_wave); past that, as that time is the square of
// their number, a workgroup sorts a token's entries by row and place and adds up the runs, in an order that
// the entries alone decide.  Up to kSortInLds they are sorted in LDS, past that in `keys`.  Bound by the
// barriers of the sort's passes.  Measured (a gradient call, 32768 x 16, us, compared/sorted): 2 tokens of 128
// entries 44, 42; of 256 78, 44; of 16384 201828, 579; 1000 tokens of 128 138, 148; of 192 153, 153; of 256
// 172, 155.
constexpr int kPairs = 192, kSortInLds = 8192;
template <bool IN_LDS>
__global__ void __launch_bounds__(1024) vocab_shares_kernel(Entries e, int vocab, uint64_t* keys, float* shares) {
    __shared__ uint64_t held[IN_LDS ? kSortInLds : 1];
    __shared__ float part[2][16];
    const long t = blockIdx.x;
    const uint32_t n = e.k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const i64* index = e.index + t * e.ld;
    const float* teacher = e.teacher + t * e.ld_teacher;
    uint64_t* const a = IN_LDS ? held : keys + (size_t)t * n;
    float m = -INFINITY, s = 0.f;
    for (uint32_t k = tid; k < n; k += 1024) {
        const i64 v = index[k];
        if (v >= 0) m = fmaxf(m, teacher[k] * e.teacher_alpha);
        a[k] = v >= 0 && v < vocab ? (uint64_t)v << 32 | k : ~0ull;  // the others are read by nothing
    }
    m = wave_max(m);
    if (lane == 0) part[0][wave] = m;
    __syncthreads();
    const float top = wave_max(part[0][lane & 15]);
    for (uint32_t k = tid; k < n; k += 1024)
        if (index[k] >= 0) s += expf(teacher[k] * e.teacher_alpha - top);
    s = wave_sum(s);
    if (lane == 0) part[1][wave] = s;
    __syncthreads();
    const float log_total = logf(wave_sum(lane < 16 ? part[1][lane] : 0.f));
    // a bitonic network of ascending comparisons alone, for which entries past n are the largest
    int log_n = 0;
    while ((1ull << log_n) < n) ++log_n;
    for (int size = 1; size <= log_n; ++size)
        for (int step = size; step > 0; --step) {
            const uint32_t width = 1u << (step - 1);
            for (uint32_t p = tid; p < 1u << (log_n - 1); p += 1024) {
                const uint32_t i = (p & ~(width - 1)) * 2 | (p & (width - 1));
                const uint32_t j = step == size ? i ^ (2 * width - 1) : i + width;
                if (j < n) {
                    const uint64_t x = a[i], y = a[j];
                    if (x > y) a[i] = y, a[j] = x;
                }
            }
            __syncthreads();
        }
    // a lane adds up the run that starts at its place, up to kRun; a wave the longer ones together
    constexpr uint32_t kRun = 64;
    auto row = [&](uint32_t j) { return (uint32_t)(a[j] >> 32); };
    auto share = [&](uint32_t j) { return expf(teacher[(uint32_t)a[j]] * e.teacher_alpha - top - log_total); };
    for (uint32_t j0 = wave * 64; j0 < n; j0 += 1024) {
        const uint32_t j = j0 + lane;
        const uint32_t r = j < n ? row(j) : ~0u;
        const bool head = r != ~0u && (j == 0 || row(j - 1) != r);
        uint32_t end = j;
        float q = 0.f;
        if (head)
            for (; end < n && end - j < kRun && row(end) == r; ++end) q += share(end);
        const bool more = head && end < n && row(end) == r;
        if (head && !more)
            for (uint32_t i = j; i < end; ++i) shares[t * n + (uint32_t)a[i]] = q;
        for (uint64_t runs = __ballot(more); runs; runs &= runs - 1) {
            const uint32_t from = j0 + __builtin_ctzll(runs), its = row(from);
            float sum = 0.f;
            uint32_t i = from + lane;
            for (; i < n && row(i) == its; i += 64) sum += share(i);
            sum = wave_sum(sum);
            for (i = from + lane; i < n && row(i) == its; i += 64) shares[t * n + (uint32_t)a[i]] = sum;
        }
    }
}

// What a token's row of D is held in.
//
// Cross entropy: with s = alpha * dloss, p the softmax and c = 1 - p[target].  D_PACKED, D_APART: p / c
// with -1 at the target, and s * c is X's weight in dW and the product's in dX.  The target's entry
// carries most of the gradient: as -1 it is exact in bf16, where s * (p - 1) would be rounded.  c
// comes from expm1, so a p close to 1 costs no digits.  A c below 2^-25, where fp32 cannot tell p from
// 1, is raised to it; in D_APART, whose fp16 planes hold no entry of 2 or more, one below c_floor, the
// error that z - lse may have: a c that came out too small by it would make the other entries p / c too
// large.  The target's entry is then less than 1 in magnitude, and s * c times D what it was.
//
// Distillation: p, and p - (sum of q over the entries that name the same vocabulary row) at the
// entries.  D_PACKED (bf16): times s, with X and the product as they are, so that dW's factors are
// rounded once (D) and not twice; D_APART (fp32): s is the weight of X and the product.
// So D's entries stay within 1 whatever a token's weight, and a token's dX is its own matter; X times the
// weights is packed apart for dW, in one power of two, since that sums over tokens.
//
// D_WHOLE, for few tokens, whose D is kept wide: s * (p - y), weight 1 (only distillation's is made
// here).
enum DForm { D_PACKED, D_APART, D_WHOLE };
// z and lse are sums of their own: 16 roundings of lse's size between them are ordinary.
__device__ inline float c_floor(float lse) { return 0x1p-20f * (1.f + fabsf(lse)); }

struct TokenArgs {
    Entries e;
    int tokens, vocab, hidden;
    float alpha;
    const void *x, *w;
    long ldx, ldw;
    float* z;                    // forward: [token][entry]
    const float *lse, *dloss, *picked;
    float *scale, *weight, *value;  // gradient, per token (value: per entry): D = exp(z - lse) * scale
    DForm form;
    bool shared;                 // gradient: value holds the entries' shares (vocab_shares_kernel)
    int per;                     // forward: a wave's entries, 1 or kPerWave
    long waves;                  // of token_wave
};
// Entries of one token that a wave takes together where there are enough for all waves: they share the
// reads of X and the waits (4096 tokens of 64 entries, 65536 x 4096 bf16: 298 us one by one, 224; 8000 x 512:
// 77, 58).
constexpr int kPerWave = 4;
__host__ inline int entries_per_wave(long tokens, long k) { return k >= kPerWave && tokens * k >= 32768 ? kPerWave : 1; }

// z[t][k] = alpha * X[t] . W[index[t][k]] by one wave; 0 where there is no entry, NaN where an entry
// lies past the vocabulary.
template <typename T>
__device__ inline float entry_logit(const TokenArgs& a, long t, long k) {
    const i64 v = a.e.index[t * a.e.ld + k];
    if (!a.e.counts(v)) return 0.f;
    if (v < 0 || v >= a.vocab) return NAN;
    return a.alpha * wave_dot((const T*)a.x + t * a.ldx, (const T*)a.w + (size_t)v * a.ldw, a.hidden);
}

// The logits of kPerWave entries from k0 on (those past the last one are not stored), each summed in
// wave_dot's order.
template <typename T>
__device__ inline void entry_logits(const TokenArgs& a, long t, long k0) {
    constexpr int N = 16 / sizeof(T), G = kPerWave;
    const int lane = threadIdx.x & 63, n = a.hidden;
    const T* x = (const T*)a.x + t * a.ldx;
    const T* w[G];
    bool counts[G], named[G], any = false;
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const i64 v = k0 + j < a.e.k ? a.e.index[t * a.e.ld + k0 + j] : -1;
        counts[j] = a.e.counts(v);
        named[j] = counts[j] && v >= 0 && v < a.vocab;
        w[j] = named[j] ? (const T*)a.w + (size_t)v * a.ldw : x;  // x: read in place of a row that is none
        any = any || named[j];
    }
    float s[G][N] = {};
    if (any) {
        int i = lane * N;
#pragma unroll 2
        for (; i + N <= n; i += 64 * N) {
            float c[N], b[G][N];
            load(x + i, c);
#pragma unroll
            for (int j = 0; j < G; ++j) load(w[j] + i, b[j]);
#pragma unroll
            for (int j = 0; j < G; ++j)
#pragma unroll
                for (int q = 0; q < N; ++q) s[j][q] = __builtin_fmaf(c[q], b[j][q], s[j][q]);
        }
        for (; i < n; ++i)
#pragma unroll
            for (int j = 0; j < G; ++j) s[j][0] = __builtin_fmaf((float)x[i], (float)w[j][i], s[j][0]);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < N; ++q) z += s[j][q];
        z = wave_sum(z);
        z = !counts[j] ? 0.f : named[j] ? a.alpha * z : NAN;
        if (lane == 0 && k0 + j < a.e.k) a.z[t * a.e.k + k0 + j] = z;
    }
}

// The work of wave i: forward, the logits of `per` entries; gradient, one token's scale, weight, values.
// Returns that weight, 0 for a token that does not count.
template <typename T, bool GRAD>
__device__ inline float token_wave(const TokenArgs& a, long i) {
    const int lane = threadIdx.x & 63;
    const Entries& e = a.e;
    if constexpr (!GRAD) {
        if (a.per > 1) {
            const long groups = (e.k + kPerWave - 1) / kPerWave;
            entry_logits<T>(a, i / groups, i % groups * kPerWave);
            return 0.f;
        }
        const float z = entry_logit<T>(a, i / e.k, i % e.k);
        if (lane == 0) a.z[i] = z;
        return 0.f;
    } else {
        const long t = i;
        const float s = a.alpha * a.dloss[t], l = a.lse[t];
        float scale, weight;
        bool counts = true;
        if (!e.teacher) {
            const i64 v = e.index[t * e.ld];
            if (!e.counts(v)) return 0.f;
            const float own = fmaxf(-expm1f(entry_logit<T>(a, t, 0) - l), 0.f);
            const float c = fmaxf(own, a.form == D_APART ? c_floor(l) : 0x1p-25f);
            const bool good = v >= 0 && v < a.vocab;
            scale = good ? 1.f / c : NAN;
            weight = good ? s * c : NAN;
            if (lane == 0) a.value[t] = a.form == D_APART ? -own / c : -1.f;
        } else {
            bool good = true, any = false;
            float top = 0.f, log_total = 0.f;
            if (!a.shared) teacher_stats(e, t, top, log_total);
            const i64* index = e.index + t * e.ld;
            const float* teacher = e.teacher + t * e.ld_teacher;
            for (int k0 = 0; k0 < e.k; k0 += 64) {
                const int k = k0 + lane;
                const i64 v = k < e.k ? index[k] : -1;
                // an entry's share of the teacher is that of all that name its row, 64 of them at a time
                // in the lanes (one by one from memory: 14 us where this takes 6.6, 16 tokens of 64 entries)
                float q = a.shared && v >= 0 ? a.value[t * e.k + k] : 0.f;
                for (int o0 = 0; o0 < e.k && !a.shared; o0 += 64) {
                    const int o = o0 + lane;
                    const i64 row = o < e.k ? index[o] : -1;
                    const float share = row >= 0 ? expf(teacher[o] * e.teacher_alpha - top - log_total) : 0.f;
                    const int rest = e.k - o0 < 64 ? e.k - o0 : 64;
                    for (int i = 0; i < rest; ++i) {
                        const uint32_t low = __builtin_amdgcn_readlane((uint32_t)row, i);
                        const uint32_t high = __builtin_amdgcn_readlane((uint32_t)(row >> 32), i);
                        const float its = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(share), i));
                        q += (i64)((uint64_t)high << 32 | low) == v ? its : 0.f;
                    }
                }
                float d = 0.f;
                if (v >= 0) {
                    any = true;
                    good = good && v < a.vocab;
                    float y = a.picked[t * e.k + k] - l;
                    if (a.form == D_APART) y = y > 0.f ? 0.f : y;  // p <= 1, for its fp16 planes
                    d = (a.form == D_APART ? 1.f : s) * (expf(y) - q);
                }
                if (k < e.k) a.value[t * e.k + k] = d;
            }
            if (!__all(good))  // an entry past the vocabulary: the whole row is NaN, as the loss is
                for (int k = lane; k < e.k; k += 64) a.value[t * e.k + k] = NAN;
            scale = __all(good) ? (a.form == D_APART ? 1.f : s) : NAN;
            weight = a.form == D_APART ? s : 1.f;
            counts = __any(any);
        }
        if (lane == 0) {
            a.scale[t] = scale;
            a.weight[t] = weight;
        }
        return counts ? weight : 0.f;
    }
}

// The largest finite |x|.
__device__ inline float finite_max(float m, float x) { return __builtin_isfinite(x) ? fmaxf(m, fabsf(x)) : m; }
template <int I = 0>
__device__ inline float block_max(float m) {  // of 256 threads; each I once in a kernel
    __shared__ float part[4];
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    return fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
}

struct ScanArgs {
    TokenArgs t;
    Counted c;
    int token_blocks;
    float* x_part;    // when wanted (gradient): token_blocks maxima of |weight * X|'s finite values
    float* w_part;    // max_blocks maxima of |W|'s finite values
    int max_blocks;
};

// One wave's part of the largest finite |x * f|, four values of a row a lane.
template <typename T>
__device__ inline float row_max(const T* s, int n, float f, float m) {
    int k = (threadIdx.x & 63) * 4;
#pragma unroll 4
    for (; k + 4 <= n; k += 256) {
        float v[4];
        load(s + k, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) m = finite_max(m, v[q] * f);
    }
    for (; k < n; ++k) m = finite_max(m, (float)s[k] * f);
    return m;
}

// All that reads the inputs alone, in one launch: workgroup 0 counts, the next token_blocks look at
// four entries or tokens at a time each, the rest (fp32) at W's magnitude.
template <typename T, bool GRAD>
__global__ void __launch_bounds__(256) vocab_scan_kernel(ScanArgs a) {
    int b = blockIdx.x;
    if (b == 0) return count_tokens(a.t.e, a.t.tokens, a.c);
    b -= 1;
    const int wave = threadIdx.x >> 6;
    if (b < a.token_blocks) {
        float m = 0.f;
        for (long i = (long)b * 4 + wave; i < a.t.waves; i += (long)a.token_blocks * 4) {
            const float weight = token_wave<T, GRAD>(a.t, i);
            if (GRAD && a.x_part && weight != 0.f) m = row_max((const T*)a.t.x + i * a.t.ldx, a.t.hidden, weight, m);
        }
        if (!GRAD || !a.x_part) return;
        m = block_max(m);
        if (threadIdx.x == 0) a.x_part[b] = m;
        return;
    }
    b -= a.token_blocks;
    float m = 0.f;
    for (long r = b * 4 + wave; r < a.t.vocab; r += a.max_blocks * 4)  // long: a step past the last row
        m = row_max((const T*)a.t.w + (size_t)r * a.t.ldw, a.t.hidden, 1.f, m);
    m = block_max<1>(m);
    if (threadIdx.x == 0) a.w_part[b] = m;
}

// N values of a row that has `cols`, zero past them (and where there is no row).
template <typename T, int N>
__device__ inline void load_row(const T* s, int k, int cols, float (&v)[N]) {
    if (s && k + N <= cols) return load(s + k, v);
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = s && k + q < cols ? (float)s[k + q] : 0.f;
}

struct PackArgs {
    int cols, kp;         // hidden size, and what it is padded to with zeros
    long pitch;
    // X: the counted tokens' rows, and zero rows to the next multiple of 256
    const void* x;
    long ldx;
    const int *rows, *count;
    int x_blocks;
    char* x_out;
    const float* weight;  // per token
    char* scaled;         // when wanted: the rows times their weight
    float* x_unit;        // P = 2: each row in its own power of two, x_unit what a packed unit stands for
    // P = 2, `scaled`: in the power of two of their largest value (x_parts maxima), x_most what a packed
    // unit stands for
    const float* x_part;
    int x_parts;
    float* x_most;
    // W: `vocab` rows, and zero rows to the next multiple of 256
    const void* w;
    long ldw;
    int vocab, w_rows;    // w_rows of them by one workgroup
    char* w_out;
    // P = 2: in the power of two of its largest value (w_parts maxima), w_unit[0] what a packed unit
    // stands for; by row: each row in its own, w_unit[row]
    const float* w_part;
    int w_parts;
    float* w_unit;
};

template <typename T, int P>
__device__ inline void pack_x(const PackArgs& a, int i) {
    const int n = *a.count;
    if (i > 0 && i >= (n + 255) / 256 * 256) return;  // the first says what x_most is, whatever n
    const int t = i < n ? a.rows[i] : 0;
    const T* s = i < n ? (const T*)a.x + (size_t)t * a.ldx : nullptr;
    const float weight = a.scaled && s ? a.weight[t] : 0.f;
    float f = 1.f, g = 1.f;
    if constexpr (P == 2) {
        if (s) {
            float m = 0.f;
            for (int k = threadIdx.x * 4; k < a.cols; k += 1024) {
                float v[4];
                load_row(s, k, a.cols, v);
#pragma unroll
                for (int q = 0; q < 4; ++q) m = finite_max(m, v[q]);
            }
            const int e = scale_exponent(block_max(m));
            f = ldexpf(1.f, e);
            if (threadIdx.x == 0) a.x_unit[i] = ldexpf(1.f, -e);
        }
        if (a.scaled) {
            float m = 0.f;
            for (int j = threadIdx.x; j < a.x_parts; j += 256) m = fmaxf(m, a.x_part[j]);
            const int e = scale_exponent(block_max<1>(m));
            g = ldexpf(1.f, e);
            if (i == 0 && threadIdx.x == 0) *a.x_most = ldexpf(1.f, -e);
        }
    }
    for (int k = threadIdx.x * 4; k < a.kp; k += 1024) {
        float v[4], x[4];
        load_row(s, k, a.cols, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = v[q] * f;
        store4<P>(a.x_out + (size_t)i * a.pitch, k, x);
        if (!a.scaled) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = v[q] * weight * g;
        store4<P>(a.scaled + (size_t)i * a.pitch, k, x);
    }
}

// Row i of W by one wave, in its own power of two.  The row is read once: up to kHeld chunks of 256 stay
// in registers between the search for its largest value and the stores.
template <typename T>
__device__ inline void pack_w_row(const PackArgs& a, int i) {
    constexpr int kHeld = 8;
    const int lane = threadIdx.x & 63;
    const T* s = i < a.vocab ? (const T*)a.w + (size_t)i * a.ldw : nullptr;
    char* out = a.w_out + (size_t)i * a.pitch;
    float v[kHeld][4], m = 0.f;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const int k = c * 256 + lane * 4;
        if (k < a.kp) load_row(s, k, a.cols, v[c]);
    }
#pragma unroll
    for (int c = 0; c < kHeld; ++c)
        if (c * 256 + lane * 4 < a.kp)
#pragma unroll
            for (int q = 0; q < 4; ++q) m = finite_max(m, v[c][q]);
    for (int k = kHeld * 256 + lane * 4; k < a.cols; k += 256) {
        float w[4];
        load_row(s, k, a.cols, w);
#pragma unroll
        for (int q = 0; q < 4; ++q) m = finite_max(m, w[q]);
    }
    m = wave_max(m);
    const int e = scale_exponent(m);
    const float f = ldexpf(1.f, e);
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const int k = c * 256 + lane * 4;
        if (k >= a.kp) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[c][q] *= f;
        store4<2>(out, k, v[c]);
    }
    for (int k = kHeld * 256 + lane * 4; k < a.kp; k += 256) {
        float w[4];
        load_row(s, k, a.cols, w);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] *= f;
        store4<2>(out, k, w);
    }
    if (lane == 0) a.w_unit[i] = ldexpf(1.f, -e);
}

// Rows of W for one workgroup: 4, in bf16 as many as give each thread 8 values (a power of two; both
// packings of a step, 400 tokens, 60000 x 100: 15 us, with 4 rows 23).  In fp32 that many are no faster
// (45 us either way), and a number that the kernel does not know costs both 28 us of 137 (1001 tokens,
// 50021 x 1000).
constexpr int kPackRows = 4;
template <int P>
__host__ inline int pack_rows(int kp) {
    int rows = kPackRows;
    while (P == 1 && rows < 32 && 2 * rows * kp <= 2048) rows *= 2;
    return rows;
}

// The packed operands, in one launch: x_blocks workgroups take a row of X each, the rest w_rows rows
// of W.  Bound by memory: 200 MB read and 200 MB written (1001 tokens, 50021 x 1000, fp32) take 68 us,
// where a copy of that size takes 74, and 96 after kernels that left the caches full of results.
template <typename T, int P, bool BY_ROW>
__global__ void __launch_bounds__(256) vocab_pack_kernel(PackArgs a) {
    if ((int)blockIdx.x < a.x_blocks) return pack_x<T, P>(a, blockIdx.x);
    const int w_rows = P == 2 ? kPackRows : a.w_rows, row0 = (blockIdx.x - a.x_blocks) * w_rows;
    if constexpr (BY_ROW) {
        static_assert(kPackRows == 4, "a wave a row");
        pack_w_row<T>(a, row0 + (threadIdx.x >> 6));
        return;
    }
    // the workgroup's rows as one line of chunks of 8 values, the first chunk read before the search
    // for the unit
    const uint32_t per = (uint32_t)a.kp / 8, chunks = per * w_rows;
    const T* s = (const T*)a.w + (size_t)row0 * a.ldw;
    char* out = a.w_out + (size_t)row0 * a.pitch;
    float v[8];
    uint32_t at = 0;
    auto fetch = [&](uint32_t i) {
        const int r = (int)(i / per), k = (int)(i - r * per) * 8;
        at = (uint32_t)(r * a.pitch) + (uint32_t)Planes<P>::at(k, 0);
        load_row(row0 + r < a.vocab ? s + r * a.ldw : nullptr, k, a.cols, v);
    };
    uint32_t i = threadIdx.x;
    if (i < chunks) fetch(i);
    float f = 1.f;
    if constexpr (P == 2) {
        float m = 0.f;
        for (int j = threadIdx.x; j < a.w_parts; j += 256) m = fmaxf(m, a.w_part[j]);
        const int e = scale_exponent(block_max<2>(m));
        f = ldexpf(1.f, e);
        if (row0 == 0 && threadIdx.x == 0) *a.w_unit = ldexpf(1.f, -e);
    }
    for (;;) {
        if (i >= chunks) break;
        typename Planes<P>::Half8 o[P];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            typename Planes<P>::Half x[P];
            split<P>(P == 2 ? v[j] * f : v[j], x);
#pragma unroll
            for (int p = 0; p < P; ++p) o[p][j] = x[p];
        }
        if constexpr (P == 1) {
            *(typename Planes<P>::Half8*)(out + at) = o[0];
        } else {
            // Four lanes hold the two planes of a slab: with the next four they trade halves, so that
            // each store writes whole lines of 128 bytes.  chunks is a multiple of 8: both have one.
            // Stored past the caches: the products read it from memory either way (a step's two: 135 us; cached 141).
            typedef int Int4 __attribute__((ext_vector_type(4)));
            const bool odd = threadIdx.x & 4;
            const Int4 hi = __builtin_bit_cast(Int4, o[0]), lo = __builtin_bit_cast(Int4, o[P - 1]);
            Int4 other;
#pragma unroll
            for (int j = 0; j < 4; ++j) other[j] = __shfl_xor(odd ? hi[j] : lo[j], 4);
            const uint32_t from = __shfl_xor((int)at, 4);
            __builtin_nontemporal_store(odd ? other : hi, (Int4*)(out + (odd ? from + 64 : at)));
            __builtin_nontemporal_store(odd ? lo : other, (Int4*)(out + (odd ? at + 64 : from)));
        }
        i += 256;
        if (i >= chunks) break;
        fetch(i);
    }
}

// lse of each counted token from its partial maxima and sums, then its loss.  A workgroup takes TX
// tokens, TY threads each: the first kHeld partials of a thread are read once, all together, and those
// past them once for the maxima and once for the sums, so that no load waits for an exponential.  Bound
// by the latency of its few dependent loads.  rows null: a token's partials stand at its own place, whether it counts or
// not, and z of a target that names no row of the vocabulary has not been written.
template <int TX>
__global__ void __launch_bounds__(1024) vocab_loss_kernel(Entries e, const int* rows, const int* count, int tokens,
                                                          int vocab, const float2* part, int parts, int tp,
                                                          const float* z, float* loss, float* lse) {
    constexpr int TY = 1024 / TX;
    __shared__ float slot[16][TX], lses[TX];
    const int n = rows ? *count : tokens, tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = blockIdx.x * TX, i = i0 + tx;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (i0 >= n) return;
    constexpr int kHeld = 8;
    float2 held[kHeld];
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
        const int p = ty + r * TY;
        held[r] = i < n && p < parts ? part[(size_t)p * tp + i] : make_float2(-INFINITY, 0.f);
    }
    float top = -INFINITY;
#pragma unroll
    for (int r = 0; r < kHeld; ++r) top = fmaxf(top, held[r].x);
    if (i < n)
#pragma unroll 8
        for (int p = ty + kHeld * TY; p < parts; p += TY) top = fmaxf(top, part[(size_t)p * tp + i].x);
#pragma unroll
    for (int o = TX; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
    if (lane < TX) slot[wave][tx] = top;
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 16; ++y) top = fmaxf(top, slot[y][tx]);
    __syncthreads();
    const float ref = top == -INFINITY ? 0.f : top;  // nothing but -inf: the sum is 0, or a NaN among its parts
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < kHeld; ++r) sum += held[r].y * expf(held[r].x - ref);
    if (i < n)
#pragma unroll 8
        for (int p = ty + kHeld * TY; p < parts; p += TY) {
            const float2 v = part[(size_t)p * tp + i];
            sum += v.y * expf(v.x - ref);
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
        const int t = rows ? rows[i] : i;
        const bool live = rows || any_entry(e, t, 0);
        lses[tx] = l;
        lse[t] = live ? l : 0.f;
        if (!e.teacher) {
            const bool named = rows || (e.index[t] >= 0 && e.index[t] < vocab);
            // z and l are sums of their own: of a confident token the difference may come out below 0
            const float d = l - (named ? z[t] : NAN);
            loss[t] = !live || d < 0.f ? 0.f : d;
        }
    }
    if (!e.teacher) return;
    __syncthreads();
    for (int y = wave; y < TX; y += 16) {
        if (i0 + y >= n) break;
        const int t = rows ? rows[i0 + y] : i0 + y;
        const float l = lses[y];
        if (!rows && !any_entry(e, t, 0)) {
            if (lane == 0) loss[t] = 0.f;
            continue;
        }
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

// Puts the values of a teacher's entries into D where they fall into this piece (P = 0: a D in fp32).
template <int P>
__global__ void __launch_bounds__(256) vocab_patch_kernel(Entries e, int tokens, int v0, int vocab, const int* pos,
                                                          const float* value, char* d, long d_pitch) {
    const long j = (long)blockIdx.x * 256 + threadIdx.x;
    if (j >= (long)tokens * e.k) return;
    const long t = j / e.k, k = j - t * e.k;
    const int i = P == 0 ? (int)t : pos[t];
    const i64 v = e.index[t * e.ld + k];
    if (i < 0 || !e.counts(v) || v < v0 || v >= v0 + vocab) return;
    if constexpr (P == 0) {
        ((float*)(d + (size_t)i * d_pitch))[v - v0] = value[j];
        return;
    }
    store1<P == 2 ? 2 : 1>(d + (size_t)i * d_pitch, v - v0, P == 2 ? value[j] * kDScale : value[j]);
}

// dX of every token: the sum of its product's parts, or 0 where it does not count.  TY groups of
// threads take every TY-th part each: 16 for few tokens, whose product has many parts, 1 for others.
// P = 0: a token's parts stand at its own place and need no scale.
template <typename T, int P, int TY>
__global__ void __launch_bounds__(256) vocab_dx_out_kernel(Entries e, const int* pos, const int* count, int hidden,
                                                           const float* acc, DxCut cut, int hp, const float* weight,
                                                           T* dx, long ld) {
    constexpr int TX = 256 / TY;
    typedef T Row __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    const int t = blockIdx.x, i = P > 0 ? pos[t] : any_entry(e, t, 0) ? t : -1;
    const int splits = P > 0 ? cut.splits(*count) : cut.groups;
    const size_t rows = P > 0 ? cut.rows(*count) : cut.bn;
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, h = (blockIdx.y * TX + tx) * 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (i >= 0 && h < hidden)
#pragma unroll 4
        for (int z = ty; z < splits; z += TY) v += *(const f32x4*)(acc + (z * rows + i) * hp + h);
    if constexpr (TY > 1) {
        __shared__ f32x4 part[TY][TX];
        part[ty][tx] = v;
        __syncthreads();
        for (int y = 1; y < TY; ++y) v += part[y][tx];
    }
    if (ty > 0 || h >= hidden) return;
    float s = 0.f;
    if (i >= 0) s = P == 0 ? 1.f : P == 1 ? weight[t] : weight[t] / kDScale;
    Row o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = (T)(i < 0 ? 0.f : v[q] * s);
    T* out = dx + (size_t)t * ld + h;
    if (h + 4 <= hidden)
        *(Row*)out = o;
    else
        for (int q = 0; h + q < hidden; ++q) out[q] = o[q];
}

}  // namespace vocab
}  // namespace libsgemm
