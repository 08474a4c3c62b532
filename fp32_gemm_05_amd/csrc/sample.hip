// sample.hip -- entry points of the drawing of tokens: argument checks, workspace, launches.
#include "../../include/sample.h"
#include "kernel_sample.hpp"

namespace libsgemm {
namespace sample {
namespace {

constexpr int kMaxRows = 1 << 21, kMaxVocab = 1 << 23;  // 2^23 probabilities of 2^40 are below 2^64

// Whether a row is shared by several workgroups: rows of more than 8 vectors a thread (32768 fp32 logits, 65536 bf16), what the
// row kernel keeps in registers, where at most 128 rows leave half of the 256 compute units idle, until about all have a
// workgroup, each with a vector a thread or more.  Four launches cost some 10 us more than one, which the passes over
// 131072 logits win back (us, shared / a workgroup a row; top_p 0.9, no filter, top_k 2000):
//   1 row    fp32 65536: 35 / 29, 23 / 20, 37 / 35;   fp32 131072: 35 / 43, 23 / 34, 37 / 53;   bf16 131072: 36 / 41, 24 / 27, 36 / 54
//   64 rows  fp32 65536: 43 / 39, 27 / 20, 42 / 36;   fp32 131072: 54 / 71, 33 / 35, 49 / 54;   bf16 131072: 50 / 64, 28 / 28, 50 / 55
//   128 rows fp32 36864: 44 / 29, 28 / 15, 44 / 28;   fp32 131072: 78 / 83, 47 / 41, 69 / 67;   bf16 131072: 66 / 66, 38 / 28, 170 / 107
// With 8 vectors or fewer sharing loses throughout (1 row of fp32 32768: 33 / 21, 22 / 12, 35 / 24; 64 of bf16 65536: 43 / 38,
// 25 / 16, 42 / 34).  In between, and of 128 rows, it loses too but for top_p of bf16: the limits stand early.
struct Split {
    int splits, vectors;
    long state, count, mass, list, bytes;
};
Split split_of(long size, long rows, long vocab) {
    const long n = 16 / size, all = (vocab + kThreads * n - 1) / (kThreads * n);
    Split p{1, (int)all, 0, 0, 0, 0, 0};
    if (all <= 8 || rows > 128 || rows == 0) return p;
    long most = 256 / rows < kMostSplits ? 256 / rows : kMostSplits;
    if (most > all) most = all;
    p.vectors = (int)((all + most - 1) / most);
    p.splits = (int)((all + p.vectors - 1) / p.vectors);
    auto take = [&](long bytes) {
        const long at = p.bytes;
        p.bytes = (at + bytes + 255) / 256 * 256;
        return at;
    };
    p.state = take(sizeof(State) * rows);
    p.count = take(4L * kBins * rows);
    p.mass = take(8L * kBins * rows);
    p.list = take(8L * kList * rows);
    return p;
}

template <typename T>
void launch(int rows, const Args& a, char* work, hipStream_t stream) {
    constexpr int N = 16 / sizeof(T);
    const Split p = split_of(sizeof(T), rows, a.vocab);
    // a small top_k of all rows needs one pass after the largest, which sharing does not pay for (64 rows of 131072 bf16, us,
    // in the row kernel / shared: top_k 50 24 / 38, 512 37 / 43; with top_p 0.9 26 / 40, 42 / 48; 1 row of 131072 fp32: 22 /
    // 31, 36 / 35)
    const bool quick = !a.top_ks && a.top_k > 0 && a.top_k <= kThreads / 2;
    if (p.splits > 1 && !quick) {
        const SplitArgs s{a, p.splits, p.vectors, (State*)(work + p.state), (uint32_t*)(work + p.count),
                          (u64*)(work + p.mass), (u64*)(work + p.list)};
        sample_top_kernel<T, 4><<<rows * p.splits, kThreads, 0, stream>>>(s);
        sample_count_kernel<T, 4><<<rows * p.splits, kThreads, 0, stream>>>(s);
        sample_border_kernel<T, 4><<<rows * p.splits, kThreads, 0, stream>>>(s);
        sample_token_kernel<T, 4><<<rows, kThreads, 0, stream>>>(s);
    } else if (a.vocab <= 4 * kThreads * N) {
        sample_row_kernel<T, 4><<<rows, kThreads, 0, stream>>>(a);
    } else {
        sample_row_kernel<T, 8><<<rows, kThreads, 0, stream>>>(a);
    }
}

int run(int dtype, int rows, const Args& a, char* work, hipStream_t stream) {
    (void)hipGetLastError();
    if (dtype == SAMPLE_F32)
        launch<float>(rows, a, work, stream);
    else
        launch<__bf16>(rows, a, work, stream);
    return (int)hipGetLastError();
}

}  // namespace
}  // namespace sample
}  // namespace libsgemm

extern "C" {

long long vocab_sample_workspace(int dtype, int T, int V) {
    if (dtype != SAMPLE_F32 && dtype != SAMPLE_BF16) return -1;
    if (T < 0 || T > libsgemm::sample::kMaxRows) return -2;
    if (V < 1 || V > libsgemm::sample::kMaxVocab) return -3;
    const libsgemm::sample::Split p = libsgemm::sample::split_of(dtype == SAMPLE_F32 ? 4 : 2, T, V);
    return p.splits > 1 ? p.bytes : 0;
}

int vocab_sample(int dtype, int T, int V, const void* logits, int ld, const float* u, float temperature,
                 const float* temperatures, long long top_k, const long long* top_ks, float top_p, const float* top_ps,
                 float min_p, const float* min_ps, long long* token, void* work, long long work_bytes,
                 hipStream_t stream) {
    const long need = vocab_sample_workspace(dtype, T, V);
    if (need < 0) return (int)need;
    if (ld < V) return -5;
    if (T == 0) return 0;
    if (!logits || (uintptr_t)logits % (dtype == SAMPLE_F32 ? 4 : 2)) return -4;
    if (!u) return -6;
    if (!temperatures && !(temperature >= 0.f && temperature < INFINITY)) return -7;
    if (!top_ps && top_p != top_p) return -11;
    if (!min_ps && min_p != min_p) return -13;
    if (!token) return -15;
    if (need > 0 && (!work || (uintptr_t)work % 16)) return -16;
    if (work_bytes < need) return -17;
    const libsgemm::sample::Args a{logits, ld, V, u, temperatures, temperature, top_ks, top_k, top_ps, top_p,
                                   min_ps, min_p, token};
    return libsgemm::sample::run(dtype, T, a, (char*)work, stream);
}

}  // extern "C"
