// sample.hip -- entry points of the drawing of tokens: argument checks, workspace, launches.
#include "../../include/sample.h"
#include "kernel_sample.hpp"

namespace libsgemm {
namespace sample {
namespace {

constexpr int kMaxRows = 1 << 21, kMaxVocab = 1 << 23;  // 2^23 probabilities of 2^40 are below 2^64

// Whether a row is shared by several workgroups: of long rows, where the rows leave half of the 256 compute units
// idle, until about all have a workgroup, each with a vector a thread or more.
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
    // a small top_k of all rows needs one pass after the largest, which sharing does not pay for (64 rows of 131072 bf16,
    // top_k 50, top_p 0.9: 24 us, shared 40; without top_k 68, shared 53)
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
