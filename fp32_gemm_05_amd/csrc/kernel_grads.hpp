// kernel_grads.hpp -- the norm of many gradients and clipping by it (gfx950).
//
// Both are bound by memory: one read for the norm, a read and a write for the clipping.  The tensors' addresses and
// sizes go with launches of grads_table_kernel, in their arguments, kTable tensors at a time (a copy from host
// memory would wait for it, or read it again when a graph is replayed), which put them into the workspace and note for
// each piece, what a workgroup takes of a tensor, whose it is.  Read from the arguments by each workgroup they would
// come from host memory, several times one after the other: the norm of 30 tensors of 8 MB took 19 us so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace libsgemm {
namespace grads {

struct Entry {
    const void* x;
    void* out;
    long cols;
    uint32_t rows, ld, ld_out;
    uint32_t first, pieces;  // of this tensor
    uint32_t half;           // bf16
};
constexpr int kTable = 72;  // a launch's arguments stay below 4 KB
struct Table {
    Entry e[kTable];
};

// A workgroup each tensor.
__global__ void __launch_bounds__(256) grads_table_kernel(Table t, uint32_t tensor0, Entry* entries, uint32_t* tensor_of) {
    const Entry e = t.e[blockIdx.x];
    const uint32_t tensor = tensor0 + blockIdx.x;
    if (threadIdx.x == 0) entries[tensor] = e;
    for (uint32_t i = threadIdx.x; i < e.pieces; i += 256) tensor_of[e.first + i] = tensor;
}

// Pieces that a tensor is cut into: parts of a row, or as many whole rows as hold at most `piece` elements.
__host__ inline long pieces_of(long rows, long cols, long piece) {
    if (rows == 0 || cols == 0) return 0;
    if (cols >= piece) return rows * ((cols + piece - 1) / piece);
    const long per = piece / cols;
    return (rows + per - 1) / per;
}

// load(slot, row, column, elements) and then use(the same) for a piece's vectors of 16 bytes, U of them on their way
// at once.  A row's last vector, where it is not whole, is given as a whole one that ends with the row, `elements` of
// whose last were not in the one before it; a row shorter than a vector is given as it is, with a column of 0.
template <typename T, int U, class L, class F>
__device__ inline void each(const Entry& e, uint32_t i, uint32_t piece, L load, F use) {
    constexpr int N = 16 / sizeof(T);
    const int x = threadIdx.x;
    if (e.cols >= piece) {
        const uint32_t parts = (uint32_t)((e.cols + piece - 1) / piece), r = i / parts;
        const long c0 = (long)(i - r * parts) * piece, c1 = c0 + piece < e.cols ? c0 + piece : e.cols;
        long c = c0 + x * N;
        for (; c + (256 * (U - 1) + 1) * N <= c1; c += 256 * U * N) {
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, r, c + 256 * u * N, N);
#pragma unroll
            for (int u = 0; u < U; ++u) use(u, r, c + 256 * u * N, N);
        }
        // (a last part shorter than a vector reaches back into the part before it)
        for (; c < c1; c += 256 * N) {
            const bool whole = c + N <= c1;
            load(0, r, whole ? c : c1 - N, whole ? N : (int)(c1 - c));
            use(0, r, whole ? c : c1 - N, whole ? N : (int)(c1 - c));
        }
        return;
    }
    const uint32_t cols = (uint32_t)e.cols, per = piece / cols, r0 = i * per;
    const uint32_t rows = r0 + per < e.rows ? per : e.rows - r0, each_row = (cols + N - 1) / N, all = rows * each_row;
    for (uint32_t v = x; v < all; v += 256 * U) {
        uint32_t row[U], col[U];
        int n[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w = v + 256 * u, r = w / each_row, c = (w - r * each_row) * N;
            row[u] = r0 + r;
            col[u] = c + N <= cols ? c : cols < N ? 0 : cols - N;
            n[u] = w >= all ? 0 : c + N <= cols ? N : (int)(cols - c);
            if (n[u] > 0) load(u, row[u], (long)col[u], n[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (n[u] > 0) use(u, row[u], (long)col[u], n[u]);
    }
}

template <typename T, int N>
struct Vec {
    T v[N];
};
// A vector of `each`; of a row shorter than one its n elements, at the end, behind zeros.
template <typename T, int N>
__device__ inline void fetch(Vec<T, N>& v, const T* p, long cols, int n) {
    if (cols >= N)
        __builtin_memcpy(v.v, p, 16);
    else
#pragma unroll
        for (int q = 0; q < N; ++q) v.v[q] = q >= N - n ? p[q - (N - n)] : (T)0.f;
}

template <typename T>
__device__ inline double squares(const Entry& e, uint32_t i, uint32_t piece) {
    constexpr int N = 16 / sizeof(T), U = 4;
    double s = 0;
    Vec<T, N> v[U];
    each<T, U>(
        e, i, piece, [&](int u, uint32_t r, long c, int n) { fetch(v[u], (const T*)e.x + (size_t)r * e.ld + c, e.cols, n); },
        [&](int u, uint32_t, long, int n) {
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const double x = q >= N - n ? (double)(float)v[u].v[q] : 0.;
                s = __builtin_fma(x, x, s);
            }
        });
    return s;
}

// The sum of a workgroup's values, in every thread.
template <int NT>
__device__ inline double block_sum(double s) {
    __shared__ double parts[NT / 64];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0;
    for (int w = 0; w < NT / 64; ++w) s += parts[w];
    return s;
}

__global__ void __launch_bounds__(256) grads_squares_kernel(const Entry* entries, const uint32_t* tensor_of,
                                                            uint32_t piece, double* sums) {
    const Entry e = entries[tensor_of[blockIdx.x]];
    const uint32_t i = blockIdx.x - e.first;
    const double s = block_sum<256>(e.half ? squares<__bf16>(e, i, piece) : squares<float>(e, i, piece));
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// norm, and the clipping's factor where it is wanted.
__global__ void __launch_bounds__(1024) grads_norm_kernel(const double* sums, long count, float* norm, float* factor,
                                                          float max_norm, float eps) {
    double s = 0;
#pragma unroll 8
    for (long i = threadIdx.x; i < count; i += 1024) s += sums[i];
    s = sqrt(block_sum<1024>(s));
    if (threadIdx.x > 0) return;
    *norm = (float)s;
    if (!factor) return;
    const double d = s + (double)eps, f = d == 0. ? 1. : (double)max_norm / d;
    *factor = f >= 1. ? 1.f : (float)f;  // a NaN stays
}

template <typename T>
__device__ inline void scale(const Entry& e, uint32_t i, uint32_t piece, float f) {
    constexpr int N = 16 / sizeof(T), U = 4;
    const bool in_place = e.out == e.x;
    Vec<T, N> v[U];
    each<T, U>(
        e, i, piece, [&](int u, uint32_t r, long c, int n) { fetch(v[u], (const T*)e.x + (size_t)r * e.ld + c, e.cols, n); },
        [&](int u, uint32_t r, long c, int n) {
            T* o = (T*)e.out + (size_t)r * e.ld_out + c;
#pragma unroll
            for (int q = 0; q < N; ++q) v[u].v[q] = (T)((float)v[u].v[q] * f);
            // the elements that two vectors share get the same values twice, but in place, where one lane
            // alone may read and write an element
            if (n == N || (e.cols >= N && !in_place)) {
                __builtin_memcpy(o, v[u].v, 16);
                return;
            }
            if (e.cols < N) o -= N - n;
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q >= N - n) o[q] = v[u].v[q];
        });
}

// From the last piece to the first: what the norm's pass has read last is still in the caches.
__global__ void __launch_bounds__(256) grads_scale_kernel(const Entry* entries, const uint32_t* tensor_of,
                                                          uint32_t piece, const float* factor) {
    const uint32_t b = gridDim.x - 1 - blockIdx.x;
    const Entry e = entries[tensor_of[b]];
    const float f = *factor;
    if (f == 1.f && e.out == e.x) return;
    if (e.half)
        scale<__bf16>(e, b - e.first, piece, f);
    else
        scale<float>(e, b - e.first, piece, f);
}

}  // namespace grads
}  // namespace libsgemm
