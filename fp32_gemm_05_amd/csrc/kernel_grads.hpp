// kernel_grads.hpp -- the norm of many gradients and clipping by it (gfx950).
//
// Both are bound by memory: one read for the norm, a read and a write for the clipping.  The tensors' addresses and
// sizes go with the launch, in its arguments, kTable tensors at a time: nothing is copied to the device beforehand.
// A workgroup takes a piece of one tensor.  The clipping walks the pieces from the last to the first, so that what the
// norm's pass has read last is found in the caches.
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
    uint32_t last;  // pieces of the tensors up to this one
};
constexpr int kTable = 90;  // of 40 bytes: a launch's arguments stay below 4 KB
struct Table {
    int count;
    uint32_t piece;   // elements of a piece, a multiple of 8
    uint32_t bf16[3]; // a bit for each tensor
    Entry e[kTable];
};

// The piece `b` of the table, or a tensor's pieces from its last to its first: the tensor, and the rows [r0, r1) and
// columns [c0, c1) of it.
struct Piece {
    int tensor;
    uint32_t r0, r1;
    long c0, c1;
};
template <bool BACK>
__device__ inline Piece piece_of(const Table& t, uint32_t b) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (b < t.e[mid].last)
            hi = mid;
        else
            lo = mid + 1;
    }
    const Entry& e = t.e[lo];
    const uint32_t i = BACK ? e.last - 1 - b : b - (lo > 0 ? t.e[lo - 1].last : 0);
    if (e.cols >= t.piece) {  // a part of a row
        const uint32_t parts = (uint32_t)((e.cols + t.piece - 1) / t.piece), r = i / parts;
        const long c0 = (long)(i - r * parts) * t.piece, c1 = c0 + t.piece;
        return {lo, r, r + 1, c0, c1 < e.cols ? c1 : e.cols};
    }
    const uint32_t per = t.piece / (uint32_t)e.cols, r0 = i * per, r1 = r0 + per;
    return {lo, r0, r1 < e.rows ? r1 : e.rows, 0, e.cols};
}

// Pieces that a tensor is cut into.
__host__ inline long pieces_of(long rows, long cols, long piece) {
    if (rows == 0 || cols == 0) return 0;
    if (cols >= piece) return rows * ((cols + piece - 1) / piece);
    const long per = piece / cols;
    return (rows + per - 1) / per;
}

template <typename T>
__device__ inline double squares(const Entry& e, const Piece& p) {
    constexpr int N = 16 / sizeof(T);
    double s = 0;
    for (uint32_t r = p.r0; r < p.r1; ++r) {
        const T* row = (const T*)e.x + (size_t)r * e.ld;
#pragma unroll 4
        for (long c = p.c0 + threadIdx.x * N; c < p.c1; c += 256 * N) {
            T v[N] = {};
            if (c + N <= p.c1)
                __builtin_memcpy(v, row + c, 16);
            else
                for (int i = 0; c + i < p.c1; ++i) v[i] = row[c + i];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const double x = (double)(float)v[i];
                s = __builtin_fma(x, x, s);
            }
        }
    }
    return s;
}

// Sums of a workgroup's values, in every thread of wave 0.
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

__global__ void __launch_bounds__(256) grads_squares_kernel(Table t, double* sums) {
    const Piece p = piece_of<false>(t, blockIdx.x);
    const Entry& e = t.e[p.tensor];
    const bool half = t.bf16[p.tensor >> 5] >> (p.tensor & 31) & 1;
    const double s = block_sum<256>(half ? squares<__bf16>(e, p) : squares<float>(e, p));
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// norm, and the clipping's factor where it is wanted.
__global__ void __launch_bounds__(1024) grads_norm_kernel(const double* sums, long count, float* norm, float* factor,
                                                          float max_norm, float eps) {
    double s = 0;
    for (long i = threadIdx.x; i < count; i += 1024) s += sums[i];
    s = sqrt(block_sum<1024>(s));
    if (threadIdx.x > 0) return;
    *norm = (float)s;
    if (!factor) return;
    const double f = (double)max_norm / (s + (double)eps);
    *factor = f >= 1. ? 1.f : (float)f;  // a NaN stays
}

template <typename T>
__device__ inline void scale(const Entry& e, const Piece& p, float f) {
    constexpr int N = 16 / sizeof(T);
    for (uint32_t r = p.r0; r < p.r1; ++r) {
        const T* row = (const T*)e.x + (size_t)r * e.ld;
        T* out = (T*)e.out + (size_t)r * e.ld_out;
#pragma unroll 4
        for (long c = p.c0 + threadIdx.x * N; c < p.c1; c += 256 * N) {
            if (c + N <= p.c1) {
                T v[N];
                __builtin_memcpy(v, row + c, 16);
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = (T)((float)v[i] * f);
                __builtin_memcpy(out + c, v, 16);
            } else {
                for (int i = 0; c + i < p.c1; ++i) out[c + i] = (T)((float)row[c + i] * f);
            }
        }
    }
}

__global__ void __launch_bounds__(256) grads_scale_kernel(Table t, const float* factor) {
    const Piece p = piece_of<true>(t, blockIdx.x);
    const Entry& e = t.e[p.tensor];
    const float f = *factor;
    if (f == 1.f && e.out == e.x) return;
    if (t.bf16[p.tensor >> 5] >> (p.tensor & 31) & 1)
        scale<__bf16>(e, p, f);
    else
        scale<float>(e, p, f);
}

}  // namespace grads
}  // namespace libsgemm
