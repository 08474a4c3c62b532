// kernel_linear.hpp -- the kernels of the linear layer with an epilogue (gfx950):
//
//   Z = X W^T + bias,  Y = act(Z) + residual;   dZ = dY act'(Z),  dX = dZ W,  dW = dZ^T X,  dbias = sum_t dZ.
//
// More than kFewTokens tokens: the tile loop of kernel_vocab.hpp, fp32 operands on the fp32 MFMA (P = 0: no
// operand is cut into parts, so infinities, NaN and values of any scale come out as an fp32 sum gives them),
// bf16 on the bf16 MFMA.  Output features are the M side of Z, hidden that of dX and dW, so that a lane holds
// four consecutive elements of one row of the result.  Operands are read in place where their rows are whole
// 16-byte quads, k that ends inside a slab included; others are packed first.
//
// At most kFewTokens tokens: one pass over W, straight from memory into the MFMA operands at any alignment
// (the modes of kernel_vocab_few.hpp).
#pragma once

#include "kernel_vocab_few.hpp"

namespace libsgemm {
namespace linear {

using vocab::K_COL;
using vocab::K_ENDS;
using vocab::K_ROW;
using vocab::Operand;
using vocab::Order;
using vocab::Planes;
using vocab::Tile;
using vocab::u32x4;

enum Act { NONE = 0, RELU = 1, GELU = 2, GELU_TANH = 3, SILU = 4 };

// N4 groups of four values of T at any alignment of T, in accesses of up to 16 bytes; the first `left` of them.
template <typename T, int N4>
__device__ inline void load(const T* p, int left, f32x4 (&v)[N4]) {
    T x[4 * N4] = {};
    if (left >= 4 * N4)
        __builtin_memcpy(x, p, sizeof(x));
    else
#pragma unroll
        for (int i = 0; i < 4 * N4 - 1; ++i)
            if (i < left) x[i] = p[i];
#pragma unroll
    for (int i = 0; i < 4 * N4; ++i) v[i / 4][i % 4] = (float)x[i];
}
template <typename T, int N4>
__device__ inline void add(const void* p, long row, long ld, int col, int left, f32x4 (&v)[N4]) {
    f32x4 x[N4];
    load((const T*)p + row * ld + col, left, x);
#pragma unroll
    for (int g = 0; g < N4; ++g) v[g] += x[g];
}
template <typename T, int N4>
__device__ inline void leave(void* p, long row, long ld, int col, int left, const f32x4 (&v)[N4]) {
    T x[4 * N4];
#pragma unroll
    for (int i = 0; i < 4 * N4; ++i) x[i] = (T)v[i / 4][i % 4];
    T* out = (T*)p + row * ld + col;
    if (left >= 4 * N4)
        __builtin_memcpy(out, x, sizeof(x));
    else
#pragma unroll
        for (int i = 0; i < 4 * N4 - 1; ++i)
            if (i < left) out[i] = x[i];
}
template <typename T>
__device__ inline f32x4 load4(const T* p, int n = 4) {
    f32x4 v[1];
    load(p, n, v);
    return v[0];
}

// The normal distribution's upper tail Q(t) = erfc(t / sqrt 2) / 2 for t >= 0 as k P(k) exp(-t^2 / 2), k = 1 /
// (1 + 0.375 t): P of degree 8 fitted to the least largest relative error, 2.3e-7 (gelu from -13 to 0 as measured: 8e-7),
// so that the far negative side of gelu keeps its digits, which 1 + erf loses.  Returns k P(k); half: exp(-t^2 / 4),
// multiplied twice, so that what is a normal number in the end is not lost on the way.
__device__ inline float upper_tail(float t, float& half) {
    // the exponent in two parts, high and low: rounded to one its error would be t^2 2^-24, 8e-6 of the tail at 12
    constexpr double c = 0.36067376022224085;  // log2(e) / 4
    const float a = (float)c * t, a_low = __builtin_fmaf((float)(c - (float)c), t, __builtin_fmaf((float)c, t, -a));
    const float e = a * t, e_low = __builtin_fmaf(a_low, t, __builtin_fmaf(a, t, -e));
    half = __builtin_amdgcn_exp2f(-e) * __builtin_fmaf(-0.69314718055994531f, e_low, 1.f);
    const float k = __builtin_amdgcn_rcpf(__builtin_fmaf(0.375f, t, 1.f));
    float p = -0.0329474956f;
    p = __builtin_fmaf(p, k, 0.137030736f);
    p = __builtin_fmaf(p, k, -0.186776593f);
    p = __builtin_fmaf(p, k, 0.0508598723f);
    p = __builtin_fmaf(p, k, 0.0155141391f);
    p = __builtin_fmaf(p, k, 0.0886697173f);
    p = __builtin_fmaf(p, k, 0.128441304f);
    p = __builtin_fmaf(p, k, 0.149604827f);
    p = __builtin_fmaf(p, k, 0.149603382f);
    return p * k;
}
__device__ inline float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}
constexpr float kTanhA = 0.79788456080286536f, kTanhB = 0.044715f;  // sqrt(2 / pi)

template <int ACT>
__device__ inline float act(float z) {
    if constexpr (ACT == RELU) return z < 0.f ? 0.f : z;  // a NaN stays
    if constexpr (ACT == GELU) {
        float half;
        const float t = fminf(fabsf(z), 20.f), q = upper_tail(t, half);  // Q is 0 in fp32 from 14 on
        return (z < 0.f ? 0.f : z) - half * (half * (t * q));
    }
    // (1 + tanh(w)) / 2 = sigmoid(2 w)
    if constexpr (ACT == GELU_TANH) return z * sigmoid(2.f * kTanhA * z * __builtin_fmaf(kTanhB * z, z, 1.f));
    if constexpr (ACT == SILU) return z * sigmoid(z);
    return z;
}
// The slope of z s, s = 1 / (1 + exp(-w)): s (1 + q (1 - s)) with q = z dw/dz.  exp(-|w|) is taken as the square of `half`,
// so that the slope keeps its digits as long as it is a normal number (exp(-|w|) itself is lost from w = -87 on, where
// the slopes are 10^-36).
__device__ inline float sigmoid_slope(float w, float q) {
    const float half = __builtin_amdgcn_exp2f(-0.72134752044448170f * fabsf(w)), e = half * half;
    const float r = __builtin_amdgcn_rcpf(1.f + e);  // s above 0, 1 - s below
    return w < 0.f ? half * (half * (r * __builtin_fmaf(q, r, 1.f))) : r * __builtin_fmaf(q, e * r, 1.f);
}

template <int ACT>
__device__ inline float slope(float z) {
    if constexpr (ACT == RELU) return z > 0.f ? 1.f : z != z ? z : 0.f;
    // from 20 on each of these slopes is 1 in fp32; below -20 that of gelu and of gelu_tanh is 0 (e^-200 and less), that
    // of silu, z exp(z) there, from -104 on.  With z held to that, z^2 below stays finite.
    constexpr float LEAST = ACT == SILU ? -110.f : -20.f;
    const float c = __builtin_elementwise_maximum(__builtin_elementwise_minimum(z, 20.f), LEAST);
    if constexpr (ACT == GELU) {
        float half;
        const float q = upper_tail(fabsf(c), half);
        return (c < 0.f ? 0.f : 1.f) + half * (half * __builtin_fmaf(c, 0.39894228040143268f, c < 0.f ? q : -q));
    }
    if constexpr (ACT == GELU_TANH) {
        const float w = 2.f * kTanhA * c, b = kTanhB * c;
        return sigmoid_slope(w * __builtin_fmaf(b, c, 1.f), w * __builtin_fmaf(3.f * b, c, 1.f));
    }
    if constexpr (ACT == SILU) return sigmoid_slope(c, c);
    return 1.f;
}
// f(integral_constant) for the activation of a call; uniform.
template <class F>
__device__ inline void by_act(int a, F f) {
    switch (a) {
        case RELU: return f(std::integral_constant<int, RELU>{});
        case GELU: return f(std::integral_constant<int, GELU>{});
        case GELU_TANH: return f(std::integral_constant<int, GELU_TANH>{});
        case SILU: return f(std::integral_constant<int, SILU>{});
        default: return f(std::integral_constant<int, NONE>{});
    }
}

// What becomes of a finished row of sums: rows of `n` tokens or of dW, columns of `m`.
struct Finish {
    int n, m;           // rows and columns of the result
    int act, wide;      // wide: out and residual are fp32 beside bf16 operands
    const void* bias;   // [m] or null
    const void* residual;
    long ld_residual;
    void* z;            // null: not kept; in the operands' type: fp32 beside bf16 operands would move twice the bytes for slopes
                        // off by 1e-3 less (the gradients by 6e-5 of their norm)
    long ld_z;
    void* out;
    long ld;
};

// The bias of 4 N consecutive columns, `left` of which exist; zeros without one.
template <typename T, int N>
__device__ inline void load_bias(const Finish& f, int col, int left, f32x4 (&bias)[N]) {
#pragma unroll
    for (int g = 0; g < N; ++g) bias[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (f.bias && left > 0) load((const T*)f.bias + col, left, bias);
}
// 4 N consecutive columns of a row, `left` of which exist.  FORWARD: not, the sums are stored as they are.
template <bool FORWARD, typename T, int N>
__device__ inline void finish(const Finish& f, const f32x4 (&bias)[N], long row, int col, int left, f32x4 (&v)[N]) {
    auto each = [&](auto body) {
#pragma unroll
        for (int g = 0; g < N; ++g) body(v[g], col + 4 * g, left - 4 * g);
    };
    if constexpr (FORWARD) {
#pragma unroll
        for (int g = 0; g < N; ++g) v[g] += bias[g];
        if (f.z) leave<T>(f.z, row, f.ld_z, col, left, v);
        by_act(f.act, [&](auto which) {
            each([&](f32x4& x, int, int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = act<decltype(which)::value>(x[i]);
            });
        });
        if (sizeof(T) == 2 && f.wide) {
            if (f.residual) add<float>(f.residual, row, f.ld_residual, col, left, v);
            return leave<float>(f.out, row, f.ld, col, left, v);
        }
        if (f.residual) add<T>(f.residual, row, f.ld_residual, col, left, v);
    }
    leave<T>(f.out, row, f.ld, col, left, v);
}

// dbias from the partial sums of `parts` workgroups: 64 columns a workgroup, four parts at a time (whatever the workgroup's
// size, so that the bits are the same).  The first product's workgroups after its tiles do it, beside them (a launch of its
// own took 3.3 - 5 us: the gradients of 777 x 5003 x 1001 bf16 60.8 us, so 58.3).
struct BiasArgs {
    const float* sums;  // [parts][pitch]
    int parts, cols;
    long pitch;
    void* out;
    __host__ __device__ int blocks() const { return (cols + 63) / 64; }
};
template <typename T>
__device__ inline void bias_columns(const BiasArgs& a, int block, float* all) {
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6, c = block * 64 + x;
    float s = 0.f;
    if (y < 4 && c < a.cols)
#pragma unroll 8
        for (int p = y; p < a.parts; p += 4) s += a.sums[(size_t)p * a.pitch + c];
    if (y < 4) all[y * 64 + x] = s;
    __syncthreads();
    if (y > 0 || c >= a.cols) return;
    for (int i = 1; i < 4; ++i) s += all[i * 64 + x];
    ((T*)a.out)[c] = (T)s;
}

struct ProductArgs {
    Operand a, b;          // M side, N side
    int tiles_m, tiles_n;
    int k, slabs, splits;  // of the long axis, cut into `splits` parts of whole slabs
    float* part;           // splits > 1: [split][row of whole tiles][pitch], summed by linear_sum_kernel
    long rows, pitch;
    Finish f;
    BiasArgs bias;         // of a gradient's first product
};

// One product.  With few tiles the long axis is cut, so that the chip is filled, and the parts are
// summed in a fixed order.
//
// What bounds it: large bf16 products power, as the vocabulary head's (8192 x 8192 x 4096: 430 us, 1.28 PFLOP/s, with gelu
// and Z kept 512); fp32 ones the MFMA (4096 x 4096 x 1024: 251 us, 137 TFLOP/s of 157, pipes 87 % busy; 2048 x 4096 x 1024:
// 134 - 150 us, 81 % busy, the rest the first loads and the stores of two rounds of tiles); short bf16 ones latency (777 x
// 5003 x 1001: 20 - 27 us where the matrix pipes need 5: 16 slabs a tile, one round and a part).
template <class T, Order OA, Order OB, bool TAIL, bool FORWARD>
__global__ void __launch_bounds__(T::NT) linear_product_kernel(ProductArgs a) {
    typedef typename Planes<T::kP>::Half E;
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    const int tiles = a.tiles_m * a.tiles_n, z = blockIdx.x / tiles;
    if constexpr (!FORWARD)
        if (z >= a.splits) return bias_columns<E>(a.bias, blockIdx.x - a.splits * tiles, (float*)lds);
    int tm, tn;
    tile_of(blockIdx.x - z * tiles, tiles, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    const int first = (int)((long)a.slabs * z / a.splits), last = (int)((long)a.slabs * (z + 1) / a.splits);
    T t;
    t.template run<OA, OB, TAIL>(lds, a.a, m0, a.b, n0, first, last - first, a.k - (last - 1) * T::BK);
    // The tile leaves through LDS, 32 rows of the result at a time and wave by wave: a lane's accumulators are four
    // columns of 32 rows, and stored from there a line of memory would be written in eight pieces (8192 x 8192 x 4096
    // bf16 with gelu and Z kept: 677 us, so 512).  Row r holds its quad q at q ^ r: writes of 16 rows at one quad
    // and reads of a row's quads in a row are both spread over the banks.
    constexpr int WM = T::kWM, QUADS = WM / 4, N4 = sizeof(E) == 2 ? 2 : 1, LANES = QUADS / N4, ROWS = 64 / LANES;
    static_assert(T::NW * 32 * WM * 4 <= T::LDS_BYTES, "a place for each wave");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 31, h = lane >> 5;
    f32x4* const own = (f32x4*)lds + wave * 32 * QUADS;
    const int m = m0 + (wave / T::WAVES_N) * WM + lane % LANES * 4 * N4, q0 = lane % LANES * N4;
    const int n_wave = n0 + (wave % T::WAVES_N) * T::kWN;
    f32x4 bias[N4];
    if constexpr (FORWARD) load_bias<E>(a.f, m, a.f.m - m, bias);
    wait_vm_lgkm0<0>();
    dl_barrier();  // every wave has read its last slab
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                own[l * QUADS + ((8 * i + 2 * g + h) ^ (l & (QUADS - 1)))] =
                    f32x4{t.acc[i][j][4 * g], t.acc[i][j][4 * g + 1], t.acc[i][j][4 * g + 2], t.acc[i][j][4 * g + 3]};
        wait_vm_lgkm0<0>();  // a wave's own writes before its reads; it shares them with no other wave
#pragma unroll 2
        for (int r = lane / LANES; r < 32; r += ROWS) {
            const int n = n_wave + j * 32 + r;
            f32x4 v[N4];
#pragma unroll
            for (int q = 0; q < N4; ++q) v[q] = own[r * QUADS + ((q0 + q) ^ (r & (QUADS - 1)))];
            if (a.splits > 1) {
                float* out = a.part + (z * a.rows + n) * a.pitch + m;
#pragma unroll
                for (int q = 0; q < N4; ++q) *(f32x4*)(out + 4 * q) = v[q];
            } else if (n < a.f.n && m < a.f.m) {
                finish<FORWARD, E>(a.f, bias, n, m, a.f.m - m, v);
            }
        }
        wait_vm_lgkm0<0>();
    }
}

// The sum of a product's parts, finished: bound by its reads (4 parts of 2048 x 1024: 7.8 us, 5.4 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) linear_sum_kernel(const float* part, int splits, long rows, long pitch, Finish f) {
    const int n = blockIdx.x, m = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (m >= f.m) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int z = 0; z < splits; ++z) v += *(const f32x4*)(part + (z * rows + n) * pitch + m);
    f32x4 one[1] = {v}, bias[1];
    load_bias<T>(f, m, f.m - m, bias);
    finish<true, T>(f, bias, n, m, f.m - m, one);
}

// Rows of an operand that cannot be read in place, copied to rows of whole slabs, 16-byte aligned, zeros at
// their ends.  Four rows a workgroup.
struct PackArgs {
    const void* in;
    long ld;
    int rows, cols;  // rows 0: read in place
    void* out;
    long pitch;
    __host__ __device__ int blocks() const { return (rows + 3) / 4; }
};
template <typename T>
__device__ inline void pack(const PackArgs& a, int block) {
    constexpr int V = 16 / sizeof(T);
    const int row = block * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (row >= a.rows) return;
    const T* src = (const T*)a.in + (size_t)row * a.ld;
    T* dst = (T*)a.out + (size_t)row * a.pitch;
#pragma unroll 4
    for (int c = lane * V; c < a.pitch; c += 64 * V) {
        T v[V] = {};
        if (c + V <= a.cols)
            __builtin_memcpy(v, src + c, 16);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < a.cols) v[i] = src[c + i];
        *(u32x4*)(dst + c) = *(const u32x4*)v;
    }
}

struct SlopeArgs {
    const void *dy, *z;  // z null: no activation
    long ld_dy, ld_z;
    int rows, cols, act;
    int per, groups_x, groups_y;  // rows of a workgroup; workgroups along columns and rows, 0: nothing to do
    void* dz;            // null: dY is read in place by the products, only its sums are wanted
    long pitch;          // whole 16 bytes
    float* sums;         // [workgroup of rows][pitch], null: not wanted
};

// dZ = dY act'(Z), in the operands' type for the products, and its column sums over `per` rows, of
// the values before they are rounded.
//
// In bf16 dZ is rounded to 8 bits for the products, as the upstream gradient of a bf16 layer is: dX and dW are off by 2.35e-3
// of their norm so, with the kept Z's rounding, which moves the slopes, by 2.41e-3 (777 x 5003 x 1001 and 8192 x 8192 x 4096
// alike), where the rounding of the results alone makes 1.66e-3.  As two bf16 parts, which up to 64 tokens take since the read of
// W hides them, dZ would make the products' long axis twice as long: dX and dW of 8192 x 8192 x 4096 908 us, so 1753; of 776 x
// 5008 x 1000 46, so 66.
template <typename T>
__device__ inline void slopes(const SlopeArgs& a, int block) {
    constexpr int V = 16 / sizeof(T), U = 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = (block % a.groups_x * 64 + lane) * V, left = a.cols - c, by = block / a.groups_x;
    const int r0 = by * a.per, r1 = imin(r0 + a.per, a.rows);
    float sum[V] = {};
    if (c < a.pitch)
        by_act(a.z ? a.act : NONE, [&](auto which) {
            constexpr int ACT = decltype(which)::value;
            for (int r = r0 + wave; r < r1; r += 4 * U) {
                f32x4 d[U][V / 4], z[U][V / 4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int n = r + 4 * u < r1 ? left : 0;
                    load((const T*)a.dy + (r + 4 * u) * a.ld_dy + c, n, d[u]);
                    if (ACT != NONE) load((const T*)a.z + (r + 4 * u) * a.ld_z + c, n, z[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    T v[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float x = d[u][i / 4][i % 4];
                        if (ACT != NONE) x = r + 4 * u < r1 && i < left ? x * slope<ACT>(z[u][i / 4][i % 4]) : 0.f;
                        sum[i] += x;
                        v[i] = (T)x;
                    }
                    if (a.dz && r + 4 * u < r1) *(u32x4*)((T*)a.dz + (r + 4 * u) * a.pitch + c) = *(const u32x4*)v;
                }
            }
        });
    if (!a.sums) return;
    __shared__ float all[4][64][V];
#pragma unroll
    for (int i = 0; i < V; ++i) all[wave][lane][i] = sum[i];
    __syncthreads();
    if (wave > 0 || c >= a.pitch) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
        a.sums[(size_t)by * a.pitch + c + i] = all[0][lane][i] + all[1][lane][i] + all[2][lane][i] + all[3][lane][i];
}

// All that reads a call's operands alone, in one launch.  Bound by memory: dY and Z of 8192 x 8192 bf16 to dZ and its sums 87
// us, 4.6 TB/s.
struct PrepareArgs {
    PackArgs w, x;
    SlopeArgs slope;
    __host__ __device__ int slopes() const { return slope.groups_x * slope.groups_y; }
};
template <typename T>
__global__ void __launch_bounds__(256) linear_prepare_kernel(PrepareArgs a) {
    int b = blockIdx.x;
    if (b < a.slopes()) return slopes<T>(a.slope, b);
    b -= a.slopes();
    if (b < a.w.blocks()) return pack<T>(a.w, b);
    pack<T>(a.x, b - a.w.blocks());
}

// dbias alone, where no product is wanted.
template <typename T>
__global__ void __launch_bounds__(256) linear_bias_kernel(BiasArgs a) {
    __shared__ float all[256];
    bias_columns<T>(a, blockIdx.x, all);
}

// A result of no tokens: zeros.
template <typename T>
__global__ void __launch_bounds__(256) linear_zero_kernel(T* out, long ld, int cols) {
    for (int c = blockIdx.y * 256 + threadIdx.x; c < cols; c += gridDim.y * 256) out[(size_t)blockIdx.x * ld + c] = (T)0.f;
}

// ---- at most kFewTokens tokens -----------------------------------------------------------------------

struct FewArgs {
    int tokens, outs, hidden;
    const void *x, *w;
    long ldx, ldw;
    int blocks, splits;  // workgroups along the output features; parts of the hidden size
    float* part;         // splits > 1: [split][16 NB][pitch], summed by linear_sum_kernel
    long pitch;
    Finish f;
};

// Z of 16 MR output features and all tokens, or a part of the hidden size of it where the features alone do not fill
// the chip.  Bound by the read of W (32768 x 1024 bf16 to 64 tokens' fp32 logits: 20.3 us, 3.7 TB/s with the 8 MB written; the
// read alone is 14 us), of 17 to 64 fp32 tokens by latency: a step's loads in flight a wave,
// and cutting both sides into three parts before the next (37 tokens, 5003 x 777: 11.6 us where the bytes take 3.6; half of the waves'
// time waits for loads, a quarter to issue, the VALU is busy for a third of it), of one token by the launch and one trip to memory (4096 x
// 1024: 4.3 us, an empty kernel 1.65).
// The NW waves of a workgroup take every NW-th group of U steps of the hidden size each and add up in LDS.
template <class C, int NB, int MR, int NW>
__global__ void __launch_bounds__(64 * NW) linear_few_kernel(FewArgs a) {
    typedef typename C::T T;
    typedef typename C::Raw Raw;
    typedef typename C::Part Part;
    constexpr int U = C::P == 3 ? (NB == 4 && MR == 2 ? 2 : 1) : MR == 4 ? 2 : 4;  // steps held in registers
    // all loads of a group before its products; not with several rows of features in fp32, where the compiler's order is faster
    constexpr bool HOLD = sizeof(T) == 2 || MR == 1;
    static_assert(NW >= NB, "a wave for each block of tokens");
    __shared__ f32x4 sums[NW][NB][64];
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    const int wave = (int)uniform_u32(threadIdx.x >> 6);
    const int split = blockIdx.x / a.blocks, r0 = (blockIdx.x - split * a.blocks) * 16 * MR;
    const T *w[MR], *x[NB];
#pragma unroll
    for (int m = 0; m < MR; ++m) w[m] = (const T*)a.w + (size_t)imin(r0 + 16 * m + l, a.outs - 1) * a.ldw + g * C::E;
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b] = (const T*)a.x + (size_t)imin(16 * b + l, a.tokens - 1) * a.ldx + g * C::E;
    f32x4 acc[MR][NB] = {};
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
            vocab::few_mma<C>(pw, px, c);
        }
    };
    const int full = a.hidden / C::STEP, groups = full / U;
    const int first = (int)((long)groups * split / a.splits), last = (int)((long)groups * (split + 1) / a.splits);
    for (int q = first + wave; q < last; q += NW) {
        Raw vw[U][MR], vx[U][NB];
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int u = 0; u < U; ++u) vw[u][m] = C::template load<Raw>(w[m] + (size_t)(q * U + u) * C::STEP);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int u = 0; u < U; ++u) vx[u][b] = C::template load<Raw>(x[b] + (size_t)(q * U + u) * C::STEP);
        if (HOLD) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(vw[u], vx[u]);
    }
    const int steps = split + 1 == a.splits ? (a.hidden + C::STEP - 1) / C::STEP : 0;  // the last part's
    for (int s = groups * U + wave; s < steps; s += NW) {
        const int n = a.hidden - s * C::STEP - g * C::E;  // elements of this lane's chunk, maybe none
        Raw vw[MR], vx[NB];
#pragma unroll
        for (int m = 0; m < MR; ++m) vw[m] = C::template load<Raw>(w[m] + (size_t)s * C::STEP, n);
#pragma unroll
        for (int b = 0; b < NB; ++b) vx[b] = C::template load<Raw>(x[b] + (size_t)s * C::STEP, n);
        multiply(vw, vx);
    }
    // An infinity, and what rounds up to one as bf16, has a NaN among its three parts, and makes NaN of all its sums: a wave
    // that finds such sums makes them anew from the values as they are (the others stay, so that a row of X or W reaches
    // its own sums alone).
    if constexpr (C::P == 3) {
        bool nan = false;
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) nan |= acc[m][b][i] != acc[m][b][i];
        if (__any(nan)) {
            int k = g * C::E;  // anew, so that the passes above keep no address for this
            asm volatile("" : "+v"(k));
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const T* const vw = (const T*)a.w + (size_t)imin(r0 + 16 * m + l, a.outs - 1) * a.ldw;
                    const T* const vx = (const T*)a.x + (size_t)imin(16 * b + l, a.tokens - 1) * a.ldx;
                    f32x4 c = {0.f, 0.f, 0.f, 0.f};
                    auto exact = [&](int h, int end) {  // hidden [h, end), whole steps
#pragma unroll 1
                        for (; h < end; h += C::STEP)
#pragma unroll 1
                            for (int q = 0; q < C::E; ++q) {
                                const bool in = h + k + q < a.hidden;
                                c = __builtin_amdgcn_mfma_f32_16x16x4f32(in ? vw[h + k + q] : 0.f, in ? vx[h + k + q] : 0.f, c, 0, 0, 0);
                            }
                    };
#pragma unroll 1
                    for (int q = first + wave; q < last; q += NW) exact(q * U * C::STEP, (q + 1) * U * C::STEP);
#pragma unroll 1
                    for (int s = groups * U + wave; s < steps; s += NW) exact(s * C::STEP, (s + 1) * C::STEP);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (acc[m][b][i] != acc[m][b][i]) acc[m][b][i] = c[i];
                }
        }
    }
    // wave b gets tokens 16 b + l, output features r0 + 16 m + 4 g + i
    f32x4 z[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        if (m > 0) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[wave][b][lane] = acc[m][b];
        __syncthreads();
        if (wave < NB) {
            z[m] = sums[0][wave][lane];
#pragma unroll
            for (int i = 1; i < NW; ++i) z[m] += sums[i][wave][lane];
        }
    }
    const int n = 16 * wave + l;
    if (wave >= NB || n >= a.tokens) return;
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        const int v = r0 + 16 * m + 4 * g;
        if (a.splits > 1) {
            *(f32x4*)(a.part + ((long)split * 16 * NB + n) * a.pitch + v) = z[m];
            continue;
        }
        f32x4 one[1] = {z[m]}, bias[1];
        load_bias<T>(a.f, v, a.outs - v, bias);
        if (v < a.outs) finish<true, T>(a.f, bias, n, v, a.outs - v, one);
    }
}

struct FewSlopeArgs {
    const void *dy, *z, *x;
    long ld_dy, ld_z, ldx;
    int tokens, outs, hidden, act;
    int groups;      // workgroups of 64 output features
    float* d;        // [16 NB][pitch]: dZ, zeros past the tokens and the output features
    long pitch;
    void* dbias;     // null: not wanted
    char* xt;        // X in the order of vocab_few_grad_kernel, `chunks` of them
    int kt, chunks;
};

// dZ and dbias of few tokens, 64 output features a workgroup; the workgroups after those put X in the order
// that dW's product takes.
template <class C, int NB>
__global__ void __launch_bounds__(256) linear_few_slope_kernel(FewSlopeArgs a) {
    typedef typename C::T T;
    if ((int)blockIdx.x >= a.groups) {
        const int i = ((int)blockIdx.x - a.groups) * 256 + (int)threadIdx.x;
        if (i >= a.chunks) return;
        const int lane = i & 63, j = (i >> 6) % a.kt, hb = (i >> 6) / a.kt;
        const int h = C::hidden_of(hb, lane & 15), t = j * C::STEP + (lane >> 4) * C::E;
        typename C::Raw v = {};
#pragma unroll
        for (int q = 0; q < C::E; ++q)
            if (t + q < a.tokens && h < a.hidden) v[q] = ((const T*)a.x)[(t + q) * a.ldx + h];
        ((typename C::Raw*)a.xt)[i] = v;
        return;
    }
    __shared__ f32x4 all[16][16];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c = blockIdx.x * 64 + 4 * tx, left = a.outs - c;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    by_act(a.z ? a.act : NONE, [&](auto which) {
        constexpr int ACT = decltype(which)::value;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int t = 16 * b + ty;
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            if (t < a.tokens && left > 0) {
                d = load4((const T*)a.dy + t * a.ld_dy + c, left);
                if (ACT != NONE) {
                    const f32x4 z = load4((const T*)a.z + t * a.ld_z + c, left);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = i < left ? d[i] * slope<ACT>(z[i]) : 0.f;
                }
            }
            *(f32x4*)(a.d + t * a.pitch + c) = d;
            sum += d;
        }
    });
    if (!a.dbias) return;
    all[ty][tx] = sum;
    __syncthreads();
    if (ty > 0 || left <= 0) return;
    for (int i = 1; i < 16; ++i) sum += all[i][tx];
    const f32x4 one[1] = {sum};
    leave<T>(a.dbias, 0, 0, c, left, one);
}

}  // namespace linear
}  // namespace libsgemm
