// kernel_vocab.hpp -- the matrix products of the vocabulary-head operators (gfx950, bf16 MFMA).
//
// One tile loop serves every product: C(m, n) = sum_k A[m][k] * B[n][k], both operands stored with
// k contiguous, multiplied with v_mfma_f32_32x32x16_bf16 and accumulated in fp32.  What differs is
// what the finished tile is used for:
//
//   vocab_lse_kernel    z = alpha * W X^T, reduced over the tile's vocabulary rows to the maximum
//                       and the sum of exponentials per token: the logits are never stored;
//   vocab_grad_kernel   z again, turned into d(loss)/dz of one piece of the vocabulary;
//   vocab_dx_kernel     dX += D W over that piece, in fp32;
//   vocab_dw_kernel     dW = D^T X of that piece.
//
// Vocabulary rows are the M side of the first two, so that a lane holds one token and 16
// vocabulary entries per 32x32 block: the reduction over the vocabulary is in registers, one
// exchange between the lane halves at its end.
//
// P is the number of bf16 planes an operand is held in.  P = 1: bf16 operands, as they are.
// P = 3: fp32 operands as the exact sum of three bf16 values (8 + 8 + 8 significand bits), a row
// stored in blocks of 32 k as [32 high][32 middle][32 low].  The six products of weight above
// 2^-24 are accumulated (hh, hm, mh, mm, hl, lh; the dropped ml, lm, ll are below one rounding of
// the fp32 product): six bf16 MFMAs do the work of an fp32 product at 16/6 of the fp32 MFMA rate.
#pragma once

#include "kernel_common.hpp"
#include "kernel_dl.hpp"

namespace libsgemm {
namespace vocab {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <int P>
struct Planes {
    static_assert(P == 1 || P == 3, "bf16 or three-plane fp32 operands");
    static constexpr int BK = P == 1 ? 64 : 32;     // k per slab
    static constexpr int QR = P == 1 ? 8 : 12;      // 16-byte quads per row and slab
    static constexpr int ROW = QR * 16;             // bytes per row and slab
    // LDS quad u of row r holds the row's quad swz(r, u), an involution.  A 128-bit read is served
    // in passes of 16 lanes of one half-wave (lanes 0-3, 12-15, 20-23, 24-27 or the others) over 64
    // banks; with 128-byte rows a pass must find 8 different quads among its even and its odd rows,
    // with 192-byte rows 4 different ones among its rows of each residue modulo 4.
    __host__ __device__ static constexpr int swz(int r, int u) {
        return P == 1 ? (u ^ ((r >> 1) & 7)) : ((u & ~3) | ((u ^ (r >> 2)) & 3));
    }
    // Byte offset of plane p of element k within a row.
    __host__ __device__ static constexpr long at(long k, int p) {
        return P == 1 ? 2 * k : (k >> 5) * 192 + p * 64 + (k & 31) * 2;
    }
    // Bytes of a row of kp elements (kp a multiple of BK).
    __host__ __device__ static constexpr long pitch(long kp) { return 2L * P * kp; }
};

// x as P bf16 values.  P = 3 is exact (each remainder fits the next value) but where the low parts
// fall below bf16's subnormals; a value that would round to infinity is cut off instead.
template <int P>
__device__ inline void split(float x, __bf16 (&v)[P]) {
    __bf16 h = (__bf16)x;
    if (P == 3) {
        float hf = (float)h;
        if (__builtin_isinf(hf) && !__builtin_isinf(x)) {
            hf = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
            h = (__bf16)hf;
        }
        const float r = __builtin_isfinite(x) ? x - hf : 0.f;
        const __bf16 m = (__bf16)r;
        v[P > 1 ? 1 : 0] = m;
        v[P > 2 ? 2 : 0] = (__bf16)(r - (float)m);
    }
    v[0] = h;
}
template <int P>
__device__ inline void store1(char* row, long k, float x) {
    __bf16 v[P];
    split<P>(x, v);
#pragma unroll
    for (int p = 0; p < P; ++p) *(__bf16*)(row + Planes<P>::at(k, p)) = v[p];
}
// Four consecutive k, the first a multiple of 4.
template <int P>
__device__ inline void store4(char* row, long k, const float (&x)[4]) {
    bf16x4 o[P];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __bf16 v[P];
        split<P>(x[j], v);
#pragma unroll
        for (int p = 0; p < P; ++p) o[p][j] = v[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) *(bf16x4*)(row + Planes<P>::at(k, p)) = o[p];
}

// A product operand: rows of `pitch` bytes, rows past `rows` read as its last row.
struct Operand {
    const char* base;
    uint32_t pitch;
    int rows;
};

// The tile loop.  The operands' slabs go straight from global memory into a ring of ST LDS stages;
// slab s + ST - 1 is requested after the barrier that opens slab s, so each load has ST - 1 slabs
// of matrix work to arrive in.
template <int P, int BM, int BN, int WM, int WN, int ST>
struct Tile {
    static constexpr int kP = P, kBM = BM, kBN = BN, kWM = WM, kWN = WN;
    static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, NW = WAVES_M * WAVES_N, NT = NW * 64;
    static constexpr int MB = WM / 32, NB = WN / 32;
    static constexpr int QR = Planes<P>::QR, ROW = Planes<P>::ROW, BK = Planes<P>::BK;
    static constexpr int LA = BM * QR / NT, LB = BN * QR / NT;
    static constexpr int STAGE = (BM + BN) * ROW;
    static constexpr int LDS_BYTES = STAGE * ST;
    static_assert(BM * QR % NT == 0 && BN * QR % NT == 0, "whole loads per thread");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static_assert((LA + LB) * (ST - 1) < 64, "vmcnt counts at most 63 loads in flight");

    f32x16 acc[MB][NB];

    template <int ROWS, int L>
    static __device__ inline void offsets(const Operand& o, int row0, int wave, int lane, uint32_t (&off)[L]) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int i = (j * NW + wave) * 64 + lane;
            const int r = i / QR, u = i - r * QR;
            const int row = imin(row0 + r, o.rows - 1) - row0;  // the tile's first row is always valid
            off[j] = (uint32_t)row * o.pitch + (uint32_t)(Planes<P>::swz(r, u) * 16);
        }
    }

    // Multiplies slabs [k0, k0 + slabs) of A rows m0.. and B rows n0..; lds: LDS_BYTES.
    __device__ inline void run(char* lds, const Operand& a, int m0, const Operand& b, int n0, int k0, int slabs) {
        const int lane = threadIdx.x & 63;
        const int wave = (int)uniform_u32(threadIdx.x >> 6);
        const int wm = wave / WAVES_N, wn = wave % WAVES_N;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
        uint32_t oa[LA], ob[LB];
        offsets<BM, LA>(a, m0, wave, lane, oa);
        offsets<BN, LB>(b, n0, wave, lane, ob);
        const char* pa = a.base + (size_t)m0 * a.pitch + (size_t)k0 * ROW;
        const char* pb = b.base + (size_t)n0 * b.pitch + (size_t)k0 * ROW;
        const uint32_t base = lds_addr((const float*)lds) + wave * 1024;
        auto issue = [&](int stage) {
            const uint32_t at = base + stage * STAGE;
#pragma unroll
            for (int j = 0; j < LA; ++j) dl_load<16>(pa, oa[j], at + j * NW * 1024);
#pragma unroll
            for (int j = 0; j < LB; ++j) dl_load<16>(pb, ob[j], at + BM * ROW + j * NW * 1024);
            pa += ROW;
            pb += ROW;
        };
        // fragment addresses: row l of a block, quad (of plane p) 2 * kk + half, swizzled
        const int l = lane & 31, h = lane >> 5;
        constexpr int KK = BK / 16;
        int fq[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) fq[kk] = l * ROW + Planes<P>::swz(l, 2 * kk + h) * 16;
        const char* fa = lds + wm * WM * ROW;
        const char* fb = lds + BM * ROW + wn * WN * ROW;
#pragma unroll
        for (int s = 0; s < ST - 1; ++s)
            if (s < slabs) issue(s);
        int stage = 0;
        for (int s = 0; s < slabs; ++s) {
            wait_slabs<LA + LB>(imin(ST - 2, slabs - 1 - s));
            dl_barrier();
            if (s + ST - 1 < slabs) issue(stage == 0 ? ST - 1 : stage - 1);
            const char* sa = fa + stage * STAGE;
            const char* sb = fb + stage * STAGE;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                bf16x8 va[P][MB], vb[P][NB];
#pragma unroll
                for (int p = 0; p < P; ++p) {
#pragma unroll
                    for (int i = 0; i < MB; ++i) va[p][i] = *(const bf16x8*)(sa + i * 32 * ROW + p * 64 + fq[kk]);
#pragma unroll
                    for (int j = 0; j < NB; ++j) vb[p][j] = *(const bf16x8*)(sb + j * 32 * ROW + p * 64 + fq[kk]);
                }
#pragma unroll
                for (int w = P - 1; w >= 0; --w)  // planes of total weight w, the smallest terms first
#pragma unroll
                    for (int p = 0; p <= w; ++p)
#pragma unroll
                        for (int i = 0; i < MB; ++i)
#pragma unroll
                            for (int j = 0; j < NB; ++j)
                                acc[i][j] =
                                    __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[p][i], vb[w - p][j], acc[i][j], 0, 0, 0);
            }
            stage = stage + 1 == ST ? 0 : stage + 1;
        }
    }

    // Element e of block (i, j) of this lane is C(m0 + row(i, e), n0 + col(j)).
    static __device__ inline int col(int j) {
        const int wave = threadIdx.x >> 6;
        return (wave % WAVES_N) * WN + j * 32 + (threadIdx.x & 31);
    }
    static __device__ inline int row(int i, int e) {
        const int wave = threadIdx.x >> 6;
        return (wave / WAVES_N) * WM + i * 32 + 8 * (e >> 2) + 4 * ((threadIdx.x & 63) >> 5) + (e & 3);
    }
};

struct LseArgs {
    Operand w, x;     // vocabulary rows of this piece, counted tokens
    const int* count; // number of counted tokens
    int tiles_m, tiles_n, slabs, vocab;
    float alpha;
    float2* part;     // [vocabulary pieces of WM rows][tp]: maximum and sum of exp(z - maximum)
    int part0, tp;
};

template <class T>
__global__ void __launch_bounds__(T::NT) vocab_lse_kernel(LseArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    if (n0 >= *a.count) return;
    T t;
    t.run(lds, a.w, m0, a.x, n0, 0, a.slabs);
    const int h = (threadIdx.x & 63) >> 5;
    const int piece = a.part0 + tm * T::WAVES_M + (threadIdx.x >> 6) / T::WAVES_N;
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float z = m0 + t.row(i, e) < a.vocab ? t.acc[i][j][e] * a.alpha : -INFINITY;
                t.acc[i][j][e] = z;
                top = z > top || z != z ? z : top;  // a NaN stays
            }
        const float other = __shfl_xor(top, 32);
        top = other > top || other != other ? other : top;
        float sum = 0.f;
        const float ref = top == -INFINITY ? 0.f : top;  // nothing but -inf here: the sum is 0
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum += __expf(t.acc[i][j][e] - ref);
        sum += __shfl_xor(sum, 32);
        if (h == 0) a.part[(size_t)piece * a.tp + n0 + t.col(j)] = make_float2(top, sum);
    }
}

struct GradArgs {
    Operand w, x;
    const int* count;
    int tiles_m, tiles_n, slabs, vocab;
    float alpha;
    const float* lse;    // per counted token
    const float* scale;  // per counted token: D = exp(z - lse) * scale
    char* d;             // [token][vocabulary piece], planes
    long d_pitch;
    char* dt;            // [vocabulary piece][token], planes; null: not wanted
    long dt_pitch;
};

template <class T>
__global__ void __launch_bounds__(T::NT) vocab_grad_kernel(GradArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    const int count = *a.count;
    if (n0 >= count) return;
    T t;
    t.run(lds, a.w, m0, a.x, n0, 0, a.slabs);
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        const bool live = n < count;
        const float lse = live ? a.lse[n] : 0.f, scale = live ? a.scale[n] : 0.f;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int m = m0 + t.row(i, 4 * g);
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // entries past the vocabulary and tokens past the count are the zeros that the
                    // products of D run over
                    v[q] = live && m + q < a.vocab ? __expf(t.acc[i][j][4 * g + q] * a.alpha - lse) * scale : 0.f;
                    if (a.dt) store1<T::kP>(a.dt + (size_t)(m + q) * a.dt_pitch, n, v[q]);
                }
                if (a.d) store4<T::kP>(a.d + (size_t)n * a.d_pitch, m, v);
            }
    }
}

struct DxArgs {
    Operand wt, d;     // [hidden][vocabulary piece], [token][vocabulary piece]
    const int* count;
    int tiles_m, tiles_n, slabs, splits;
    float* acc;        // [splits][tp][hp]
    long tp;
    int hp;
    int add;           // not the first piece
};

template <class T>
__global__ void __launch_bounds__(T::NT) vocab_dx_kernel(DxArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    const int count = *a.count;
    if (n0 >= count) return;
    const int z = blockIdx.y;
    const int first = (int)((long)a.slabs * z / a.splits), last = (int)((long)a.slabs * (z + 1) / a.splits);
    T t;
    t.run(lds, a.wt, m0, a.d, n0, first, last - first);
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        if (n >= count) continue;
        float* out = a.acc + ((size_t)z * a.tp + n) * a.hp + m0;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4* p = (f32x4*)(out + t.row(i, 4 * g));
                f32x4 v = {t.acc[i][j][4 * g], t.acc[i][j][4 * g + 1], t.acc[i][j][4 * g + 2], t.acc[i][j][4 * g + 3]};
                if (a.add) v += *p;
                *p = v;
            }
    }
}

struct DwArgs {
    Operand xt, dt;    // [hidden][token], [vocabulary piece][token]
    const int* count;
    int tiles_m, tiles_n, hidden, vocab;
    void* out;         // [vocabulary piece][hidden] in the operands' type
    long ld;
    int vec;           // rows hold whole aligned groups of four
};

template <class T>
__global__ void __launch_bounds__(T::NT) vocab_dw_kernel(DwArgs a) {
    using O = typename std::conditional<T::kP == 1, __bf16, float>::type;
    typedef O O4 __attribute__((ext_vector_type(4)));
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    T t;
    t.run(lds, a.xt, m0, a.dt, n0, 0, (*a.count + T::BK - 1) / T::BK);
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        if (n >= a.vocab) continue;
        O* out = (O*)a.out + (size_t)n * a.ld;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int m = m0 + t.row(i, 4 * g);
                if (a.vec) {
                    O4 v;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = (O)t.acc[i][j][4 * g + q];
                    if (m < a.hidden) *(O4*)(out + m) = v;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (m + q < a.hidden) out[m + q] = (O)t.acc[i][j][4 * g + q];
                }
            }
    }
}

}  // namespace vocab
}  // namespace libsgemm
