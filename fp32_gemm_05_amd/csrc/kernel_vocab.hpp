// kernel_vocab.hpp -- the matrix products of the vocabulary-head operators (gfx950, 16-bit MFMA).
//
// One tile loop serves every product: C(m, n) = sum_k A(m, k) * B(n, k), each operand stored with k
// along its rows or down its columns (then read from LDS with transposing loads), multiplied with
// v_mfma_f32_32x32x16 (bf16 or fp16) and accumulated in fp32.  No matrix is transposed in memory.  What
// differs is what the finished tile is used for:
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
// P is the number of 16-bit planes an operand is held in.  P = 1: bf16 operands, as they are.
// P = 2: fp32 operands as the sum of two fp16 values, a row stored in blocks of 32 k as [32 high]
// [32 low].  The operand -- a row of X, a row of W in the forward call, the whole of W in the gradient's,
// whose dX sums over its rows -- is scaled by a power of two first, so that its largest value lies in
// [2^14, 2^15); high + low then holds every value down to 2^-16 of the largest to 2^-23 of itself (23 bits:
// a quarter of all fp32 values are off by their last one) and smaller ones to 2^-40 of the largest.  Three
// products (hl, lh, hh) are accumulated in fp32; the one left out, ll, is up to 2^-22 of the whole, 2^-25 in
// the mean and of either sign.  Three fp16 MFMAs do the work of an fp32 product at 16/3 of the fp32 MFMA
// rate, from operands of the same size.
#pragma once

#include "kernel_common.hpp"
#include "kernel_dl.hpp"

namespace libsgemm {
namespace vocab {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int P>
struct Planes {
    static_assert(P == 1 || P == 2, "bf16, or fp32 as two fp16 planes");
    typedef typename std::conditional<P == 1, __bf16, _Float16>::type Half;
    typedef Half Half8 __attribute__((ext_vector_type(8)));
    typedef Half Half4 __attribute__((ext_vector_type(4)));
    static constexpr int BK = 64 / P;    // k per slab
    static constexpr int QR = 8;         // 16-byte quads per row and slab
    static constexpr int ROW = QR * 16;  // bytes per row and slab
    // LDS quad u of row r holds the row's quad swz(r, u), an involution.  A 128-bit read is served
    // in passes of 16 lanes of one half-wave (lanes 0-3, 12-15, 20-23, 24-27 or the others) over 64
    // banks, two rows: a pass must find 8 different quads among its even and among its odd rows.
    __host__ __device__ static constexpr int swz(int r, int u) { return u ^ ((r >> 1) & 7); }
    // Byte offset of plane p of element k within a row.
    __host__ __device__ static constexpr long at(long k, int p) {
        return P == 1 ? 2 * k : (k >> 5) * 128 + p * 64 + (k & 31) * 2;
    }
    // Bytes of a row of kp elements (kp a multiple of BK).
    __host__ __device__ static constexpr long pitch(long kp) { return 2L * P * kp; }
};

// x as P values; infinities and NaN have no low part.
template <int P>
__device__ inline void split(float x, typename Planes<P>::Half (&v)[P]) {
    typedef typename Planes<P>::Half Half;
    v[0] = (Half)x;
    if constexpr (P == 2) v[1] = __builtin_isfinite(x) ? (Half)(x - (float)v[0]) : (Half)0.f;
}
template <int P>
__device__ inline void store1(char* row, long k, float x) {
    typename Planes<P>::Half v[P];
    split<P>(x, v);
#pragma unroll
    for (int p = 0; p < P; ++p) *(typename Planes<P>::Half*)(row + Planes<P>::at(k, p)) = v[p];
}
// Four consecutive k, the first a multiple of 4.
template <int P>
__device__ inline void store4(char* row, long k, const float (&x)[4]) {
    typename Planes<P>::Half4 o[P];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        typename Planes<P>::Half v[P];
        split<P>(x[j], v);
#pragma unroll
        for (int p = 0; p < P; ++p) o[p][j] = v[p];
    }
#pragma unroll
    for (int p = 0; p < P; ++p) *(typename Planes<P>::Half4*)(row + Planes<P>::at(k, p)) = o[p];
}
template <int P>
__device__ inline f32x16 mfma(typename Planes<P>::Half8 a, typename Planes<P>::Half8 b, f32x16 c) {
    if constexpr (P == 1)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

__device__ inline float wave_sum(float s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    return s;
}
__device__ inline float wave_max(float s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s = fmaxf(s, __shfl_xor(s, o));
    return s;
}

// The scale of P = 2 operands: the power of two that brings a largest value m into [2^14, 2^15).
// m of 0 (or nothing finite) gives 1; an m so small or large that the power would leave fp32's
// range gives the nearest that does not.
__device__ inline int scale_exponent(float m) {
    if (!(m > 0.f)) return 0;
    const int e = 14 - ilogbf(m);
    return e > 126 ? 126 : e < -126 ? -126 : e;
}
// Of D, whose entries are at most 1 in magnitude, but for the error of z - lse.  That is of any size where
// logits are: past kDMost, which fp16 still holds, an entry is cut off there, by no more than that error.
constexpr float kDScale = 0x1p15f, kDMost = 0x1.fp0f;

// A product operand, stored with k along its rows (K_ROW: A[m][k], the rows whole slabs; K_ENDS: rows
// that may end inside one) or down its columns (K_COL: A[k][m]); rows past `rows` read as its last row,
// quads past row_bytes as the row's last quad.  Neither kind of stand-in reaches a result: past-the-end
// m or n are never stored, past-the-end k meet zeros of the other operand.
struct Operand {
    const char* base;
    uint32_t pitch, row_bytes;
    int rows;
};
enum Order { K_ROW, K_ENDS, K_COL };

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// One operand's side of the tile: R rows (m or n) of a slab of BK k, NT threads.
template <int P, Order O, int R, int W, int NT>
struct Side {
    static constexpr int BK = Planes<P>::BK, NW = NT / 64;
    static constexpr int BYTES = R * BK * 2 * P;                            // of a slab in LDS
    static constexpr int QUADS = O != K_COL ? Planes<P>::QR : R * P / 8;    // per stored row
    static constexpr int ROW = QUADS * 16;
    static constexpr int L = BYTES / 16 / NT;                               // loads per thread
    static constexpr int B = W / 32;                                        // 32-row blocks of a wave
    static constexpr int KK = BK / 16;
    static_assert(BYTES / 16 % NT == 0, "whole loads per thread");

    // K_COL: chunk c (64 bytes: 32 m of one plane) of LDS row r holds chunk c ^ flip(r).  A transposed
    // 64-bit read is served in passes of 32 lanes, which read one chunk each of four consecutive
    // rows: the flips put those on the four different quarters of the 64 banks.
    static constexpr int CHUNKS = R * P / 32;
    static_assert(O != K_COL || CHUNKS % 2 == 0, "chunks pair up");
    __host__ __device__ static constexpr int flip(int r) { return CHUNKS % 4 == 0 ? (r & 3) : ((r >> 1) & 1); }
    __host__ __device__ static constexpr int source_quad(int r, int u) {
        return O != K_COL ? Planes<P>::swz(r, u) : (u ^ (flip(r) << 2));
    }

    const char* at;       // next slab
    size_t step;          // bytes from slab to slab
    uint32_t off[L];
    uint32_t end[O == K_ENDS ? L : 1];  // its row's last quad
    int left;             // K_COL: rows from `at` to the operand's end
    uint32_t lane_at[O != K_COL ? KK * P : B * P];  // LDS offsets of this lane's fragments
    int frag;             // wave's part of them

    __device__ inline void init(const Operand& o, int row0, int k0, int wave, int lane, int wave_at) {
        if (O != K_COL) {
            at = o.base + (size_t)first_row(o, row0) * o.pitch + (O == K_ENDS ? 0 : (size_t)k0 * ROW);
            step = O == K_ENDS ? 0 : ROW;
            left = 0;
        } else {
            at = o.base + (size_t)k0 * BK * o.pitch + (size_t)row0 * 2 * P;
            step = (size_t)BK * o.pitch;
            left = o.rows - k0 * BK;
        }
        set_offsets(o, row0, wave, lane);
        if (O == K_ENDS) advance(k0 * ROW);
        const int l = lane & 31, h = lane >> 5;
        if (O != K_COL) {
            // row l of a block, quad 2 * kk + h of plane p
            frag = wave_at * W * ROW;
#pragma unroll
            for (int q = 0; q < KK * P; ++q) lane_at[q] = l * ROW + Planes<P>::swz(l, 2 * q + h) * 16;
        } else {
            // lane i of a group of 16 points at k = i / 4, m = 4 * (i % 4) and gets k = 0 .. 3 of m = i
            const int i = lane & 15, r = 8 * h + (i >> 2), f = flip(i >> 2);
            frag = 0;
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int c = ((wave_at * B + b) * P + p) ^ f;
                    lane_at[b * P + p] = r * ROW + c * 64 + ((lane >> 4) & 1) * 32 + (i & 3) * 8;
                }
        }
    }
    // A tile may lie past the operand's rows as a whole (the zero padding of D): it reads the last row.
    static __device__ inline int first_row(const Operand& o, int row0) { return imin(row0, o.rows - 1); }
    __device__ inline void set_offsets(const Operand& o, int row0, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int i = (j * NW + wave) * 64 + lane;
            const int r = i / QUADS, u = i - r * QUADS;
            if (O != K_COL) {
                const int row = imin(row0 + r, o.rows - 1) - first_row(o, row0);
                const uint32_t quad = source_quad(r, u) * 16, last = o.row_bytes - 16;
                off[j] = (uint32_t)row * o.pitch + (O == K_ENDS && quad > last ? last : quad);
                if (O == K_ENDS) end[j] = (uint32_t)row * o.pitch + last;
            } else {
                const uint32_t q = (uint32_t)row0 * 2 * P + (uint32_t)(source_quad(r, u) * 16);
                const uint32_t last = o.row_bytes - 16;
                off[j] = (uint32_t)imin(r, left - 1) * o.pitch + (q < last ? q : last) - (uint32_t)row0 * 2 * P;
            }
        }
    }
    // K_ENDS: the loads' places `bytes` further on, their row's last quad at most.
    __device__ inline void advance(uint32_t bytes) {
#pragma unroll
        for (int j = 0; j < L; ++j) off[j] = off[j] + bytes < end[j] ? off[j] + bytes : end[j];
    }
    // Requests loads [from, to) of the next slab into LDS at `lds`.
    __device__ inline void issue(uint32_t lds, int from, int to) const {
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (j >= from && j < to) dl_load<16>(at, off[j], lds + j * NW * 1024);
    }
    __device__ inline void next(const Operand& o, int row0, int wave, int lane) {
        if (O == K_ENDS) return advance(ROW);
        at += step;
        if (O == K_COL) {
            left -= BK;
            if (left < BK && left > 0) set_offsets(o, row0, wave, lane);
        }
    }
    // The fragments of k-step kk: of a lane, 8 consecutive k of its row in each block and plane.
    __device__ inline void read(const char* slab, int kk, typename Planes<P>::Half8 (&v)[P][B]) const {
        typedef typename Planes<P>::Half8 Half8;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (O != K_COL) {
                    v[p][b] = *(const Half8*)(slab + frag + b * 32 * ROW + lane_at[p * KK + kk]);
                } else {
                    const char* a = slab + lane_at[b * P + p] + kk * 16 * ROW;
                    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
                    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * ROW));
                    v[p][b] = __builtin_bit_cast(Half8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
            }
    }
};

// The tile loop.  The operands' slabs go straight from global memory into rings of SA and SB LDS
// stages.  A slab's first fragments are read, and the stages of the slab before it are requested
// anew, behind the barrier that comes before the last k-step of that slab: the matrix unit has that
// k-step to do while the reads are on their way.  The requests stand one by one between MFMAs: a
// wave issues in order, and one that queues them all at once is held until the memory pipe has taken
// them, its MFMAs behind them.  With SA = SB + 1 A's requests have a slab longer to arrive, and are
// spread over the first k-steps of the next slab.
template <int P, int BM, int BN, int WM, int WN, int SA, int SB>
struct Tile {
    static constexpr int kP = P, kBM = BM, kBN = BN, kWM = WM, kWN = WN;
    static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, NW = WAVES_M * WAVES_N, NT = NW * 64;
    static constexpr int MB = WM / 32, NB = WN / 32;
    static constexpr int BK = Planes<P>::BK, KK = BK / 16;
    static constexpr int BYTES_A = BM * BK * 2 * P, BYTES_B = BN * BK * 2 * P;
    static constexpr int LDS_BYTES = BYTES_A * SA + BYTES_B * SB;
    static constexpr int MFMAS = MB * NB * (P == 2 ? 3 : 1);  // per k-step
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
    static_assert(SB >= 2 && (SA == SB || SA == SB + 1), "stages");

    f32x16 acc[MB][NB];

    // Multiplies slabs [k0, k0 + slabs) of A rows m0.. and B rows n0..; lds: LDS_BYTES.
    template <Order OA, Order OB>
    __device__ inline void run(char* lds, const Operand& a, int m0, const Operand& b, int n0, int k0, int slabs) {
        using A = Side<P, OA, BM, WM, NT>;
        using B = Side<P, OB, BN, WN, NT>;
        constexpr int LA = A::L, LB = B::L;
        static_assert((LA + LB) * SB < 64, "vmcnt counts at most 63 loads in flight");
        const int lane = threadIdx.x & 63;
        const int wave = (int)uniform_u32(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
        if (slabs <= 0) return;
        A sa;
        B sb;
        sa.init(a, m0, k0, wave, lane, wave / WAVES_N);
        sb.init(b, n0, k0, wave, lane, wave % WAVES_N);
        char* const lds_b = lds + SA * BYTES_A;
        const uint32_t base_a = lds_addr((const float*)lds) + wave * 1024, base_b = base_a + SA * BYTES_A;
        typename Planes<P>::Half8 va[2][P][MB], vb[2][P][NB];
        // the MFMAs of k-step kk, `loads` calls of issue(0 ..) spread between them if there is `more`
        auto multiply = [&](int kk, bool more, int loads, auto issue) {
            int x = 0, q = 0;
#pragma unroll
            for (int w = P - 1; w >= 0; --w)  // planes of total weight w, the smallest terms first
#pragma unroll
                for (int p = 0; p <= w; ++p)
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            acc[i][j] = mfma<P>(va[kk & 1][p][i], vb[kk & 1][w - p][j], acc[i][j]);
                            ++x;
                            if (loads > 0) {
                                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                                for (; q < loads && q * MFMAS < x * loads; ++q)
                                    if (more) issue(q);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
        };
        constexpr int SMAX = SA > SB ? SA : SB;
#pragma unroll
        for (int s = 0; s < SMAX; ++s) {
            if (s >= slabs) continue;
            if (s < SA) {
                sa.issue(base_a + s * BYTES_A, 0, LA);
                sa.next(a, m0, wave, lane);
            }
            if (s < SB) {
                sb.issue(base_b + s * BYTES_B, 0, LB);
                sb.next(b, n0, wave, lane);
            }
        }
        if (slabs >= SMAX)
            wait_vm_lgkm0<LA*(SA - 1) + LB*(SB - 1)>();
        else
            wait_vm_lgkm0<0>();
        dl_barrier();
        sa.read(lds, 0, va[0]);
        sb.read(lds_b, 0, vb[0]);
        int ta = 0, tb = 0;  // stages of slab s
        for (int s = 0; s < slabs; ++s) {
            const int ta1 = ta + 1 == SA ? 0 : ta + 1, tb1 = tb + 1 == SB ? 0 : tb + 1;
            // SA > SB: the stage of slab s - 1 takes slab s - 1 + SA
            const bool early = SA > SB && s > 0 && s - 1 + SA < slabs;
            const uint32_t at_early = base_a + (ta == 0 ? SA - 1 : ta - 1) * BYTES_A;
#pragma unroll
            for (int kk = 0; kk < KK - 1; ++kk) {
                sa.read(lds + ta * BYTES_A, kk + 1, va[(kk + 1) & 1]);
                sb.read(lds_b + tb * BYTES_B, kk + 1, vb[(kk + 1) & 1]);
                const int from = LA * kk / (KK - 1), to = LA * (kk + 1) / (KK - 1);
                multiply(kk, early, SA > SB ? to - from : 0,
                         [&](int q) { sa.issue(at_early, from + q, from + q + 1); });
            }
            if (early) sa.next(a, m0, wave, lane);
            if (s + 1 < slabs) {
                // this wave's reads of slab s are done, its parts of slab s + 1 have landed
                if (s + SMAX <= slabs)
                    wait_vm_lgkm0<LA*(SA - 2) + LB*(SB - 2)>();
                else
                    wait_vm_lgkm0<0>();
                dl_barrier();
                sa.read(lds + ta1 * BYTES_A, 0, va[0]);
                sb.read(lds_b + tb1 * BYTES_B, 0, vb[0]);
            }
            const uint32_t at_a = base_a + ta * BYTES_A, at_b = base_b + tb * BYTES_B;
            multiply(KK - 1, s + SB < slabs, (SA == SB ? LA : 0) + LB, [&](int q) {
                if (q < LB)
                    sb.issue(at_b, q, q + 1);
                else
                    sa.issue(at_a, q - LB, q - LB + 1);
            });
            if (s + SB < slabs) {
                sb.next(b, n0, wave, lane);
                if (SA == SB) sa.next(a, m0, wave, lane);
            }
            ta = ta1;
            tb = tb1;
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
    Operand w, x;          // vocabulary rows of this piece, counted tokens
    const int* count;      // number of counted tokens
    const float *w_unit, *x_unit;  // P = 2: what a packed unit of each row of W, of X stands for
    int tiles_m, tiles_n, slabs, vocab;
    float alpha;
    float2* part;          // [vocabulary pieces of WM rows][tp]: maximum and sum of exp(z - maximum)
    int part0, tp;
};

constexpr float kLog2E = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// The tile's maxima and sums.  Its exponentials cost as much as 10 slabs of products if each value is
// masked, compared and rescaled; PLAIN, for a tile of valid rows and alpha >= 0, takes the maximum of the
// accumulators as they are and one fma, one v_exp_f32 and one add for each.  A NaN may be missed by the
// maximum, but not by the sum.
template <bool PLAIN, class T>
__device__ inline void lse_tile(T& t, const LseArgs& a, int m0, int n0, int count, int piece) {
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        float c = a.alpha * kLog2E;
        if (T::kP == 2) c *= n < count ? a.x_unit[n] : 0.f;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int m = m0 + t.row(i, 4 * g);
                f32x4 unit = {1.f, 1.f, 1.f, 1.f};
                if (T::kP == 2) unit = *(const f32x4*)(a.w_unit + m);  // to the end of the tile, as the rows
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float z = t.acc[i][j][4 * g + q];
                    if (T::kP == 2) z *= unit[q];
                    if (!PLAIN) z = m + q < a.vocab ? z * c : -INFINITY;
                    top = fmaxf(top, z);
                    t.acc[i][j][4 * g + q] = z;
                }
            }
        top = fmaxf(top, __shfl_xor(top, 32));
        // z * log2(e) of the largest; nothing but -inf here: the sum is 0
        const float ref = top == -INFINITY ? 0.f : PLAIN ? top * c : top;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                sum += __builtin_amdgcn_exp2f(PLAIN ? __builtin_fmaf(t.acc[i][j][e], c, -ref) : t.acc[i][j][e] - ref);
        sum += __shfl_xor(sum, 32);
        if ((threadIdx.x & 63) < 32)
            a.part[(size_t)piece * a.tp + n] = make_float2(top == -INFINITY ? top : ref * kLn2, sum);
    }
}

template <class T, Order W>
__global__ void __launch_bounds__(T::NT) vocab_lse_kernel(LseArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    const int count = *a.count;
    if (n0 >= count) return;
    T t;
    t.template run<W, K_ROW>(lds, a.w, m0, a.x, n0, 0, a.slabs);
    const int piece = a.part0 + tm * T::WAVES_M + (threadIdx.x >> 6) / T::WAVES_N;
    if (m0 + T::kBM <= a.vocab && a.alpha >= 0.f)
        lse_tile<true>(t, a, m0, n0, count, piece);
    else
        lse_tile<false>(t, a, m0, n0, count, piece);
}

struct GradArgs {
    Operand w, x;
    const int *count, *rows;       // the counted tokens
    const float *w_unit, *x_unit;  // P = 2: what a packed unit of W, of each row of X stands for
    int tiles_m, tiles_n, slabs, vocab;
    float alpha;
    const float *lse, *scale;      // per token: D = exp(z - lse) * scale
    const long long* target;       // cross entropy: the entries that take `value`, per token
    const float* value;
    long long v0;                  // first vocabulary row of this piece
    char* d;                       // [counted token][vocabulary piece], planes
    long d_pitch;
};

// D of a token's column in this wave, stored.  PLAIN: no row past the vocabulary and no target among
// these, as nearly everywhere: a fma, an exponential, a product and the rounding of each are left.
// most (P = 2): of the exponent, that of kDMost (the minimum keeps a NaN).
template <bool PLAIN, class T>
__device__ inline void grad_column(const T& t, const GradArgs& a, int j, int n, int m0, float lse, float scale,
                                   float alpha, float most, int entry, float value) {
    typedef typename Planes<T::kP>::Half Half;
    typedef typename Planes<T::kP>::Half4 Half4;
    const int h = (threadIdx.x & 63) >> 5;
    char* out = a.d + (size_t)n * a.d_pitch;
    const float c = alpha * kLog2E, l = lse * kLog2E;
#pragma unroll
    for (int i = 0; i < T::MB; ++i)
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            Half4 v[2][T::kP];
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int e = 4 * (g + f) + q, m = m0 + t.row(i, e);
                    // with one rounding less where D keeps 22 bits
                    float x = T::kP == 2 ? __builtin_fmaf(t.acc[i][j][e], alpha, -lse) * kLog2E
                                         : __builtin_fmaf(t.acc[i][j][e], c, -l);
                    if (T::kP == 2) x = __builtin_elementwise_minimum(x, most);
                    x = __builtin_amdgcn_exp2f(x) * scale;
                    if (!PLAIN) {
                        // rows past the vocabulary are the zeros that dX's product runs over
                        x = m < a.vocab ? x : 0.f;
                        x = m == entry ? value : x;
                    }
                    // one x for the high part that is stored and for the one that the low part is measured
                    // from: a product drawn into one of the two conversions rounds once, the other twice
                    if (T::kP == 2) asm("" : "+v"(x));
                    v[f][0][q] = (Half)x;
                    if constexpr (T::kP == 2) v[f][1][q] = (Half)(x - (float)v[f][0][q]);
                }
            // the lane halves hold entries 0-3, 8-11 and 4-7, 12-15 of sixteen: they trade, so that
            // each stores eight in a row
            const int m = m0 + t.row(i, 4 * g) + 4 * h;
#pragma unroll
            for (int p = 0; p < T::kP; ++p) {
                const u32x2 x = __builtin_bit_cast(u32x2, v[0][p]), y = __builtin_bit_cast(u32x2, v[1][p]);
                const auto s0 = __builtin_amdgcn_permlane32_swap(x[0], y[0], false, false);
                const auto s1 = __builtin_amdgcn_permlane32_swap(x[1], y[1], false, false);
                *(u32x4*)(out + Planes<T::kP>::at(m, p)) = u32x4{s0[0], s1[0], s0[1], s1[1]};
            }
        }
}

template <class T, Order W>
__global__ void __launch_bounds__(T::NT) vocab_grad_kernel(GradArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    const int count = *a.count, h = (threadIdx.x & 63) >> 5;
    if (n0 >= count) return;
    T t;
    t.template run<W, K_ROW>(lds, a.w, m0, a.x, n0, 0, a.slabs);
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        const bool live = n < count;
        const int token = live ? a.rows[n] : 0;
        // a token past the count has a row of zeros for X: its entries come out as 0 by their scale
        float lse = live ? a.lse[token] : 0.f, scale = live ? a.scale[token] : 0.f, alpha = a.alpha, value = 0.f;
        int entry = -1;  // the target's place in this piece
        if (a.target && live) {
            const long long v = a.target[token] - a.v0;
            entry = v >= 0 && v < a.vocab ? (int)v : -1;
            value = a.value[token];
        }
        const float most = T::kP == 2 && live ? log2f(kDMost / scale) : 0.f;
        if (T::kP == 2 && live) {
            alpha *= *a.w_unit * a.x_unit[n];
            scale *= kDScale;
            value *= kDScale;
        }
        const int first = m0 + t.row(0, 0) - 4 * h;  // of this wave's rows
        const bool plain = first + T::kWM <= a.vocab && !__any(entry >= first && entry < first + T::kWM);
        if (plain)
            grad_column<true>(t, a, j, n, m0, lse, scale, alpha, most, entry, value);
        else
            grad_column<false>(t, a, j, n, m0, lse, scale, alpha, most, entry, value);
    }
}

// How dX's product is cut: its tiles are few when tokens or hidden are, so the vocabulary is split
// until `groups` workgroups have work.  The same for every piece of a call and for vocab_dx_out.
struct DxCut {
    int tiles_m, bn, groups, most;
    __device__ int splits(int count) const {
        const int tiles = tiles_m * ((count + bn - 1) / bn);
        const int s = tiles > 0 ? groups / tiles : 1;
        return s < 1 ? 1 : s > most ? most : s;
    }
    __device__ size_t rows(int count) const { return (size_t)((count + bn - 1) / bn) * bn; }
};

struct DxArgs {
    Operand w, d;      // [vocabulary piece][hidden], [token][vocabulary piece]
    const int* count;
    const float* w_unit;
    DxCut cut;
    int slabs;
    float* acc;        // [splits][rows][hp]
    int hp;
    int add;           // not the first piece
};

template <class T>
__global__ void __launch_bounds__(T::NT) vocab_dx_kernel(DxArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    const int count = *a.count;
    const int splits = a.cut.splits(count), tiles_n = (count + T::kBN - 1) / T::kBN;
    const int tiles = a.cut.tiles_m * tiles_n;
    if ((int)blockIdx.x >= tiles * splits) return;
    const int z = blockIdx.x / tiles;
    int tm, tn;
    tile_of(blockIdx.x - z * tiles, tiles, a.cut.tiles_m, tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    const int first = (int)((long)a.slabs * z / splits), last = (int)((long)a.slabs * (z + 1) / splits);
    T t;
    t.template run<K_COL, K_ROW>(lds, a.w, m0, a.d, n0, first, last - first);
    const float unit = T::kP == 2 ? *a.w_unit : 1.f;
    const size_t rows = a.cut.rows(count);
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        if (n >= count) continue;
        float* out = a.acc + (z * rows + n) * a.hp + m0;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4* p = (f32x4*)(out + t.row(i, 4 * g));
                f32x4 v = {t.acc[i][j][4 * g], t.acc[i][j][4 * g + 1], t.acc[i][j][4 * g + 2], t.acc[i][j][4 * g + 3]};
                if (T::kP == 2) v *= unit;
                if (a.add) v += *p;
                *p = v;
            }
    }
}

struct DwArgs {
    Operand x, d;      // [token][hidden]; [token][vocabulary piece]
    const int* count;
    const float* x_most;  // P = 2: what a packed unit of X stands for
    int tiles_m, tiles_n, hidden, vocab;
    void* out;         // [vocabulary piece][hidden] in the operands' type
    long ld;
};

template <class T>
__global__ void __launch_bounds__(T::NT) vocab_dw_kernel(DwArgs a) {
    using O = typename std::conditional<T::kP == 1, __bf16, float>::type;
    __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
    int tm, tn;
    tile_of(blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, 4, tm, tn);
    const int m0 = tm * T::kBM, n0 = tn * T::kBN;
    T t;
    t.template run<K_COL, K_COL>(lds, a.x, m0, a.d, n0, 0, (*a.count + T::BK - 1) / T::BK);
    // 16 bytes a lane, at any alignment of O: two groups of four bf16 after the lane halves have traded
    // (as in vocab_grad_kernel), or one of fp32
    constexpr int E = 16 / sizeof(O), F = E / 4;
    typedef O Row __attribute__((ext_vector_type(E), aligned(sizeof(O))));
    const float unit = T::kP == 2 ? *a.x_most / kDScale : 1.f;
    const int h = (threadIdx.x & 63) >> 5;
    const bool whole = m0 + T::kBM <= a.hidden;
#pragma unroll
    for (int j = 0; j < T::NB; ++j) {
        const int n = n0 + t.col(j);
        O* out = (O*)a.out + (size_t)n * a.ld;
#pragma unroll
        for (int i = 0; i < T::MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; g += F) {
                O v[4 * F];
#pragma unroll
                for (int q = 0; q < 4 * F; ++q) v[q] = (O)(t.acc[i][j][4 * g + q] * unit);
                int m = m0 + t.row(i, 4 * g);
                u32x4 x;
                __builtin_memcpy(&x, v, 16);
                if constexpr (F == 2) {
                    const auto s0 = __builtin_amdgcn_permlane32_swap(x[0], x[2], false, false);
                    const auto s1 = __builtin_amdgcn_permlane32_swap(x[1], x[3], false, false);
                    x = u32x4{s0[0], s1[0], s0[1], s1[1]};
                    m += 4 * h;
                }
                if (n >= a.vocab) continue;
                if (whole || m + E <= a.hidden) {
                    *(Row*)(out + m) = __builtin_bit_cast(Row, x);
                } else {
                    __builtin_memcpy(v, &x, 16);
                    for (int q = 0; q < E; ++q)
                        if (m + q < a.hidden) out[m + q] = v[q];
                }
            }
    }
}

}  // namespace vocab
}  // namespace libsgemm
