// linear.hip -- entry points of the linear layer with an epilogue: argument checks, workspace, launches.
#include <limits.h>

#include "../../include/linear.h"
#include "kernel_linear.hpp"

namespace libsgemm {
namespace linear {
namespace {

constexpr int kMaxTokens = 1 << 24, kMaxOuts = 1 << 21, kMaxHidden = 1 << 20;
constexpr long kMaxElements = 1L << 35;  // of a result: its tiles' threads then are a grid
constexpr long kMaxPitch = 1L << 24;     // bytes: a tile's rows stay within 32-bit offsets

long up(long x, long to) { return (x + to - 1) / to * to; }

template <int P>
using Big = Tile<P, 256, 256, 128, 64, 3, 2>;
template <int P>
using Mid = typename std::conditional<P == 0, Tile<0, 128, 128, 64, 64, 2, 2>, Tile<1, 128, 128, 64, 32, 2, 2>>::type;
template <int P>
using Small = typename std::conditional<P == 0, Tile<0, 64, 64, 32, 32, 3, 3>, Tile<1, 128, 64, 64, 32, 3, 3>>::type;
enum Shape { SMALL, MID, BIG };

// A product's tile shape and the parts that its long axis is cut into.
struct Plan {
    Shape shape;
    int bm, bn, splits;
    long rows, pitch;  // of the parts
    long part_bytes() const { return splits > 1 ? 4L * splits * rows * pitch : 0; }
};

// The plan that takes least by an estimate in us: the rounds of workgroups over the chip's 256 compute units, each with
// what its slabs take at `rate` TFLOP/s of the whole chip and `end` us for its first loads and its stores; a last round
// that leaves a unit one workgroup of `places` takes `solo` of a round, of three places two 0.67; and for a cut product 3
// us, 0.1 a part and the pass over them.  The numbers are fitted to the products of 20 layers, each with every shape and cut:
// the plan takes 1 % more than the best of them in the mean.  Measured (us, M x N x k of the product, shape / splits):
//   fp32  4096 x 1024 x 4096: M/2 253, M/1 257, S/1 270;   4096 x 4096 x 1024: M/1 252, S/1 267;
//         5008 x 777 x 1000: S/1 90, M/4 102, M/1 128;     1000 x 777 x 5008: S/2 90, M/8 92, S/1 107;
//         640 x 1500 x 640: S/1 18, S/2 21, M/4 25, M/1 45;
//   bf16  8192 x 8192 x 4096: B/1 444, M/1 533, S/1 723;   4096 x 2048 x 1024: M/1 24, S/1 29, B/1 37;
//         1024 x 4096 x 4096: S/1 43, M/1 48, M/2 48;      4096 x 100 x 8192: S/4 22, M/8 29;
//         2048 x 2048 x 8192: M/2 79, B/4 80, S/1 82;      4096 x 8192 x 100: M/1 29, B/1 36, S/1 36.
// (64 parts at most: 64 x 128 x 131072 fp32 with its slopes 204 with 16, 83 with 64; bf16 76, 43.)
Plan plan_of(int P, long rows_m, long rows_n, long k) {
    const long slabs = up(k, P == 0 ? 32 : 64) / (P == 0 ? 32 : 64);
    Plan best{};
    double least = 0;
    auto look = [&](Shape shape, int bm, int bn, int places, double rate, double end, double solo) {
        const long tiles = up(rows_m, bm) / bm * (up(rows_n, bn) / bn), slots = 256L * places;
        for (int s = 1; s <= 64 && (s == 1 || s * 4 <= slabs); s *= 2) {
            const long groups = tiles * s, full = groups / slots, rest = groups - full * slots;
            const double last = rest == 0 ? 0 : rest <= 256 ? solo : places == 3 && rest <= 512 ? 0.67 : 1;
            const double flops = 2. * bm * bn * (P == 0 ? 32 : 64) * ((slabs + s - 1) / s);
            double us = (full + last) * (end + places * flops / (rate * 1e6 / 256));
            if (s > 1) us += 3 + 0.1 * s + 4. * (s + 1) * rows_m * rows_n / (P == 0 ? 6e6 : 4.5e6);
            if (least == 0 || us < least) {
                least = us;
                best = {shape, bm, bn, s, up(rows_n, bn), up(rows_m, bm)};
            }
        }
    };
    if (P == 0) {
        look(SMALL, 64, 64, 3, 135, 4, 0.4);
        look(MID, 128, 128, 2, 154, 8, 0.56);
    } else {
        look(SMALL, 128, 64, 2, 940, 3, 0.6);
        look(MID, 128, 128, 2, 1150, 2.2, 0.67);
        look(BIG, 256, 256, 1, 1375, 5, 1);
    }
    return best;
}

// The workspace: byte offsets of its arrays.  It goes by the sizes alone, so that it can be asked for beforehand;
// the packed operands have their places also where the operands will be read in place.
struct Layout {
    Plan z, dx, dw;
    int per, row_groups;  // of the slope's rows
    long hp, np;          // bytes of a packed row of hidden, of output features
    long x, w, dz, sums, part, bytes;
};

Layout layout(int P, bool grad, long T, long N, long H) {
    Layout l{};
    const long size = P == 0 ? 4 : 2;
    l.hp = up(H * size, 128);
    l.np = up(N * size, 128);
    long at = 0, part = 0;
    auto take = [&](long bytes) {
        const long o = at;
        at = up(at + bytes, 1024);
        return o;
    };
    l.x = take(l.hp * T);
    l.w = take(l.hp * N);
    if (!grad) {
        l.z = plan_of(P, N, T, H);
        part = l.z.part_bytes();
    } else {
        l.dx = plan_of(P, H, T, N);
        l.dw = plan_of(P, H, N, T);
        part = l.dx.part_bytes() > l.dw.part_bytes() ? l.dx.part_bytes() : l.dw.part_bytes();
        // workgroups of 1 KB of columns and so many rows that a compute unit has several, 16 rows at least
        const long cols = up(l.np, 1024) / 1024, want = 2048 / cols < 1 ? 1 : 2048 / cols;
        l.per = (int)up((T + want - 1) / want, 16);
        l.row_groups = (int)((T + l.per - 1) / l.per);
        l.dz = take(l.np * T);
        l.sums = take(4L * l.row_groups * (l.np / size));
    }
    l.part = take(part);
    l.bytes = at;
    return l;
}

bool few(int T) { return T <= vocab::kFewTokens; }

// The gradient of few tokens: dZ in fp32, X in the order that dW's product takes, dX's parts.
struct FewLayout {
    int nb, kt, splits;
    long hb, hp, vp, d, xt, acc, bytes;
};
FewLayout few_layout(bool f32, int T, int N, int H) {
    FewLayout l{};
    l.nb = T > 32 ? 4 : T > 16 ? 2 : 1;
    const int e = f32 && l.nb == 1 ? vocab::Fp32::E : 8, he = f32 ? 4 : 8;
    l.kt = (int)up(16 * l.nb, 4 * e) / (4 * e);
    l.hb = up(H, 8 * he) / 16;
    l.hp = up(H, 16 * he);
    l.vp = up(N, 64);
    // dX's pass over W in enough parts to fill the chip four times, each of 8 or 16 steps or more
    const long strips = l.hp / (16 * he), most = l.vp / 256, s = 1024 / strips < most ? 1024 / strips : most;
    l.splits = (int)(s < 1 ? 1 : s);
    long at = 0;
    auto take = [&](long bytes) {
        const long o = at;
        at = up(at + bytes, 1024);
        return o;
    };
    l.d = take(4L * 16 * l.nb * l.vp);
    l.xt = take(64L * e * (f32 ? 4 : 2) * l.hb * l.kt);
    l.acc = take(4L * l.splits * 16 * l.nb * l.hp);
    l.bytes = at;
    return l;
}

struct Call {
    bool f32, wide;
    int T, N, H, activation;
    const void* X;
    long ldx;
    const void* W;
    long ldw;
    const void *bias, *residual;
    long ldr;
    void* Y;
    long ldy;
    const void* dY;
    long lddy;
    const void* Z;
    long ldz;
    void* dX;
    long lddx;
    void* dW;
    long lddw;
    void* dbias;
    char* work;
    hipStream_t stream;
    Finish forward() const { return {T, N, activation, wide, bias, residual, ldr, const_cast<void*>(Z), ldz, Y, ldy}; }
    static Finish plain(int rows, int cols, void* out, long ld) {
        return {rows, cols, NONE, 0, nullptr, nullptr, 0, nullptr, 0, out, ld};
    }
};

// A matrix that the tile loop may read in place: whole aligned 16-byte quads, rows not too far apart.
bool in_place(const void* p, long ld, long cols, long size) {
    return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0 && cols * size % 16 == 0 && ld * size < kMaxPitch;
}

// The operand as the products read it, and what is to be packed for it, if anything.
Operand operand(const void* p, long ld, int rows, int cols, long size, char* packed, long pitch, PackArgs& pack) {
    if (in_place(p, ld, cols, size)) return {(const char*)p, (uint32_t)(ld * size), (uint32_t)(cols * size), rows};
    pack = {p, ld, rows, cols, packed, pitch / size};
    return {packed, (uint32_t)pitch, (uint32_t)pitch, rows};
}
template <typename T>
void prepare(const PrepareArgs& a, hipStream_t stream) {
    const int blocks = a.slopes() + a.w.blocks() + a.x.blocks();
    if (blocks > 0) linear_prepare_kernel<T><<<blocks, 256, 0, stream>>>(a);
}

template <int P, class F>
void by_shape(Shape shape, F f) {
    if constexpr (P == 1)
        if (shape == BIG) return f((Big<P>*)nullptr);
    if (shape == MID)
        f((Mid<P>*)nullptr);
    else
        f((Small<P>*)nullptr);
}

template <typename T, int P, Order OA, Order OB, bool TAIL>
void product(const Call& c, const Plan& p, const Operand& a, const Operand& b, long rows_m, long rows_n, long k,
             char* part, const Finish& f, const BiasArgs& bias = {}) {
    by_shape<P>(p.shape, [&](auto* shape) {
        using S = typename std::remove_pointer<decltype(shape)>::type;
        const int tm = (int)(up(rows_m, S::kBM) / S::kBM), tn = (int)(up(rows_n, S::kBN) / S::kBN);
        const ProductArgs args{a, b, tm, tn, (int)k, (int)(up(k, S::BK) / S::BK), p.splits, (float*)part, p.rows, p.pitch, f, bias};
        const long blocks = (long)tm * tn * p.splits + bias.blocks();
        linear_product_kernel<S, OA, OB, TAIL, OA != K_COL><<<(unsigned)blocks, S::NT, 0, c.stream>>>(args);
    });
    if (p.splits > 1)
        linear_sum_kernel<T><<<dim3((unsigned)rows_n, (unsigned)(up(rows_m, 1024) / 1024)), 256, 0, c.stream>>>(
            (const float*)part, p.splits, p.rows, p.pitch, f);
}

template <typename T, int P>
int forward(const Call& c) {
    const Layout l = layout(P, false, c.T, c.N, c.H);
    PrepareArgs p{};
    const Operand x = operand(c.X, c.ldx, c.T, c.H, sizeof(T), c.work + l.x, l.hp, p.x);
    const Operand w = operand(c.W, c.ldw, c.N, c.H, sizeof(T), c.work + l.w, l.hp, p.w);
    prepare<T>(p, c.stream);
    char* const part = c.work + l.part;
    if (x.row_bytes % 128 == 0 && w.row_bytes % 128 == 0)
        product<T, P, K_ROW, K_ROW, false>(c, l.z, w, x, c.N, c.T, c.H, part, c.forward());
    else
        product<T, P, K_ENDS, K_ENDS, true>(c, l.z, w, x, c.N, c.T, c.H, part, c.forward());
    return (int)hipGetLastError();
}

template <typename T, int P>
int gradient(const Call& c) {
    constexpr long size = sizeof(T);
    const Layout l = layout(P, true, c.T, c.N, c.H);
    const bool slope = c.activation != NONE, copy = slope || !in_place(c.dY, c.lddy, c.N, size);
    Operand d{(const char*)c.dY, (uint32_t)(c.lddy * size), (uint32_t)(c.N * size), c.T};
    if (copy) d = {c.work + l.dz, (uint32_t)l.np, (uint32_t)l.np, c.T};
    PrepareArgs p{};
    Operand w{}, x{};
    if (c.dX) w = operand(c.W, c.ldw, c.N, c.H, size, c.work + l.w, l.hp, p.w);
    if (c.dW) x = operand(c.X, c.ldx, c.T, c.H, size, c.work + l.x, l.hp, p.x);
    if (copy || c.dbias)
        p.slope = {c.dY, slope ? c.Z : nullptr, c.lddy, c.ldz, c.T, c.N, c.activation, l.per,
                   (int)(up(l.np, 1024) / 1024), l.row_groups, copy ? c.work + l.dz : nullptr, l.np / size,
                   c.dbias ? (float*)(c.work + l.sums) : nullptr};
    prepare<T>(p, c.stream);
    BiasArgs bias{};
    if (c.dbias) bias = {(const float*)(c.work + l.sums), l.row_groups, c.N, l.np / size, c.dbias};
    if (c.dbias && !c.dX && !c.dW) linear_bias_kernel<T><<<(unsigned)bias.blocks(), 256, 0, c.stream>>>(bias);
    char* const part = c.work + l.part;
    if (c.dX) {
        const Finish f = Call::plain(c.T, c.H, c.dX, c.lddx);
        if (d.row_bytes % 128 == 0)
            product<T, P, K_COL, K_ROW, true>(c, l.dx, w, d, c.H, c.T, c.N, part, f, bias);
        else
            product<T, P, K_COL, K_ENDS, true>(c, l.dx, w, d, c.H, c.T, c.N, part, f, bias);
    }
    if (c.dW)
        product<T, P, K_COL, K_COL, true>(c, l.dw, x, d, c.H, c.N, c.T, part, Call::plain(c.N, c.H, c.dW, c.lddw),
                                          c.dX ? BiasArgs{} : bias);
    return (int)hipGetLastError();
}

// Few tokens' forward product: 16 mr output features a workgroup of nw waves, the hidden size in `splits` parts ("mr x nw /
// splits" below).  Many features a workgroup read the tokens' side less often, and cut it into parts less often in fp32; few,
// and parts of the hidden size, fill the chip, but parts cost a second launch and a pass over their sums, some 2.5 us and
// more.  Each rule stands with the figures (us) of both its sides.  Of 98 sizes a type and number of tokens, 500 x 256 to
// 32768 x 2048 and 6144 x 8192, the plan takes 4 - 5 % more than the best of all in the mean with up to 16 tokens, 7 - 11 %
// with more: long sums of few features are cut too little there (fp32 64 tokens, 500 x 2048: 20.8, best 8.3 with 1x8/8; 20
// tokens, 6144 x 8192: 75, best 45 with 2x4/4).
struct FewPlan {
    int mr, nw, splits;
    long pitch;
};
FewPlan few_plan(bool f32, int T, int N, int H) {
    const int nb = T > 32 ? 4 : T > 16 ? 2 : 1, steps = (int)(up(H, 32) / (f32 && nb == 1 ? 16 : 32));
    FewPlan p{1, 8, 1, up(N, 64)};
    // 33 tokens and more: 64 features a workgroup once three of four compute units have one (bf16 64 tokens, 32768 x 1024: 20
    // with 4x4/1, 39 with 1x8/1; 12288 x 1024: 12.5, 16.7; 8192 x 1024 they are even, 12.1, 12.2; fp32 12288 x 1024: 23.5,
    // 31.2); from half of that on with the hidden size in two, where it is long (bf16 64 tokens, 6144 x 2048: 15.3 with
    // 4x4/2, 18.8 with 4x4/1, 20.9 with 1x8/1; 4096 x 2048: 14.6, 18.7, 12.4)
    if (nb == 4 && (N >= 64 * 192 || (N >= 64 * 96 && steps >= 64))) {
        p.mr = 4, p.nw = 4, p.splits = N >= 64 * 192 ? 1 : 2;
        return p;
    }
    // fp32: cutting the tokens' values into parts, anew for each workgroup, is what counts: 64 features a workgroup as above,
    // with as many parts as give about as many workgroups, if each wave keeps four steps (64 tokens, 2048 x 4096: 18.9 with
    // 4x4/8, 25 with 1x8/4, 38 with 1x8/1; 8192 x 1024: 18.2 with 4x4/2, 21.7 with 1x8/1; with two steps, 4096 x 1024: 14.9
    // with 4x4/4, 12.9 with 1x8/1)
    if (f32 && nb == 4) {
        const long groups = up(N, 64) / 64;
        int s = 1;
        while (s < 16 && groups * s < 184) s *= 2;
        if (groups * s >= 184 && steps / (4 * s) >= 4) {
            p.mr = 4, p.nw = 4, p.splits = s;
            return p;
        }
    }
    // 17 to 32: 32 features once all compute units have a workgroup (20 tokens, 32768 x 1024: bf16 16.5 with 2x4/1, 20.5 with
    // 1x8/1; 8192 x 1024: fp32 11.7, 13.3; bf16 7.1, 7.4; 4096 x 1024: fp32 11.3, 8.4; bf16 6.5, 5.0)
    if (nb == 2 && N >= 32 * 256) {
        p.mr = 2, p.nw = 4;
        return p;
    }
    // else 16 features a workgroup, of four waves from 64 workgroups on, of eight before, and of eight with 33 tokens or more
    // and where fp32 is cut into parts (bf16 1 token, 32768 x 1024: 12.0 with 1x4/1, 12.1 with 1x8/1; 2048 x 1024: 4.4, 4.4;
    // 1000 x 1024: 4.6, 4.4; fp32 20 tokens, 4096 x 1024: 8.9, 8.4)
    const long blocks = up(N, 16) / 16;
    if (!(f32 && nb == 2) && nb < 4 && blocks >= 64) p.nw = 4;
    // a sum is cut once a wave has `from` steps or more of it, in two again and again until it has at most `to` or the
    // workgroups are 256 (bf16 1 token, 1000 x 8192: 8.0 with 1x8/4, 11.3 with 1x8/1; 500 x 4096, 16 steps: 6.7, 6.9; 4096 x
    // 4096: 8.9 with 1x4/1, 10.8 with 1x4/2; fp32 1 token, 500 x 4096: 7.1 with 1x8/8, 11.7 with 1x8/1; 500 x 2048: 7.3 with
    // 1x8/4, 7.2 with 1x8/1; 32 tokens, 2048 x 4096: 16.5 with 1x8/2, 23.7 with 1x8/1; 40 tokens, 500 x 4096: 9.4 with 1x8/8,
    // 28.5 with 1x8/1; 4096 x 1024: 10.3 with 1x8/1, 13.3 with 1x8/2)
    const int from = p.nw == 4 ? 32 : nb > 1 ? 12 : f32 ? 16 : 32, to = nb == 1 ? (f32 ? 4 : 8) : f32 ? 2 : 4;  // steps of a wave
    if (steps / p.nw >= from)
        while (steps / (p.nw * p.splits) > to && blocks * p.splits < 256 && p.splits < 16) p.splits *= 2;
    return p;
}

template <class C, int NB>
int few_forward(const Call& c) {
    const FewPlan p = few_plan(c.f32, c.T, c.N, c.H);
    const int blocks = (int)(up(c.N, 16 * p.mr) / (16 * p.mr)), grid = blocks * p.splits;
    const FewArgs a{c.T, c.N, c.H, c.X, c.W, c.ldx, c.ldw, blocks, p.splits, (float*)c.work, p.pitch, c.forward()};
    constexpr int MR = NB == 3 ? 4 : NB;
    if constexpr (NB > 1)
        if (p.mr == MR) linear_few_kernel<C, NB, MR, 4><<<grid, 256, 0, c.stream>>>(a);
    if constexpr (NB < 3)
        if (p.mr == 1 && p.nw == 4) linear_few_kernel<C, NB, 1, 4><<<grid, 256, 0, c.stream>>>(a);
    if (p.mr == 1 && p.nw == 8) linear_few_kernel<C, NB, 1, 8><<<grid, 512, 0, c.stream>>>(a);
    if (p.splits > 1)
        linear_sum_kernel<typename C::T><<<dim3(c.T, (unsigned)(up(c.N, 1024) / 1024)), 256, 0, c.stream>>>(
            a.part, p.splits, 16 * NB, p.pitch, a.f);
    return (int)hipGetLastError();
}

template <class C, int NB>
int few_gradient(const Call& c) {
    typedef typename C::T T;
    const FewLayout l = few_layout(c.f32, c.T, c.N, c.H);
    const int chunks = c.dW ? (int)(64 * l.hb * l.kt) : 0, groups = (int)(l.vp / 64);
    float *const d = (float*)(c.work + l.d), *const acc = (float*)(c.work + l.acc);
    const FewSlopeArgs s{c.dY, c.activation != NONE ? c.Z : nullptr, c.X, c.lddy, c.ldz, c.ldx, c.T, c.N, c.H,
                         c.activation, groups, d, l.vp, c.dbias, c.work + l.xt, l.kt, chunks};
    linear_few_slope_kernel<C, NB><<<(unsigned)(groups + (chunks + 255) / 256), 256, 0, c.stream>>>(s);
    // dW: 256 rows of it and as many groups of 128 bytes as leave eight workgroups a compute unit, two or more
    const long row_groups = up(c.N, 256) / 256, all = up(c.H, 8 * C::HE) / (8 * C::HE);
    const long cols = 2048 / row_groups < 1 ? 1 : 2048 / row_groups, even = (all + cols - 1) / cols;
    const long own = even < 2 ? 2 : even, dw_blocks = c.dW ? row_groups * ((all + own - 1) / own) : 0;
    const int strips = c.dX ? (int)(l.hp / (16 * C::HE)) : 0;
    if (strips * l.splits + dw_blocks > 0) {
        const vocab::FewGradArgs g{d, l.vp, c.T, c.N, c.H, c.W, c.ldw, strips, l.splits, acc, (int)l.hp, 0,
                                   c.work + l.xt, (int)own, (int)row_groups, c.dW, c.lddw};
        vocab::vocab_few_grad_kernel<C, NB><<<(unsigned)(strips * l.splits + dw_blocks), 256, 0, c.stream>>>(g);
    }
    if (c.dX)
        linear_sum_kernel<T><<<dim3(c.T, (unsigned)(up(c.H, 1024) / 1024)), 256, 0, c.stream>>>(
            acc, l.splits, 16 * NB, l.hp, Call::plain(c.T, c.H, c.dX, c.lddx));
    return (int)hipGetLastError();
}

template <class F>
int by_mode(bool f32, int T, F f) {
    using vocab::Bf16;
    using vocab::Fp32;
    using vocab::Fp32Split;
    if (T <= 16) return f32 ? f((Fp32*)nullptr, std::integral_constant<int, 1>{}) : f((Bf16*)nullptr, std::integral_constant<int, 1>{});
    if (T <= 32)
        return f32 ? f((Fp32Split*)nullptr, std::integral_constant<int, 2>{}) : f((Bf16*)nullptr, std::integral_constant<int, 2>{});
    return f32 ? f((Fp32Split*)nullptr, std::integral_constant<int, 4>{}) : f((Bf16*)nullptr, std::integral_constant<int, 4>{});
}

template <typename T>
int zeros(const Call& c) {
    if (c.dW)
        linear_zero_kernel<T><<<dim3(c.N, (unsigned)(c.H < 65536 ? up(c.H, 256) / 256 : 256)), 256, 0, c.stream>>>(
            (T*)c.dW, c.lddw, c.H);
    if (c.dbias)
        linear_zero_kernel<T><<<dim3(1, (unsigned)(up(c.N, 256) / 256)), 256, 0, c.stream>>>((T*)c.dbias, c.N, c.N);
    return (int)hipGetLastError();
}

int run(const Call& c, bool grad) {
    if (c.T == 0 && !c.dW && !c.dbias) return 0;
    (void)hipGetLastError();
    if (c.T == 0) return c.f32 ? zeros<float>(c) : zeros<__bf16>(c);
    // 33 to 48 tokens are three blocks of 16 forward (40 tokens, with four us, so: fp32 5003 x 777: 13.7, 11.7; 2048 x
    // 4096: 26.7, 19.3; bf16 5003 x 777: 16.4, 15.0; 32768 x 1024: 19.4, 18.0), but not in fp32 with four rows of features
    // (32768 x 1024: 34.8 with four blocks, 40.1 with three; 8192 x 4096: 41.2, 46.6)
    if (!grad && c.T > 32 && c.T <= 48 && !(c.f32 && few_plan(true, c.T, c.N, c.H).mr == 4))
        return c.f32 ? few_forward<vocab::Fp32Split, 3>(c) : few_forward<vocab::Bf16, 3>(c);
    if (few(c.T))
        return by_mode(c.f32, c.T, [&](auto* mode, auto nb) {
            using C = typename std::remove_pointer<decltype(mode)>::type;
            return grad ? few_gradient<C, decltype(nb)::value>(c) : few_forward<C, decltype(nb)::value>(c);
        });
    if (grad) return c.f32 ? gradient<float, 0>(c) : gradient<__bf16, 1>(c);
    return c.f32 ? forward<float, 0>(c) : forward<__bf16, 1>(c);
}

// Position (from 0) of the first size out of range, or -1.
int bad_size(long T, long N, long H) {
    if (T < 0 || T > kMaxTokens) return 0;
    if (N < 1 || N > kMaxOuts || T * N > kMaxElements) return 1;
    if (H < 1 || H > kMaxHidden || T * H > kMaxElements) return 2;
    return -1;
}

// A row-major matrix's span, first to last addressed byte.
struct Span {
    const void* p;
    long rows, ld, cols, size;
    bool meets(const Span& o) const {
        if (!p || !o.p || rows == 0 || o.rows == 0) return false;
        const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
        return a < b + ((o.rows - 1) * o.ld + o.cols) * o.size && b < a + ((rows - 1) * ld + cols) * size;
    }
};
bool aligned(const void* p, long size) { return (uintptr_t)p % size == 0; }

}  // namespace
}  // namespace linear
}  // namespace libsgemm

using namespace libsgemm::linear;

extern "C" {

long long linear_workspace(int dtype, int grad, int T, int N, int H) {
    if (dtype != LINEAR_F32 && dtype != LINEAR_BF16) return -1;
    const int bad = bad_size(T, N, H);
    if (bad >= 0) return -3 - bad;
    if (T == 0) return 0;
    if (few(T) && !grad) {
        const FewPlan p = few_plan(dtype == LINEAR_F32, T, N, H);
        return p.splits > 1 ? 4L * p.splits * (T > 32 ? 64 : T > 16 ? 32 : 16) * p.pitch : 0;
    }
    if (few(T)) return few_layout(dtype == LINEAR_F32, T, N, H).bytes;
    return layout(dtype == LINEAR_F32 ? 0 : 1, grad != 0, T, N, H).bytes;
}

int linear_act(int dtype, int out_dtype, int T, int N, int H, const void* X, int ldx, const void* W, int ldw,
               const void* bias, const void* residual, int ldr, int activation, void* Y, int ldy, void* Z, int ldz,
               void* work, long long work_bytes, hipStream_t stream) {
    if (dtype != LINEAR_F32 && dtype != LINEAR_BF16) return -1;
    if (out_dtype != dtype && out_dtype != LINEAR_F32) return -2;
    const int bad = bad_size(T, N, H);
    if (bad >= 0) return -3 - bad;
    const long size = dtype == LINEAR_F32 ? 4 : 2, out_size = out_dtype == LINEAR_F32 ? 4 : 2;
    if (ldx < H) return -7;
    if (ldw < H) return -9;
    if (residual && ldr < N) return -12;
    if (activation < LINEAR_NONE || activation > LINEAR_SILU) return -13;
    if (ldy < N) return -15;
    if (Z && ldz < N) return -17;
    if (T == 0) return 0;
    if (!X || !aligned(X, size)) return -6;
    if (!W || !aligned(W, size)) return -8;
    if (!aligned(bias, size)) return -10;
    if (!aligned(residual, out_size)) return -11;
    if (!Y || !aligned(Y, out_size)) return -14;
    if (!aligned(Z, size)) return -16;
    const long need = linear_workspace(dtype, 0, T, N, H);
    if (need > 0 && (!work || !aligned(work, 16))) return -18;
    if (work_bytes < need) return -19;
    const Span y{Y, T, ldy, N, out_size}, z{Z, T, ldz, N, size};
    const Span in[] = {{X, T, ldx, H, size}, {W, N, ldw, H, size}, {bias, 1, N, N, size}, {residual, T, ldr, N, out_size}};
    for (const Span& s : in) {
        if (y.meets(s)) return -14;
        if (z.meets(s)) return -16;
    }
    if (z.meets(y)) return -16;
    Call c{};
    c.f32 = dtype == LINEAR_F32, c.wide = out_dtype != dtype;
    c.T = T, c.N = N, c.H = H, c.activation = activation;
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw, c.bias = bias, c.residual = residual, c.ldr = ldr;
    c.Y = Y, c.ldy = ldy, c.Z = Z, c.ldz = ldz;
    c.work = (char*)work, c.stream = stream;
    return run(c, false);
}

int linear_act_grad(int dtype, int T, int N, int H, const void* X, int ldx, const void* W, int ldw, const void* dY,
                    int lddy, const void* Z, int ldz, int activation, void* dX, int lddx, void* dW, int lddw,
                    void* dbias, void* work, long long work_bytes, hipStream_t stream) {
    if (dtype != LINEAR_F32 && dtype != LINEAR_BF16) return -1;
    const int bad = bad_size(T, N, H);
    if (bad >= 0) return -2 - bad;
    const long size = dtype == LINEAR_F32 ? 4 : 2;
    if (ldx < H) return -6;
    if (ldw < H) return -8;
    if (lddy < N) return -10;
    if (activation < LINEAR_NONE || activation > LINEAR_SILU) return -13;
    if (activation != LINEAR_NONE && ldz < N) return -12;
    if (dX && lddx < H) return -15;
    if (dW && lddw < H) return -17;
    if (!dX && !dW && !dbias) return 0;
    if (!aligned(dX, size)) return -14;
    if (!aligned(dW, size)) return -16;
    if (!aligned(dbias, size)) return -18;
    if (T > 0) {
        if ((dW && !X) || !aligned(X, size)) return -5;
        if ((dX && !W) || !aligned(W, size)) return -7;
        if (!dY || !aligned(dY, size)) return -9;
        if (activation != LINEAR_NONE && (!Z || !aligned(Z, size))) return -11;
    }
    const long need = linear_workspace(dtype, 1, T, N, H);
    if (need > 0 && (!work || !aligned(work, 16))) return -19;
    if (work_bytes < need) return -20;
    const Span out[] = {{dX, T, lddx, H, size}, {dW, N, lddw, H, size}, {dbias, 1, N, N, size}};
    const Span in[] = {{X, T, ldx, H, size}, {W, N, ldw, H, size}, {dY, T, lddy, N, size},
                       {activation != LINEAR_NONE ? Z : nullptr, T, ldz, N, size}};
    for (int o = 0; o < 3; ++o) {
        for (const Span& s : in)
            if (out[o].meets(s)) return -14 - 2 * o;
        for (int p = 0; p < o; ++p)
            if (out[o].meets(out[p])) return -14 - 2 * o;
    }
    Call c{};
    c.f32 = dtype == LINEAR_F32;
    c.T = T, c.N = N, c.H = H, c.activation = activation;
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
    c.dY = dY, c.lddy = lddy, c.Z = Z, c.ldz = ldz;
    c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw, c.dbias = dbias;
    c.work = (char*)work, c.stream = stream;
    return run(c, true);
}

}  // extern "C"
