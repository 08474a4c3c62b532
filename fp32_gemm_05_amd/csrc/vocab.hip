// vocab.hip -- entry points of the vocabulary-head operators: cross entropy and distillation over
// the logits z = alpha * X W^T, forward and gradient, without the T x V logits in memory.
//
// Forward: one product whose tiles end as per-token maxima and sums of exponentials (log-sum-exp),
// and one dot product per named entry.  Gradient: the vocabulary is taken in pieces (one, where it fits
// kPieceBytes); a piece's logits are recomputed into D = d(loss)/dz (bf16, or two fp16 planes for fp32),
// from which dX += D W and dW = D^T X follow.  The tokens that do not count are left out at the start: the
// others are packed together, so they cost no product, and whatever their rows hold reaches no
// gradient.
#include <limits.h>

#include "../../include/vocab.h"
#include "kernel_vocab_few.hpp"

namespace libsgemm {
namespace vocab {
namespace {

constexpr int kMaxRows = INT_MAX - 1024;
constexpr int kMaxHidden = 1 << 20;                // a tile's packed rows stay within 32-bit byte offsets
constexpr int kMaxTokens = 1 << 21;
constexpr long kPieceBytes = 768L << 20;           // workspace of one piece of the vocabulary

struct Call {
    bool f32, grad;
    bool distill;  // not e.teacher: of no tokens that may be null
    int T, V, H;
    Entries e;
    float alpha;
    const void* X;
    long ldx;
    const void* W;
    long ldw;
    float *loss, *lse_out, *picked_out;
    const float *lse, *picked, *dloss;
    void* dX;
    long lddx;
    void* dW;
    long lddw;
    char* work;
    hipStream_t stream;
};

long up(long x, long to) { return (x + to - 1) / to * to; }

// What the sort of the entries takes of the workspace, and its launch (distillation's gradient).
long keys_bytes(int T, int K) { return K > kSortInLds ? 8L * T * K : 0; }
bool shared(const Call& c) { return c.grad && c.distill && c.e.k > kPairs && c.T > 0; }
void launch_shares(const Call& c, long keys, long value) {
    if (!shared(c)) return;
    uint64_t* const k = (uint64_t*)(c.work + keys);
    float* const v = (float*)(c.work + value);
    if (c.e.k > kSortInLds)
        vocab_shares_kernel<false><<<c.T, 1024, 0, c.stream>>>(c.e, c.V, k, v);
    else
        vocab_shares_kernel<true><<<c.T, 1024, 0, c.stream>>>(c.e, c.V, k, v);
}

// Tile shapes.  The large one has a compute unit to itself, of the others two share one.
template <int P>
using Big = Tile<P, 256, 256, 128, 64, 3, 2>;
template <int P>
using Mid = Tile<P, 128, 128, 64, 32, 2, 2>;
template <int P>
using Small = Tile<P, 128, 64, 64, 32, 3, 3>;
enum Shape { SMALL, MID, BIG };

// The workspace: byte offsets of its arrays for a call's sizes (the pointers of the call are not
// looked at, so that its size can be asked for beforehand; so a packed W has its place also where bf16 W will
// be read as it stands).
struct Layout {
    int tp, hk, hp;     // padded tokens, hidden as a product's k, hidden as a product's rows
    int piece, pieces;  // vocabulary rows of a piece (a multiple of 256), number of pieces
    DxCut cut;
    Shape dx_shape;
    long count, rows, pos, z, scale, weight, keys, x_unit, x_most, x_part, w_part, w_unit, value, x, xs, w, d, part, acc, bytes;
};

constexpr int kMaxBlocks = 1024;  // workgroups that look for W's largest value
// and at the tokens or entries: in a gradient call so many that their maxima are few, in a forward call all
// that a grid of less than 2^32 threads holds with room to spare
constexpr int kMostTokenBlocks = 2048, kMostEntryBlocks = 1 << 20;
constexpr int kPartRows = 64;  // the fewest vocabulary rows behind one partial sum

// The shape for a product of rows_m x rows_n: the one whose rounds over the chip's 256 compute units
// take least.  A round costs the area that a compute unit works on over the rate that the shape reaches
// in long products (2048 tokens, 32768 x 2048: the middle one 0.92 of the large one's in fp32 and 0.82
// in bf16, the small one 0.77 and 0.68); a last round that leaves each unit one tile of two takes 0.6
// of a round's time.  Measured (fp32, forward product, us, small/middle/large): 1362 tokens, 15116 x 444:
// 68, 60, 70; 500 tokens, 60000 x 256: 60, 52, 49; 300 tokens, 20000 x 1000: 55, 53, 74; 2142 tokens,
// 576 x 3392: 50, 77, -.
Shape shape_of(int P, long rows_m, long rows_n) {
    auto cost = [&](long bm, long bn, int places, double rate) {
        const long tiles = up(rows_m, bm) / bm * (up(rows_n, bn) / bn), slots = 256L * places;
        const long full = tiles / slots, rest = tiles - full * slots;
        const double last = rest == 0 ? 0 : places > 1 && rest <= 256 ? 0.6 : 1;
        return (full + last) * places * bm * bn / rate;
    };
    const double small = cost(128, 64, 2, P == 2 ? 0.77 : 0.68), mid = cost(128, 128, 2, P == 2 ? 0.92 : 0.82);
    const double big = cost(256, 256, 1, 1);
    return big <= mid && big <= small ? BIG : mid < small ? MID : SMALL;
}

Layout layout(int P, bool grad, int T, int V, int H, int K, bool teacher) {
    Layout l{};
    const int bk = 64 / P;
    l.tp = (int)up(T > 0 ? T : 1, 256);
    l.hk = (int)up(H, bk);
    l.hp = (int)up(H, 256);
    const long vp = up(V, 256);
    const long element = 2L * P;  // bytes in planes
    const long per = element * (l.hk + (grad ? l.tp : 0));
    long piece = kPieceBytes / per / 256 * 256;
    // a launch's grid stays below 2^22 tiles, a packed row below 2^24 bytes
    const long most = 128L * ((1L << 22) / (l.tp / 64)) / 256 * 256;
    if (piece > most) piece = most;
    if (piece > 1L << 21) piece = 1L << 21;
    if (piece < 256) piece = 256;
    if (piece > vp) piece = vp;
    const long pieces = (vp + piece - 1) / piece;
    l.piece = (int)up((vp + pieces - 1) / pieces, 256);
    l.pieces = (int)((vp + l.piece - 1) / l.piece);
    // dX's workgroups: its tiles, or about as many as the chip has places for (one large tile a
    // compute unit, two of the others), with 8 slabs or more each.  Large tiles if they fill most places
    // and cover no more than the middle ones do; these if each place gets 600 vocabulary rows of a tile
    // or more, as the small ones have less to fill and to sum at the ends.  Measured (dX and its sum,
    // fp32, us, small/middle/large): 1001 tokens, 50021 x 1000: 342, 292, 271; 500 tokens, 60000 x 256:
    // 98, 86, 71; 777 tokens, 5003 x 1001: 40, 42, 52; 300 tokens, 20000 x 1000: 73, 68, 80; 128 tokens,
    // 30000 x 2048: 89, 78, -; 1340 tokens, 3070 x 174: 18, 22, -.
    const int slabs = l.piece / bk, most_cuts = slabs / 8 > 1 ? slabs / 8 : 1;
    auto cut = [&](int bm, int bn, int places) {
        const int tiles_m = (int)(up(H, bm) / bm), tiles = tiles_m * (int)(up(l.tp, bn) / bn);
        return DxCut{tiles_m, bn, tiles > places ? tiles : places / tiles * tiles, most_cuts};
    };
    const long large = up(H, 256) * up(T, 256), middle = up(H, 128) * up(T, 128);
    if (T > 128 && H > 128 && large / (256 * 256) * most_cuts >= 192 && middle * 10 > large * 9)
        l.dx_shape = BIG, l.cut = cut(256, 256, 256);
    else if ((double)middle * l.piece >= 600. * 512 * 128 * 128)
        l.dx_shape = MID, l.cut = cut(128, 128, 512);
    else
        l.dx_shape = SMALL, l.cut = cut(128, 64, 512);
    long at = 0;
    auto take = [&](long bytes) {
        const long o = at;
        at = up(at + bytes, 1024);
        return o;
    };
    l.count = take(4);
    l.rows = take(4L * l.tp);
    l.pos = take(4L * l.tp);
    if (!teacher) l.z = take(4L * l.tp);
    l.x_unit = take(4L * l.tp);
    l.w_unit = take(4L * l.piece);
    l.w_part = take(4L * kMaxBlocks);
    l.x = take(element * l.hk * l.tp);
    l.w = take(element * l.hk * l.piece);
    if (grad) {
        l.scale = take(4L * l.tp);
        l.weight = take(4L * l.tp);
        l.keys = take(keys_bytes(T, K));
        l.value = take(4L * T * K);
        if (P == 2) l.x_most = take(4), l.x_part = take(4L * kMostTokenBlocks);
        if (P == 2 || !teacher) l.xs = take(element * l.hk * l.tp);
        l.d = take(element * l.tp * l.piece);
        l.acc = take(4L * l.hp * ((long)l.cut.groups / l.cut.tiles_m * l.cut.bn));
    } else {
        l.part = take(8L * (vp / kPartRows) * l.tp);
    }
    l.bytes = at;
    return l;
}

// At most kFewTokens tokens (kernel_vocab_few.hpp).  nb: blocks of 16 tokens.
struct FewLayout {
    int nb, kt, piece, pieces, splits;
    long hb, hp, vp, z, scale, weight, keys, value, xtf, d, part, acc, bytes;
};

FewLayout few_layout(bool f32, bool grad, int T, int V, int H, int K) {
    FewLayout l{};
    l.nb = T > 32 ? 4 : T > 16 ? 2 : 1;
    const int e = f32 && l.nb == 1 ? Fp32::E : 8, he = f32 ? 4 : 8;
    l.kt = (int)up(16 * l.nb, 4 * e) / (4 * e);
    l.hb = up(H, 8 * he) / 16;  // dW's groups are 128 bytes of hidden
    l.hp = up(H, 16 * he);
    const long vp = up(V, 64);
    l.piece = (int)(vp < 1L << 21 ? vp : 1L << 21);
    l.pieces = (int)((vp + l.piece - 1) / l.piece);
    l.vp = l.piece;
    // dX's pass over W in enough parts to fill the chip four times, each of 8 or 16 steps or more
    const long strips = l.hp / (16 * he), most = l.vp / 256;
    const long s = 1024 / strips < most ? 1024 / strips : most;
    l.splits = (int)(s < 1 ? 1 : s);
    long at = 0;
    auto take = [&](long bytes) {
        const long o = at;
        at = up(at + bytes, 1024);
        return o;
    };
    l.z = take(4 * kFewTokens);
    if (grad) {
        l.scale = take(4 * kFewTokens);
        l.weight = take(4 * kFewTokens);
        l.keys = take(keys_bytes(T, K));
        l.value = take(4L * T * K);
        l.xtf = take(64L * e * (f32 ? 4 : 2) * l.hb * l.kt);
        l.d = take(4L * 16 * l.nb * l.vp);
        l.acc = take(4L * l.splits * 16 * l.nb * l.hp);
    } else {
        l.part = take(8L * kFewTokens * (vp / 32));
    }
    l.bytes = at;
    return l;
}

bool few(int T) { return T > 0 && T <= kFewTokens; }

TokenArgs token_args(const Call& c, char* ws, float* z, long scale, long weight, long value, DForm form) {
    const int per = entries_per_wave(c.T, c.e.k);
    return {c.e, c.T, c.V, c.H, c.alpha, c.X, c.W, c.ldx, c.ldw, z, c.lse, c.dloss, c.picked,
            (float*)(ws + scale), (float*)(ws + weight), (float*)(ws + value), form, shared(c), per,
            c.grad ? c.T : c.T * (up(c.e.k, per) / per)};
}
// Workgroups of four waves for the entries (forward) or the tokens (gradient).
unsigned token_blocks(const Call& c, const TokenArgs& t) {
    const long blocks = up(t.waves, 4) / 4, most = c.grad ? kMostTokenBlocks : kMostEntryBlocks;
    return (unsigned)(blocks < most ? blocks : most);
}

template <class C, int NB>
int run_few(const Call& c, const FewLayout& l) {
    typedef typename C::T T;
    char* ws = c.work;
    auto floats = [&](long at) { return (float*)(ws + at); };
    const T* W = (const T*)c.W;
    const hipStream_t st = c.stream;
    // vocabulary rows of a workgroup's logits: 64 where three in four compute units get one (40 tokens,
    // fp32 20000 x 2000: 67 us against 88 us with 32, as the tokens' side is read and cut half as often),
    // 32 where they do not (40 tokens, fp32 2000 x 300: 13 us against 8 us).  fp32's 32 in three parts have a
    // compute unit to themselves, so there 64 are taken once 32 would need a second round (60 tokens,
    // 12000 x 1000: 25 us against 33; 50 tokens, 8300 x 1000: 24 against 31)
    const bool wide = NB == 4 && c.V >= (C::P == 3 ? 32 * 256 + 1 : 64 * 192);
    const int per = wide ? 64 : 32;
    (void)hipGetLastError();

    float* const z = c.distill ? c.picked_out : floats(l.z);
    if (c.distill) {
        launch_shares(c, l.keys, l.value);
        const TokenArgs t = token_args(c, ws, z, l.scale, l.weight, l.value, D_WHOLE);
        if (c.grad)
            vocab_few_token_kernel<T, true><<<token_blocks(c, t), 256, 0, st>>>(t);
        else
            vocab_few_token_kernel<T, false><<<token_blocks(c, t), 256, 0, st>>>(t);
    }
    int part = 0;
    for (int p = 0; p < l.pieces; ++p) {
        const int v0 = p * l.piece, vn = c.V - v0 < l.piece ? c.V - v0 : l.piece;
        const T* Wp = W + (size_t)v0 * c.ldw;
        const int groups = (int)(up(vn, per) / per);
        const int chunks = c.grad && c.dW && p == 0 ? (int)(64 * l.hb * l.kt) : 0;
        const FewArgs a{c.e, c.T, c.X, Wp, c.ldx, c.ldw, vn, c.H, groups, c.V, c.alpha, v0,
                        (float2*)(ws + l.part) + (size_t)part * kFewTokens, z, c.lse, c.dloss, floats(l.scale),
                        floats(l.d), l.vp, ws + l.xtf, l.kt, chunks};
        const unsigned blocks = groups + (chunks + 255) / 256;
        if (c.grad && wide)
            vocab_few_logits_kernel<C, NB, NB == 4 ? 4 : 2, true><<<blocks, 256, 0, st>>>(a);
        else if (c.grad)
            vocab_few_logits_kernel<C, NB, 2, true><<<blocks, 256, 0, st>>>(a);
        else if (wide)
            vocab_few_logits_kernel<C, NB, NB == 4 ? 4 : 2, false><<<blocks, 256, 0, st>>>(a);
        else
            vocab_few_logits_kernel<C, NB, 2, false><<<blocks, 256, 0, st>>>(a);
        if (!c.grad) {
            part += groups;
            continue;
        }
        if (c.distill)
            vocab_patch_kernel<0><<<(unsigned)(up((long)c.T * c.e.k, 256) / 256), 256, 0, st>>>(
                c.e, c.T, v0, vn, nullptr, floats(l.value), ws + l.d, l.vp * 4);
        // dW: 256 vocabulary rows and as many groups as leave eight workgroups a compute unit, but two
        // groups or more: a wave reads its rows' D first
        const long row_groups = up(vn, 256) / 256, all = up(c.H, 8 * C::HE) / (8 * C::HE);
        const long cols = 2048 / row_groups < 1 ? 1 : 2048 / row_groups;
        const long even = (all + cols - 1) / cols, own = even < 2 ? 2 : even;
        const int strips = c.dX ? (int)(l.hp / (16 * C::HE)) : 0;
        const FewGradArgs g{floats(l.d), l.vp, c.T, vn, c.H, Wp, c.ldw, strips, l.splits, floats(l.acc), (int)l.hp,
                            p > 0, ws + l.xtf, (int)own, (int)row_groups, (T*)c.dW + (size_t)v0 * c.lddw, c.lddw};
        const long dw_blocks = c.dW ? row_groups * ((all + own - 1) / own) : 0;
        vocab_few_grad_kernel<C, NB><<<(unsigned)(strips * l.splits + dw_blocks), 256, 0, st>>>(g);
    }
    if (!c.grad) {
        vocab_loss_kernel<2><<<(unsigned)(up(c.T, 2) / 2), 1024, 0, st>>>(
            c.e, nullptr, nullptr, c.T, c.V, (const float2*)(ws + l.part), part, kFewTokens, z, c.loss, c.lse_out);
    } else if (c.dX) {
        const DxCut cut{1, 16 * NB, l.splits, l.splits};
        vocab_dx_out_kernel<T, 0, 16><<<dim3(c.T, (unsigned)(up(c.H, 64) / 64)), 256, 0, st>>>(
            c.e, nullptr, nullptr, c.H, floats(l.acc), cut, (int)l.hp, nullptr, (T*)c.dX, c.lddx);
    }
    return (int)hipGetLastError();
}

int run_few(const Call& c) {
    const FewLayout l = few_layout(c.f32, c.grad, c.T, c.V, c.H, c.e.k);
    if (!c.f32) return l.nb == 1 ? run_few<Bf16, 1>(c, l) : l.nb == 2 ? run_few<Bf16, 2>(c, l) : run_few<Bf16, 4>(c, l);
    // Fp32Split from 17 tokens: 100000 x 1536 with 17 tokens scored in 145 us against 170 us by Fp32, with
    // 33 tokens in 177 us against 265 us
    return l.nb == 1 ? run_few<Fp32, 1>(c, l) : l.nb == 2 ? run_few<Fp32Split, 2>(c, l) : run_few<Fp32Split, 4>(c, l);
}

template <int P, class F>
void by_shape(Shape shape, F f) {
    if (shape == BIG)
        f((Big<P>*)nullptr);
    else if (shape == MID)
        f((Mid<P>*)nullptr);
    else
        f((Small<P>*)nullptr);
}

template <typename T, int P>
int run(const Call& c) {
    using Pl = Planes<P>;
    const Layout l = layout(P, c.grad, c.T, c.V, c.H, c.e.k, c.distill);
    char* ws = c.work;
    auto floats = [&](long at) { return (float*)(ws + at); };
    int *count = (int*)(ws + l.count), *rows = (int*)(ws + l.rows), *pos = (int*)(ws + l.pos);
    float *const x_unit = floats(l.x_unit), *const x_most = floats(l.x_most), *const w_unit = floats(l.w_unit);
    const T* W = (const T*)c.W;
    const hipStream_t st = c.stream;
    const long x_pitch = Pl::pitch(l.hk), d_pitch = Pl::pitch(l.piece);
    const int slabs = l.hk / Pl::BK;
    // W is read in place when its rows are whole aligned slabs, or whole aligned quads and the products
    // are short: rows that end inside a slab, and so between two lines of memory, slow those by 8 %, and
    // packing W costs most where it is large (a bf16 step, us, packed/in place: 300 tokens, 20000 x 1000:
    // 152, 138; 1001 tokens, 50021 x 1000: 574, 529; 777 tokens, 5003 x 1000: 111, 114; 3000 tokens,
    // 8000 x 504: 188, 193)
    const bool direct = P == 1 && (c.H % Pl::BK == 0 || (c.H % 8 == 0 && (long)c.V * c.H >= 16384L * c.T)) &&
                        c.ldw % 8 == 0 && (uintptr_t)c.W % 16 == 0 && c.ldw < (1L << 22);
    const bool ends = direct && c.H % Pl::BK != 0;  // kernels of their own: the others take 2 % less time
    // dW's product takes X times each token's weight, but for bf16 distillation, whose D has it
    char* const xs = c.grad && c.dW && (P == 2 || !c.distill) ? ws + l.xs : nullptr;
    (void)hipGetLastError();

    float* const z = c.distill ? c.picked_out : floats(l.z);
    // the gradient's W is packed in one power of two, that of its largest value
    const int max_blocks = P == 2 && c.grad ? (int)(up(c.V, 4) / 4 < kMaxBlocks ? up(c.V, 4) / 4 : kMaxBlocks) : 0;
    const TokenArgs tokens = token_args(c, ws, z, l.scale, l.weight, l.value, P == 2 ? D_APART : D_PACKED);
    const int look = (int)token_blocks(c, tokens);
    const ScanArgs scan{tokens,
                        {rows, pos, count, c.grad ? nullptr : c.loss, c.lse_out},
                        look, P == 2 && xs ? floats(l.x_part) : nullptr, floats(l.w_part), max_blocks};
    const unsigned scan_blocks = 1 + look + max_blocks;
    launch_shares(c, l.keys, l.value);
    if (c.grad)
        vocab_scan_kernel<T, true><<<scan_blocks, 256, 0, st>>>(scan);
    else
        vocab_scan_kernel<T, false><<<scan_blocks, 256, 0, st>>>(scan);
    const Operand x{ws + l.x, (uint32_t)x_pitch, (uint32_t)x_pitch, l.tp};
    const Operand x_dw{xs ? xs : ws + l.x, (uint32_t)x_pitch, (uint32_t)x_pitch, l.tp};
    const Operand d{ws + l.d, (uint32_t)d_pitch, (uint32_t)d_pitch, l.tp};
    int part = 0;
    for (int p = 0; p < l.pieces; ++p) {
        const int v0 = p * l.piece, vn = c.V - v0 < l.piece ? c.V - v0 : l.piece;
        const T* Wp = W + (size_t)v0 * c.ldw;
        Operand w{(const char*)Wp, (uint32_t)(c.ldw * 2), (uint32_t)(c.H * 2), vn};
        if (!direct) w = Operand{ws + l.w, (uint32_t)x_pitch, (uint32_t)x_pitch, (int)up(vn, 256)};
        if (p == 0 || !direct) {
            const int x_blocks = p == 0 ? l.tp : 0;
            const int w_rows = pack_rows<P>(l.hk);
            const PackArgs pack{c.H, l.hk, x_pitch, c.X, c.ldx, rows, count, x_blocks, ws + l.x,
                                floats(l.weight), xs, x_unit, floats(l.x_part), look, x_most, Wp, c.ldw, vn, w_rows,
                                ws + l.w, floats(l.w_part), max_blocks, w_unit};
            const unsigned blocks = x_blocks + (direct ? 0 : (unsigned)up(vn, 256) / w_rows);
            if (P == 2 && !c.grad)
                vocab_pack_kernel<T, P, P == 2><<<blocks, 256, 0, st>>>(pack);
            else
                vocab_pack_kernel<T, P, false><<<blocks, 256, 0, st>>>(pack);
        }
        if (c.T == 0) {
            // only dW, which is 0, is left to do
        } else if (!c.grad) {
            by_shape<P>(shape_of(P, vn, c.T), [&](auto* shape) {
                using S = typename std::remove_pointer<decltype(shape)>::type;
                const int tm = (int)up(vn, S::kBM) / S::kBM, tn = (int)up(c.T, S::kBN) / S::kBN;
                const LseArgs a{w, x, count, w_unit, x_unit, tm, tn, slabs, vn, c.alpha, (float2*)(ws + l.part), part,
                                l.tp};
                if (P == 1 && ends)
                    vocab_lse_kernel<S, P == 1 ? K_ENDS : K_ROW><<<tm * tn, S::NT, 0, st>>>(a);
                else
                    vocab_lse_kernel<S, K_ROW><<<tm * tn, S::NT, 0, st>>>(a);
                part += tm * S::WAVES_M;
            });
            continue;
        } else {
            by_shape<P>(shape_of(P, vn, c.T), [&](auto* shape) {
                using S = typename std::remove_pointer<decltype(shape)>::type;
                // whole 256-row tiles of D, so that the products find zeros, not old values, past vn
                const int tm = (int)up(vn, 256) / S::kBM, tn = (int)up(c.T, S::kBN) / S::kBN;
                const GradArgs a{w, x, count, rows, w_unit, x_unit, tm, tn, slabs, vn, c.alpha, c.lse, floats(l.scale),
                                 c.distill ? nullptr : c.e.index, floats(l.value), v0, ws + l.d, d_pitch};
                if (P == 1 && ends)
                    vocab_grad_kernel<S, P == 1 ? K_ENDS : K_ROW><<<tm * tn, S::NT, 0, st>>>(a);
                else
                    vocab_grad_kernel<S, K_ROW><<<tm * tn, S::NT, 0, st>>>(a);
            });
            if (c.distill)
                vocab_patch_kernel<P><<<(unsigned)(up((long)c.T * c.e.k, 256) / 256), 256, 0, st>>>(
                    c.e, c.T, v0, vn, pos, floats(l.value), ws + l.d, d_pitch);
            if (c.dX) {
                const DxArgs a{w, d, count, w_unit, l.cut, (int)up(vn, Pl::BK) / Pl::BK, floats(l.acc), l.hp, p > 0};
                by_shape<P>(l.dx_shape, [&](auto* shape) {
                    using S = typename std::remove_pointer<decltype(shape)>::type;
                    vocab_dx_kernel<S><<<l.cut.groups, S::NT, 0, st>>>(a);
                });
            }
        }
        if (c.dW)
            by_shape<P>(shape_of(P, c.H, vn), [&](auto* shape) {
                using S = typename std::remove_pointer<decltype(shape)>::type;
                const int tm = (int)up(c.H, S::kBM) / S::kBM, tn = (int)up(vn, S::kBN) / S::kBN;
                T* out = (T*)c.dW + (size_t)v0 * c.lddw;
                const DwArgs a{x_dw, d, count, x_most, tm, tn, c.H, vn, out, c.lddw};
                vocab_dw_kernel<S><<<tm * tn, S::NT, 0, st>>>(a);
            });
    }
    if (!c.grad) {
        // fewer tokens a workgroup until every compute unit has one (100 tokens, 131072 rows: 17.6 us with
        // 32, 8.9 with 8; 2048 tokens: 10.9, 8.1)
        auto loss = [&](auto kernel, int tokens) {
            kernel<<<l.tp / tokens, 1024, 0, st>>>(c.e, rows, count, c.T, c.V, (const float2*)(ws + l.part), part, l.tp,
                                                   z, c.loss, c.lse_out);
        };
        if (c.T <= 2048)
            loss(vocab_loss_kernel<8>, 8);
        else
            loss(vocab_loss_kernel<32>, 32);
    } else if (c.T > 0 && c.dX) {
        auto out = [&](auto kernel, long cols) {
            kernel<<<dim3(c.T, (unsigned)(up(c.H, cols) / cols)), 256, 0, st>>>(
                c.e, pos, count, c.H, floats(l.acc), l.cut, l.hp, floats(l.weight), (T*)c.dX, c.lddx);
        };
        if (c.T < 512)
            out(vocab_dx_out_kernel<T, P, 16>, 64);
        else
            out(vocab_dx_out_kernel<T, P, 1>, 1024);
    }
    return (int)hipGetLastError();
}

int dispatch(const Call& c) {
    if (few(c.T)) return run_few(c);
    return c.f32 ? run<float, 2>(c) : run<__bf16, 1>(c);
}

bool sizes_ok(int T, int V, int H, int K, int& bad, const int pos[4]) {
    if (T < 0 || T > kMaxTokens) return bad = pos[0], false;
    if (V < 1 || V > kMaxRows) return bad = pos[1], false;
    if (H < 1 || H > kMaxHidden) return bad = pos[2], false;
    if (K < 1 || (long)K * T > INT_MAX) return bad = pos[3], false;
    return true;
}

// Whether two row-major matrices' spans, first to last addressed byte, meet.
bool meet(const void* a, long rows_a, long lda, const void* b, long rows_b, long ldb, long cols, long size) {
    if (!a || !b || rows_a == 0 || rows_b == 0) return false;
    const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
    return p < q + ((rows_b - 1) * ldb + cols) * size && q < p + ((rows_a - 1) * lda + cols) * size;
}
// 1: dX overlaps an input, 2: dW overlaps an input or dX.
int outputs_meet(const Call& c) {
    const long s = c.f32 ? 4 : 2;
    if (meet(c.dX, c.T, c.lddx, c.X, c.T, c.ldx, c.H, s) || meet(c.dX, c.T, c.lddx, c.W, c.V, c.ldw, c.H, s)) return 1;
    if (meet(c.dW, c.V, c.lddw, c.X, c.T, c.ldx, c.H, s) || meet(c.dW, c.V, c.lddw, c.W, c.V, c.ldw, c.H, s) ||
        meet(c.dW, c.V, c.lddw, c.dX, c.T, c.lddx, c.H, s))
        return 2;
    return 0;
}

}  // namespace
}  // namespace vocab
}  // namespace libsgemm

using libsgemm::vocab::Call;

extern "C" {

long long vocab_workspace(int dtype, int grad, int T, int V, int H, int K) {
    static const int pos[4] = {3, 4, 5, 6};
    int bad = 0;
    if (dtype != VOCAB_F32 && dtype != VOCAB_BF16) return -1;
    if (!libsgemm::vocab::sizes_ok(T, V, H, K > 0 ? K : 1, bad, pos) || K < 0) return K < 0 ? -6 : -bad;
    if (libsgemm::vocab::few(T))
        return libsgemm::vocab::few_layout(dtype == VOCAB_F32, grad != 0, T, V, H, K > 0 ? K : 1).bytes;
    return libsgemm::vocab::layout(dtype == VOCAB_F32 ? 2 : 1, grad != 0, T, V, H, K > 0 ? K : 1, K > 0).bytes;
}

int vocab_ce(int dtype, int T, int V, int H, float alpha, const void* X, int ldx, const void* W, int ldw,
             const long long* target, long long ignore_index, float* loss, float* lse, void* work,
             long long work_bytes, hipStream_t stream) {
    static const int pos[4] = {2, 3, 4, 2};
    int bad = 0;
    if (dtype != VOCAB_F32 && dtype != VOCAB_BF16) return -1;
    if (!libsgemm::vocab::sizes_ok(T, V, H, 1, bad, pos)) return -bad;
    if (ldx < H) return -7;
    if (ldw < H) return -9;
    if (T == 0) return 0;
    if (!X) return -6;
    if (!W) return -8;
    if (!target) return -10;
    if (!loss) return -12;
    if (!lse) return -13;
    if (!work || (uintptr_t)work % 16) return -14;
    if (work_bytes < vocab_workspace(dtype, 0, T, V, H, 0)) return -15;
    Call c{};
    c.f32 = dtype == VOCAB_F32;
    c.T = T, c.V = V, c.H = H, c.alpha = alpha;
    c.e = {target, 1, 1, ignore_index, nullptr, 0, 0.f};
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
    c.loss = loss, c.lse_out = lse;
    c.work = (char*)work, c.stream = stream;
    return libsgemm::vocab::dispatch(c);
}

int vocab_ce_grad(int dtype, int T, int V, int H, float alpha, const void* X, int ldx, const void* W, int ldw,
                  const long long* target, long long ignore_index, const float* lse, const float* dloss, void* dX,
                  int lddx, void* dW, int lddw, void* work, long long work_bytes, hipStream_t stream) {
    static const int pos[4] = {2, 3, 4, 2};
    int bad = 0;
    if (dtype != VOCAB_F32 && dtype != VOCAB_BF16) return -1;
    if (!libsgemm::vocab::sizes_ok(T, V, H, 1, bad, pos)) return -bad;
    if (ldx < H) return -7;
    if (ldw < H) return -9;
    if (dX && lddx < H) return -15;
    if (dW && lddw < H) return -17;
    if (!dX && !dW) return 0;
    if (T > 0) {
        if (!X) return -6;
        if (!target) return -10;
        if (!lse) return -12;
        if (!dloss) return -13;
    }
    if (!W) return -8;
    if (!work || (uintptr_t)work % 16) return -18;
    if (work_bytes < vocab_workspace(dtype, 1, T, V, H, 0)) return -19;
    Call c{};
    c.f32 = dtype == VOCAB_F32, c.grad = true;
    c.T = T, c.V = V, c.H = H, c.alpha = alpha;
    c.e = {target, 1, 1, ignore_index, nullptr, 0, 0.f};
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
    c.lse = lse, c.dloss = dloss;
    c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
    c.work = (char*)work, c.stream = stream;
    const int bad_out = libsgemm::vocab::outputs_meet(c);
    if (bad_out) return bad_out == 1 ? -14 : -16;
    return libsgemm::vocab::dispatch(c);
}

int vocab_distill(int dtype, int T, int V, int H, int K, float alpha, float teacher_alpha, const void* X, int ldx,
                  const void* W, int ldw, const long long* index, int ldi, const float* teacher, int ldt, float* loss,
                  float* lse, float* picked, void* work, long long work_bytes, hipStream_t stream) {
    static const int pos[4] = {2, 3, 4, 5};
    int bad = 0;
    if (dtype != VOCAB_F32 && dtype != VOCAB_BF16) return -1;
    if (!libsgemm::vocab::sizes_ok(T, V, H, K, bad, pos)) return -bad;
    if (ldx < H) return -9;
    if (ldw < H) return -11;
    if (ldi < K) return -13;
    if (ldt < K) return -15;
    if (T == 0) return 0;
    if (!X) return -8;
    if (!W) return -10;
    if (!index) return -12;
    if (!teacher) return -14;
    if (!loss) return -16;
    if (!lse) return -17;
    if (!picked) return -18;
    if (!work || (uintptr_t)work % 16) return -19;
    if (work_bytes < vocab_workspace(dtype, 0, T, V, H, K)) return -20;
    Call c{};
    c.f32 = dtype == VOCAB_F32;
    c.T = T, c.V = V, c.H = H, c.alpha = alpha;
    c.e = {index, ldi, K, 0, teacher, ldt, teacher_alpha}, c.distill = true;
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
    c.loss = loss, c.lse_out = lse, c.picked_out = picked;
    c.work = (char*)work, c.stream = stream;
    return libsgemm::vocab::dispatch(c);
}

int vocab_distill_grad(int dtype, int T, int V, int H, int K, float alpha, float teacher_alpha, const void* X,
                       int ldx, const void* W, int ldw, const long long* index, int ldi, const float* teacher,
                       int ldt, const float* lse, const float* picked, const float* dloss, void* dX, int lddx,
                       void* dW, int lddw, void* work, long long work_bytes, hipStream_t stream) {
    static const int pos[4] = {2, 3, 4, 5};
    int bad = 0;
    if (dtype != VOCAB_F32 && dtype != VOCAB_BF16) return -1;
    if (!libsgemm::vocab::sizes_ok(T, V, H, K, bad, pos)) return -bad;
    if (ldx < H) return -9;
    if (ldw < H) return -11;
    if (ldi < K) return -13;
    if (ldt < K) return -15;
    if (dX && lddx < H) return -20;
    if (dW && lddw < H) return -22;
    if (!dX && !dW) return 0;
    if (T > 0) {
        if (!X) return -8;
        if (!index) return -12;
        if (!teacher) return -14;
        if (!lse) return -16;
        if (!picked) return -17;
        if (!dloss) return -18;
    }
    if (!W) return -10;
    if (!work || (uintptr_t)work % 16) return -23;
    if (work_bytes < vocab_workspace(dtype, 1, T, V, H, K)) return -24;
    Call c{};
    c.f32 = dtype == VOCAB_F32, c.grad = true;
    c.T = T, c.V = V, c.H = H, c.alpha = alpha;
    c.e = {index, ldi, K, 0, teacher, ldt, teacher_alpha}, c.distill = true;
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
    c.lse = lse, c.picked = picked, c.dloss = dloss;
    c.dX = dX, c.lddx = lddx, c.dW = dW, c.lddw = lddw;
    c.work = (char*)work, c.stream = stream;
    const int bad_out = libsgemm::vocab::outputs_meet(c);
    if (bad_out) return bad_out == 1 ? -19 : -21;
    return libsgemm::vocab::dispatch(c);
}

}  // extern "C"
