// grads.hip -- entry points of the gradients' norm and clipping: argument checks, workspace, launches.
#include <algorithm>
#include <memory>
#include <new>

#include "../../include/grads.h"
#include "kernel_grads.hpp"

namespace libsgemm {
namespace grads {
namespace {

constexpr int kMaxTensors = 1 << 20;
constexpr long kMaxElements = 1L << 40;

long size_of(const GradTensor& t) { return t.dtype == GRADS_F32 ? 4 : 2; }
bool empty(const GradTensor& t) { return t.rows == 0 || t.cols == 0; }

bool sizes_ok(const GradTensor& t) {
    if (t.dtype != GRADS_F32 && t.dtype != GRADS_BF16) return false;
    if (t.rows < 0 || t.rows >= 1L << 31 || t.cols < 0 || t.cols > kMaxElements) return false;
    if (t.rows > 1 && (t.ld < t.cols || t.ld >= 1L << 31)) return false;
    return t.rows == 0 || t.cols <= kMaxElements / t.rows;
}

// Elements of a workgroup's piece: 8 KB where the gradients are few, so that all compute units have some, up to
// 64 KB of bf16 where they are many.
long piece_size(int count, const GradTensor* t, long& pieces) {
    long elements = 0;
    for (int i = 0; i < count; ++i) elements += t[i].rows * t[i].cols;
    long piece = 4096;
    while (piece < 32768 && elements / piece > 4096) piece *= 2;
    while (true) {
        pieces = 0;
        for (int i = 0; i < count; ++i) pieces += pieces_of(t[i].rows, t[i].cols, piece);
        if (pieces < 1L << 24) return piece;
        piece *= 2;  // 2^24 workgroups of 256 threads are the most that a grid holds
        if (piece > 1L << 30) return 0;
    }
}

// The workspace: byte offsets of its arrays.
struct Layout {
    long piece, pieces, entries, tensor_of, sums, bytes;
};
Layout layout(int count, const GradTensor* t) {
    Layout l{};
    l.piece = piece_size(count, t, l.pieces);
    auto up = [](long x) { return (x + 255) / 256 * 256; };
    l.entries = 256;  // the factor stands before them
    l.tensor_of = l.entries + up((long)sizeof(Entry) * count);
    l.sums = l.tensor_of + up(4 * l.pieces);
    l.bytes = l.sums + 8 * l.pieces;
    return l;
}

int launch(int count, const GradTensor* tensors, bool clip, float max_norm, float eps, float* norm, char* work,
           hipStream_t stream) {
    (void)hipGetLastError();
    const Layout l = layout(count, tensors);
    double* const sums = (double*)(work + l.sums);
    float* const factor = clip ? (float*)work : nullptr;
    Entry* const entries = (Entry*)(work + l.entries);
    uint32_t* const tensor_of = (uint32_t*)(work + l.tensor_of);
    long first = 0;
    uint32_t sent = 0;
    for (int i = 0; i < count;) {
        Table t;
        uint32_t n = 0;
        for (; i < count && n < kTable; ++i) {
            const GradTensor& g = tensors[i];
            if (empty(g)) continue;
            const long own = pieces_of(g.rows, g.cols, l.piece);
            t.e[n++] = {g.x, g.out, (long)g.cols, (uint32_t)g.rows, (uint32_t)g.ld, (uint32_t)g.ld_out, (uint32_t)first,
                        (uint32_t)own, g.dtype == GRADS_BF16};
            first += own;
        }
        if (n > 0) grads_table_kernel<<<n, 256, 0, stream>>>(t, sent, entries, tensor_of);
        sent += n;
    }
    if (l.pieces > 0) grads_squares_kernel<<<(unsigned)l.pieces, 256, 0, stream>>>(entries, tensor_of, (uint32_t)l.piece, sums);
    grads_norm_kernel<<<1, 1024, 0, stream>>>(sums, l.pieces, norm, factor, max_norm, eps);
    if (clip && l.pieces > 0)
        grads_scale_kernel<<<(unsigned)l.pieces, 256, 0, stream>>>(entries, tensor_of, (uint32_t)l.piece, factor);
    return (int)hipGetLastError();
}

struct Span {
    uintptr_t from, to;
    int index;
};
Span span(const void* p, const GradTensor& t, long ld, int i) {
    return {(uintptr_t)p, (uintptr_t)p + ((t.rows - 1) * ld + t.cols) * size_of(t), i};
}

// Whether an out overlaps a tensor other than its own, or another out.
bool outs_meet(int count, const GradTensor* t, bool& no_memory) {
    std::unique_ptr<Span[]> outs(new (std::nothrow) Span[count + 1]);
    no_memory = !outs;
    if (no_memory) return false;
    int n = 0;
    for (int i = 0; i < count; ++i)
        if (!empty(t[i])) outs[n++] = span(t[i].out, t[i], t[i].ld_out, i);
    std::sort(outs.get(), outs.get() + n, [](const Span& a, const Span& b) { return a.from < b.from; });
    for (int i = 1; i < n; ++i)
        if (outs[i].from < outs[i - 1].to) return true;
    for (int i = 0; i < count; ++i) {
        if (empty(t[i])) continue;
        const Span x = span(t[i].x, t[i], t[i].ld, i);
        // the outs are disjoint and in order: those that end behind x's start
        const Span* o = std::upper_bound(outs.get(), outs.get() + n, x.from, [](uintptr_t v, const Span& s) { return v < s.to; });
        for (; o != outs.get() + n && o->from < x.to; ++o)
            if (o->index != i || t[i].out != t[i].x || (t[i].rows > 1 && t[i].ld != t[i].ld_out)) return true;
    }
    return false;
}

int run(int count, const GradTensor* t, bool clip, float max_norm, float eps, float* norm, void* work,
        long long work_bytes, hipStream_t stream, const int pos[3]) {
    const long need = grad_workspace(count, t);
    if (need < 0) return (int)need;
    if (clip && !(max_norm >= 0.f)) return -3;
    if (clip && !(eps >= 0.f)) return -4;
    for (int i = 0; i < count; ++i) {
        if (empty(t[i])) continue;
        if (!t[i].x || (uintptr_t)t[i].x % size_of(t[i])) return -2;
        if (!clip) continue;
        if (!t[i].out || (uintptr_t)t[i].out % size_of(t[i])) return -2;
        if (t[i].rows > 1 && (t[i].ld_out < t[i].cols || t[i].ld_out >= 1L << 31)) return -2;
    }
    if (!norm) return -pos[0];
    if (!work || (uintptr_t)work % 16) return -pos[1];
    if (work_bytes < need) return -pos[2];
    bool no_memory = false;
    if (clip && outs_meet(count, t, no_memory)) return -2;
    if (no_memory) return (int)hipErrorOutOfMemory;
    return launch(count, t, clip, max_norm, eps, norm, (char*)work, stream);
}

}  // namespace
}  // namespace grads
}  // namespace libsgemm

extern "C" {

long long grad_workspace(int count, const GradTensor* tensors) {
    using namespace libsgemm::grads;
    if (count < 0 || count > kMaxTensors) return -1;
    if (count > 0 && !tensors) return -2;
    for (int i = 0; i < count; ++i)
        if (!sizes_ok(tensors[i])) return -2;
    const Layout l = layout(count, tensors);
    return l.piece == 0 ? -2 : l.bytes;
}

int grad_norm(int count, const GradTensor* tensors, float* norm, void* work, long long work_bytes, hipStream_t stream) {
    static const int pos[3] = {3, 4, 5};
    return libsgemm::grads::run(count, tensors, false, 0.f, 0.f, norm, work, work_bytes, stream, pos);
}

int clip_grad_norm(int count, const GradTensor* tensors, float max_norm, float eps, float* norm, void* work,
                   long long work_bytes, hipStream_t stream) {
    static const int pos[3] = {5, 6, 7};
    return libsgemm::grads::run(count, tensors, true, max_norm, eps, norm, work, work_bytes, stream, pos);
}

}  // extern "C"
