// Checks of arguments that the entry points share (abi_layer.cu, abi_block.cu):
// alignment, strided views, and which memory may overlap which.  Host code only.
#pragma once

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "common.cuh"

namespace la {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_width(int d) { return d >= 16 && d <= 256 && d % 16 == 0; }

inline bool valid_dtype(la_dtype t) { return t == LA_DTYPE_F32 || t == LA_DTYPE_BF16; }

inline size_t elem_size(la_dtype t) { return t == LA_DTYPE_BF16 ? 2 : 4; }

inline la_status cuda_status(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

// A 4-D tensor whose rows of d elements are dense: three sizes and strides (elements).
struct View {
    const void* p;
    long long size[3], stride[3];
    int d;
    size_t es;

    long long row_end() const {  // elements from the first row's start to the last row's end
        long long e = d;
        for (int i = 0; i < 3; ++i) e += (size[i] - 1) * stride[i];
        return e;
    }
    size_t bytes() const { return (size_t)row_end() * es; }
};

// Elements a view may span: byte offsets then stay far inside 63 bits.
constexpr long long kMaxSpan = 1ll << 44;

// Fill in the view of p with strides as given (null: dense, the last size fastest).
// False for a null or misaligned pointer, a stride that is negative, not a multiple
// of 16 bytes, or too large.  A size of one needs no stride: it becomes 0.
inline bool make_view(View* v, const void* p, const long long* strides, long long n0, long long n1,
                      long long n2, int d, la_dtype dtype) {
    v->p = p;
    v->d = d;
    v->es = elem_size(dtype);
    v->size[0] = n0; v->size[1] = n1; v->size[2] = n2;
    const long long dense[3] = {n1 * n2 * d, n2 * d, d};
    if (!p || !aligned16(p)) return false;
    long long span = d;
    for (int i = 0; i < 3; ++i) {
        long long s = strides ? strides[i] : dense[i];
        if (v->size[i] == 1) s = 0;
        if (s < 0 || s > kMaxSpan || s * (long long)v->es % 16 != 0) return false;
        if (s > 0 && v->size[i] - 1 > (kMaxSpan - span) / s) return false;
        span += (v->size[i] - 1) * s;
        v->stride[i] = s;
    }
    return true;
}

// An output's rows must not overlap each other: taken from the smallest stride up,
// each one clears what lies inside it.
inline bool rows_apart(const View& v) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (v.stride[order[j]] < v.stride[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    long long inner = v.d;
    for (int i : order) {
        if (v.size[i] == 1) continue;
        if (v.stride[i] < inner) return false;
        inner += (v.size[i] - 1) * v.stride[i];
    }
    return true;
}

inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

inline bool overlap(const View& v, const void* b, size_t nb) { return ranges_overlap(v.p, v.bytes(), b, nb); }

// Are two views of one buffer apart modulo `period`?  Where it divides every stride that
// is not smaller, each view lies in the footprint of its smaller strides, repeated; the
// views share no element where the two footprints are apart within one period.
inline bool apart_modulo(const View& a, const View& b, long long period) {
    long long foot[2];
    for (int k = 0; k < 2; ++k) {
        const View& v = k ? b : a;
        foot[k] = v.d;
        for (int i = 0; i < 3; ++i) {
            if (v.stride[i] < period) foot[k] += (v.size[i] - 1) * v.stride[i];
            else if (v.stride[i] % period != 0) return false;
        }
    }
    const intptr_t bytes = (intptr_t)((uintptr_t)b.p - (uintptr_t)a.p);
    if (bytes % (intptr_t)a.es != 0) return false;
    long long delta = (long long)(bytes / (intptr_t)a.es) % period;
    if (delta < 0) delta += period;
    return delta >= foot[0] && delta + foot[1] <= period;
}

// Slices of a packed row may interleave without sharing an element, token by token (q's
// heads beside k's) or head by head (each head's q beside its k): apart modulo one of
// their strides.
inline bool overlap(const View& a, const View& b) {
    if (!ranges_overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
    if (a.es != b.es) return true;
    for (const View* v : {&a, &b})
        for (long long s : v->stride)
            if (s > 0 && apart_modulo(a, b, s)) return false;
    return true;
}

inline void keep(long long (&to)[3], const View& v) { std::memcpy(to, v.stride, sizeof(to)); }

struct Region {
    const void* p;
    size_t n;
};

inline bool any_misaligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (p && !aligned16(p)) return true;
    return false;
}

// Every output apart from every input and from the other outputs.
inline bool clash(std::initializer_list<Region> ins, std::initializer_list<Region> outs) {
    for (const Region* o = outs.begin(); o != outs.end(); ++o) {
        for (const Region& i : ins)
            if (ranges_overlap(o->p, o->n, i.p, i.n)) return true;
        for (const Region* o2 = o + 1; o2 != outs.end(); ++o2)
            if (ranges_overlap(o->p, o->n, o2->p, o2->n)) return true;
    }
    return false;
}

}  // namespace la
