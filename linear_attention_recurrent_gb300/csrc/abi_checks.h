// abi_checks.h -- checks of tensor descriptors that the entry points around the
// recurrent state decode share.  Host code only.
#pragma once

#include <stdint.h>

#include "lar.h"

namespace lar {

inline bool is_float(const lar_tensor* t) { return t->dtype == LAR_F32 || t->dtype == LAR_BF16; }
inline bool is_index(const lar_tensor* t) { return t->dtype == LAR_I32 || t->dtype == LAR_I64; }
inline int64_t elem_size(int32_t dt) { return dt == LAR_E4M3 ? 1 : dt == LAR_BF16 ? 2 : dt == LAR_I64 ? 8 : 4; }

inline bool empty(const lar_tensor* t) {
    for (int i = 0; i < t->ndim && i < 5; ++i)
        if (t->shape[i] == 0) return true;
    return false;
}

// Rank in [lo, hi], non-negative sizes and strides, a pointer (unless empty) that is
// aligned to the elements.
inline lar_status check(const lar_tensor* t, int lo, int hi, bool index) {
    if (!t) return LAR_ERR_NULL;
    if (t->ndim < 1 || t->ndim > 5 || t->ndim < lo || t->ndim > hi) return LAR_ERR_RANK;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] < 0) return LAR_ERR_SHAPE;
        if (t->stride[i] < 0) return LAR_ERR_STRIDE;
    }
    if (!t->data && !empty(t)) return LAR_ERR_NULL;
    if (index ? !is_index(t) : !is_float(t)) return LAR_ERR_DTYPE;
    if (reinterpret_cast<uintptr_t>(t->data) % elem_size(t->dtype)) return LAR_ERR_ALIGN;
    return LAR_OK;
}

#define LAR_TRY(expr)                                  \
    do {                                               \
        const lar_status st_ = (expr);                 \
        if (st_ != LAR_OK) return st_;                 \
    } while (0)

// Half-open byte range that a view can touch.
struct Range {
    uintptr_t lo = 0, hi = 0;
};

inline Range range_of(const lar_tensor* t) {
    Range r;
    if (!t || !t->data || empty(t)) return r;
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) last += (t->shape[i] - 1) * t->stride[i];
    r.lo = reinterpret_cast<uintptr_t>(t->data);
    r.hi = r.lo + static_cast<uintptr_t>((last + 1) * elem_size(t->dtype));
    return r;
}

inline bool meet(const Range& a, const Range& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// Outputs (the error word among them) clear of one another and of every input.
inline lar_status check_aliasing(const lar_tensor* const* outs, int n_out, const lar_tensor* const* ins, int n_in,
                          const int32_t* dev_err) {
    Range e;
    if (dev_err) {
        e.lo = reinterpret_cast<uintptr_t>(dev_err);
        e.hi = e.lo + sizeof(int32_t);
        if (e.lo % alignof(int32_t) != 0) return LAR_ERR_ALIGN;
    }
    for (int i = 0; i < n_out; ++i) {
        const Range a = range_of(outs[i]);
        if (meet(a, e)) return LAR_ERR_ALIAS;
        for (int j = i + 1; j < n_out; ++j)
            if (meet(a, range_of(outs[j]))) return LAR_ERR_ALIAS;
        for (int j = 0; j < n_in; ++j)
            if (meet(a, range_of(ins[j]))) return LAR_ERR_ALIAS;
    }
    for (int j = 0; j < n_in; ++j)
        if (meet(e, range_of(ins[j]))) return LAR_ERR_ALIAS;
    return LAR_OK;
}

// Two elements of an output at one address would be written by two threads:
// strides, taken from the smallest, step over everything that the smaller ones reach.
inline bool overlaps_itself(const lar_tensor* t) {
    if (empty(t)) return false;
    bool used[5] = {false, false, false, false, false};
    int64_t reach = 0;
    for (int k = 0; k < t->ndim; ++k) {
        int best = -1;
        for (int i = 0; i < t->ndim; ++i)
            if (!used[i] && (best < 0 || t->stride[i] < t->stride[best] ||
                             (t->stride[i] == t->stride[best] && t->shape[i] < t->shape[best])))
                best = i;
        used[best] = true;
        if (t->shape[best] == 1) continue;
        if (t->stride[best] <= reach) return true;
        reach += (t->shape[best] - 1) * t->stride[best];
    }
    return false;
}

// Strides (sequence, token, rest...) of a per-token tensor: [B, T, rest...], or
// [B, rest...] with T = 1, or packed [tokens, rest...].  `rest` sizes in r[0..nr).
inline lar_status token_view(const lar_tensor* t, bool packed, int64_t B, int64_t T, const int64_t* r, int nr, int64_t* st) {
    const int64_t lead[2] = {B, T};
    const int nl = packed || t->ndim == 1 + nr ? 1 : 2;
    if (t->ndim != nl + nr) return LAR_ERR_RANK;
    if (!packed && nl == 1 && T != 1) return LAR_ERR_RANK;
    if (packed) {
        if (t->shape[0] != T) return LAR_ERR_SHAPE;
        st[0] = 0;
        st[1] = t->stride[0];
    } else {
        for (int i = 0; i < nl; ++i)
            if (t->shape[i] != lead[i]) return LAR_ERR_SHAPE;
        st[0] = t->stride[0];
        st[1] = nl == 2 ? t->stride[1] : 0;
    }
    for (int i = 0; i < nr; ++i) {
        if (t->shape[nl + i] != r[i]) return LAR_ERR_SHAPE;
        st[2 + i] = t->stride[nl + i];
    }
    return LAR_OK;
}

// A [n] vector; index vectors and float vectors alike.
inline lar_status vec_view(const lar_tensor* t, int64_t n, bool index, const void** data, int64_t* stride, int* dt) {
    LAR_TRY(check(t, 1, 1, index));
    if (t->shape[0] != n) return LAR_ERR_SHAPE;
    *data = t->data;
    *stride = t->stride[0];
    *dt = t->dtype;
    return LAR_OK;
}

inline lar_status f32_vec(const lar_tensor* t, int64_t n, const float** data, int64_t* stride) {
    int dt;
    const void* d;
    LAR_TRY(vec_view(t, n, false, &d, stride, &dt));
    if (dt != LAR_F32) return LAR_ERR_DTYPE;
    *data = static_cast<const float*>(d);
    return LAR_OK;
}

// 16-byte accesses of 8 neighbouring channels fit a [.., C] view: channel
// stride 1, aligned base, every other stride a multiple of 16 bytes.
inline bool vec8(const void* data, int dt, const int64_t* st, int n_lead, int64_t c_stride) {
    const int64_t es = elem_size(dt);
    if (c_stride != 1 || reinterpret_cast<uintptr_t>(data) % 16) return false;
    for (int i = 0; i < n_lead; ++i)
        if ((st[i] * es) % 16) return false;
    return true;
}

}  // namespace lar
