// What the host entry points share: arrays and their overlaps, the checks of a call's arguments.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "block_kernels.h"
#include "ssdc_kernels.h"

namespace ssdc {
namespace block {

constexpr int64_t kBig = int64_t(1) << 40;  // most elements of one array

// SSDC_OK where the current device is one the kernels are built for.
int check_device();

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline size_t type_bytes(int type) { return type == SSD_TYPE_F32 ? 4 : type == SSD_TYPE_BF16 ? 2 : 1; }

// A three-level array: `outer` rows of `mid` rows of `inner` contiguous elements. Dense
// arrays and rows are special cases. lo, hi: the bytes it spans.
struct Array {
    const void* p;
    int64_t outer, mid, inner, s_outer, s_mid;
    size_t elem;
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const {
        return lo() + (uintptr_t)((outer - 1) * s_outer + (mid - 1) * s_mid + inner) * elem;
    }
    bool operator==(const Array& o) const {
        return p == o.p && s_outer == o.s_outer && s_mid == o.s_mid && elem == o.elem;
    }
};

// A stride that is never taken may be anything (the row stride of a single row): it counts as zero.
inline int64_t taken(int64_t stride, int64_t count) { return count > 1 ? stride : 0; }

inline Array rows(const void* p, int64_t ld, int64_t M, int64_t D, size_t elem) { return Array{p, 1, M, D, 0, taken(ld, M), elem}; }
inline Array dense(const void* p, int64_t n, size_t elem = 4) { return Array{p, 1, 1, n, 0, 0, elem}; }

// Whether two arrays may share a byte. Arrays whose spans meet are still apart where they
// have the same strides and element size and, in every period of the smaller stride, their
// columns are apart (slices of one wider array) or, in every period of the larger one, the
// blocks below it are (planes of one array for each sequence).
inline bool overlaps(const Array& a, const Array& b) {
    if (a.p == nullptr || b.p == nullptr || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (a.elem != b.elem || a.s_mid != b.s_mid || (a.s_outer != b.s_outer && a.outer > 1)) return true;
    const uintptr_t d = a.lo() > b.lo() ? a.lo() - b.lo() : b.lo() - a.lo();
    if (d % a.elem) return true;
    const bool a_after = a.lo() > b.lo();
    // apart: whether the later array's `second` elements lie after the earlier one's `first` in every period of `step`
    auto apart = [&](int64_t step, int64_t first, int64_t second) {
        const int64_t off = (int64_t)(d / a.elem) % step;
        return off >= first && off + second <= step;
    };
    const Array &early = a_after ? b : a, &late = a_after ? a : b;
    // the larger stride, if there are two
    if (a.outer > 1 && a.mid > 1) {
        const bool outer = a.s_outer >= a.s_mid;
        const int64_t step = outer ? a.s_outer : a.s_mid;
        auto block = [&](const Array& r) { return (outer ? (r.mid - 1) * r.s_mid : (r.outer - 1) * r.s_outer) + r.inner; };
        if (step > 0 && apart(step, block(early), block(late))) return false;
    }
    // the smaller stride; every other stride has to be a multiple of it
    int64_t step = a.mid > 1 ? a.s_mid : 0;
    if (a.outer > 1 && (step == 0 || a.s_outer < step)) step = a.s_outer;
    if (step <= 0 || (a.mid > 1 && a.s_mid % step) || (a.outer > 1 && a.s_outer % step)) return true;
    return !apart(step, early.inner, late.inner);
}

// An output's rows must be apart from each other.
inline bool self_apart(const Array& a) {
    const bool m = a.mid > 1, o = a.outer > 1;
    if (m && a.s_mid < a.inner) return false;
    if (o && a.s_outer < a.inner) return false;
    if (!m || !o) return true;
    return a.s_outer >= (a.mid - 1) * a.s_mid + a.inner || a.s_mid >= (a.outer - 1) * a.s_outer + a.inner;
}

inline bool in_range(const Array& a) {
    return a.s_outer >= 0 && a.s_mid >= 0 && a.s_outer <= kBig && a.s_mid <= kBig &&
           (double)(a.outer - 1) * (double)a.s_outer + (double)(a.mid - 1) * (double)a.s_mid + (double)a.inner <=
               (double)kBig;
}

// Inputs, outputs and the pairs that may be one array (an output updated in place).
struct Args {
    Array in[10], out[6];
    int n_in = 0, n_out = 0;
    int rc = SSDC_OK;
    void fail(int code) {
        if (rc == SSDC_OK) rc = code;
    }
    void check(const Array& a) {
        if (!in_range(a)) return fail(SSDC_ERR_INVALID);
        if (!aligned_to(a.p, a.elem)) fail(SSDC_ERR_ALIGN);
    }
    void input(const Array& a, bool needed = true) {
        if (a.p == nullptr) {
            if (needed) fail(SSDC_ERR_INVALID);
            return;
        }
        check(a);
        in[n_in++] = a;
    }
    // same: an input that this output may be
    void output(const Array& a, bool needed = true, const void* same1 = nullptr, const void* same2 = nullptr) {
        if (a.p == nullptr) {
            if (needed) fail(SSDC_ERR_INVALID);
            return;
        }
        check(a);
        if (rc != SSDC_OK) return;
        if (!self_apart(a)) return fail(SSDC_ERR_INVALID);
        for (int k = 0; k < n_in; ++k) {
            const bool same = (same1 != nullptr && in[k].p == same1) || (same2 != nullptr && in[k].p == same2);
            if (!(same && in[k] == a) && overlaps(a, in[k])) return fail(SSDC_ERR_INVALID);
        }
        for (int k = 0; k < n_out; ++k)
            if (overlaps(a, out[k])) return fail(SSDC_ERR_INVALID);
        out[n_out++] = a;
    }
};

inline int done(int launches) {
    if (launches < 0) return launches;
    if (cudaGetLastError() != cudaSuccess) return SSDC_ERR_CUDA;
    ssdc::set_last_launch_count(launches);
    return SSDC_OK;
}

inline int64_t groups(int64_t n) { return (n + SSD_FP8_GROUP - 1) / SSD_FP8_GROUP; }

// The row stride that a kernel is given: that of a single row as tensor maps want it, a whole number
// of 16-byte units that holds the row.
inline int64_t row_stride(int64_t ld, int64_t count, int64_t cols, size_t elem) {
    const int64_t unit = 16 / (int64_t)elem;
    return count > 1 ? ld : (cols + unit - 1) / unit * unit;
}

// Rows of 8-bit values: a whole number of 16-byte units, as the copies into shared memory need.
inline int check_fp8_rows(const void* p, int64_t ld, int64_t count, int64_t cols) {
    if (p == nullptr) return SSDC_OK;
    if (count > 1 && ld < cols) return SSDC_ERR_INVALID;
    if (taken(ld, count) % 16 != 0 || !aligned_to(p, 16)) return SSDC_ERR_ALIGN;
    return SSDC_OK;
}

}  // namespace block
}  // namespace ssdc
