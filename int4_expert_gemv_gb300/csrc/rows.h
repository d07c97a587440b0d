// rows.h -- arrays of rows as the calls are given them, and whether two of
// them share memory.
#pragma once

#include <cstddef>
#include <cstdint>

#include "common.cuh"

namespace moe {

struct Rows {                            // n rows of `width` bytes, `stride` bytes apart
    const char *name;
    const void *at;
    size_t n, width, stride;

    bool same(const Rows &o) const { return at == o.at && width == o.width && (n <= 1 || stride == o.stride); }

    // Whether a byte belongs to both.  Rows of one stride may lie between each
    // other's (parts of one projection); of different strides, the spans from
    // the first byte to the last count.
    bool overlaps(const Rows &o) const {
        if (!at || !o.at || !n || !o.n || !width || !o.width) return false;
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(o.at);
        const size_t la = (n - 1) * stride + width, lb = (o.n - 1) * o.stride + o.width;
        if (a >= b + lb || b >= a + la) return false;
        if (stride != o.stride || n == 1 || o.n == 1 || width > stride || o.width > stride) return true;
        const size_t off = a >= b ? (a - b) % stride : (stride - (b - a) % stride) % stride;   // of a's rows in b's
        return off < o.width || off + width > stride;
    }
};

inline bool off(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline size_t bytes_of(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : dtype == MOE_DTYPE_BF16 ? 2 : 1; }

// Rows on `align`-byte boundaries; the stride of a single row does not matter.
inline int check_rows(const char *who, const Rows &r, size_t align = 16) {
    if (!r.at || off(r.at, align)) return fail(MOE_EINVAL, "%s: NULL or misaligned %s", who, r.name);
    if (r.n > 1 && (r.stride < r.width || r.stride % align || r.stride > (SIZE_MAX >> 1) / r.n))
        return fail(MOE_EINVAL, "%s: rows of %s %zu bytes apart (need >= %zu, a multiple of %zu)", who, r.name, r.stride, r.width, align);
    return MOE_OK;
}

}  // namespace moe
