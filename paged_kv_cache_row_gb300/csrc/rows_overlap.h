// rows_overlap.h -- whether two sets of token rows share memory.
//
// Plain C++ without CUDA, so that the tests compile it for the host and compare
// it with a look at every byte.
#pragma once
#include <cstdint>

namespace minisgl {

// Whether [a, a + na) and [b, b + nb) (in bytes) share memory.
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// n >= 1 rows of `row` bytes, `stride` >= row bytes apart.
struct Rows {
    const void *base;
    int64_t row, stride;
    int64_t span(int64_t n) const { return (n - 1) * stride + row; }
};

// Whether any of n rows of a shares memory with any of n rows of b.  Rows that
// lie between one another's (slices of one projection's output) do not.
inline bool rows_overlap(const Rows &a, const Rows &b, int64_t n) {
    if (!overlap(a.base, a.span(n), b.base, b.span(n))) return false;
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
    if (a.stride == b.stride) {
        // b's row i + k begins `after` bytes (below a stride) behind where a's row i begins
        const int64_t after = (off % a.stride + a.stride) % a.stride, k = (after - off) / a.stride;
        return (after < a.row && k > -n && k < n) || (a.stride - after < b.row && k - 1 > -n && k - 1 < n);
    }
    for (int64_t i = 0; i < n; ++i) {
        const int64_t at = i * a.stride - off;                              // a's row, from b's first
        const int64_t j = at < b.row ? 0 : (at - b.row) / b.stride + 1;     // b's first row that ends behind it
        if (j >= n) break;
        if (j * b.stride < at + a.row) return true;
    }
    return false;
}

}  // namespace minisgl
