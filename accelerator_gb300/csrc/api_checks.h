// api_checks.h -- what the argument checks of the C entry points share.
#pragma once

#include <cstdint>

#include "gemm.h"

namespace libgemm {

constexpr int64_t kIndexMax = 0x7FFFFFFF;          // sizes held in 32 bits, grids
constexpr int64_t kElemMax = INT64_MAX / 64;

inline bool type_ok(int type) { return type == GEMM_TYPE_F32 || type == GEMM_TYPE_BF16 || type == GEMM_TYPE_F16; }
inline int64_t type_size(int type) { return type == GEMM_TYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }

inline bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return abytes > 0 && bbytes > 0 && x < y + (uint64_t)bbytes && y < x + (uint64_t)abytes;
}

// Bytes spanned by rows x cols elements of row stride ld.
inline int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

inline bool strides_ok(int64_t rows, int64_t heads, int64_t row, int64_t head) {
    return row >= 0 && head >= 0 && row <= kElemMax / 4 / (rows > 0 ? rows : 1) && head <= kElemMax / 4 / heads;
}

inline int64_t rows_span(int64_t rows, int64_t heads, int64_t dim, int64_t row, int64_t head, int64_t es) {
    return rows > 0 ? ((rows - 1) * row + (heads - 1) * head + dim) * es : 0;
}

// Whether two elements of rows x heads x dim with these strides are one: a
// result that many threads write has to have a place for each.
inline bool overlap_within(int64_t rows, int64_t heads, int64_t dim, int64_t row, int64_t head) {
    if ((rows > 1 && row < dim) || (heads > 1 && head < dim)) return true;
    if (rows <= 1 || heads <= 1 || row >= (heads - 1) * head + dim || head >= (rows - 1) * row + dim) return false;
    for (int64_t h = 1; h < heads; ++h) {   // neither lies inside the other: h heads on as far as r rows on, or nearly?
        const int64_t below = h * head / row;
        for (int64_t r = below > 0 ? below : 1; r <= below + 1 && r < rows; ++r)
            if (r * row - h * head < dim && h * head - r * row < dim) return true;
    }
    return false;
}

// Whether two sets of rows (a and b, each rows of heads x dim elements of es
// bytes) surely have no byte in common: apart as a whole, or slices of one array
// whose rows, or whose heads, lie between each other's.
inline bool rows_apart(const void* a, int64_t a_row, int64_t a_head, int64_t a_heads, const void* b, int64_t b_row, int64_t b_head,
                       int64_t b_heads, int64_t rows, int64_t dim, int64_t es) {
    if (!overlap(a, rows_span(rows, a_heads, dim, a_row, a_head, es), b, rows_span(rows, b_heads, dim, b_row, b_head, es))) return true;
    if (a_row == b_row && a_head == b_head && a_head > 0 && a_row % a_head == 0) {   // likewise within each head's place
        const int64_t step = a_head * es, apart = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
        const int64_t from = (apart % step + step) % step;
        if (from >= dim * es && from + dim * es <= step) return true;
    }
    const int64_t a_width = rows_span(1, a_heads, dim, a_row, a_head, es), b_width = rows_span(1, b_heads, dim, b_row, b_head, es);
    const int64_t step = a_row * es;
    if (a_row != b_row || step <= 0) return false;
    const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const int64_t from = (apart % step + step) % step;   // b's rows begin so far behind a's
    return from >= a_width && from + b_width <= step;
}

}  // namespace libgemm
