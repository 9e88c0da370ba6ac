// tdg_check.h -- argument checks shared by the operators whose rows pick
// their weights (routed rows, grouped products, adapters).  Nothing here
// calls HIP.
#pragma once

#include <stdint.h>

namespace tdg {

// Largest rows, columns or k: the kernels form (tile start + tile extent) on
// 32-bit indices, so every size keeps a margin of 2^16 below 2^31.
constexpr int64_t kMaxSize = ((int64_t)1 << 31) - ((int64_t)1 << 16);

inline bool size_ok(int64_t n) { return n >= 0 && n <= kMaxSize; }

// A row-major rows x cols matrix of `es`-byte elements: leading dimension at
// least max(1, cols), a pointer unless it is empty, its bytes within int64.
inline bool matrix_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
    if (ld < (cols > 1 ? cols : 1)) return false;
    if (rows > 0 && ld > INT64_MAX / es / rows) return false;
    return p || rows == 0 || cols == 0;
}

// `count` such matrices, `stride` elements apart (rows * ld fits: checked
// before).  Matrices that share memory are refused when `apart` (outputs).
inline bool stack_ok(const void *p, int64_t count, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                     int64_t es, bool apart) {
    if (!matrix_ok(count > 0 ? p : (const void *)1, rows, cols, ld, es)) return false;
    if (count <= 1) return true;
    if (stride < 0 || stride > INT64_MAX / es / 2 / count) return false;
    return !apart || rows == 0 || cols == 0 || stride >= (rows - 1) * ld + cols;
}

// Bytes from a matrix's (or a stack's) first element through its last.
inline uint64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t es, int64_t count = 1,
                           int64_t stride = 0) {
    if (rows <= 0 || cols <= 0 || count <= 0) return 0;
    return (uint64_t)((count - 1) * stride + (rows - 1) * ld + cols) * (uint64_t)es;
}

inline bool overlaps(const void *a, uint64_t alen, const void *b, uint64_t blen) {
    if (!a || !b || !alen || !blen) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + blen && y < x + alen;
}

inline bool aligned_to(const void *p, uintptr_t bytes) { return (uintptr_t)p % bytes == 0; }

// Chunks of 16 bytes sit on a 16-byte grid from each row's start, and the last
// one of a matrix, whose last row (`cols` 2-byte elements) is at `row`, can reach
// past its last element.  Where it would reach into another 4 KiB page, which
// need not be mapped: that page's address, so that the kernels load what they
// need of it element by element.  kNoStop: nowhere.  (The kernels call it too.)
constexpr uint64_t kNoStop = ~(uint64_t)0;
constexpr uint64_t page_stop(uint64_t row, int64_t cols) {
    const uint64_t last = row + (uint64_t)cols * 2 - 1, end = row + (uint64_t)((cols - 1) / 8 * 16 + 15);
    return last >> 12 == end >> 12 ? kNoStop : ((last >> 12) + 1) << 12;
}

// The same of a matrix, or of the last of a stack.
inline uint64_t chunk_stop(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t count = 1,
                           int64_t stride = 0) {
    if (rows <= 0 || cols <= 0 || count <= 0) return kNoStop;
    return page_stop((uint64_t)(uintptr_t)p + (uint64_t)((count - 1) * stride + (rows - 1) * ld) * 2, cols);
}

// Whether a stack's matrices need a stop each: their last chunks can reach past
// them, into a page that neither they nor the next matrix has a byte of.  (Where
// the next one begins less than a page behind, it has.)
inline bool stops_each(int64_t rows, int64_t cols, int64_t ld, int64_t count, int64_t stride) {
    if (rows <= 0 || cols <= 0 || count <= 1 || cols % 8 == 0) return false;
    return stride - ((rows - 1) * ld + cols) >= 2048;
}

inline int64_t ceil_quot(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace tdg
