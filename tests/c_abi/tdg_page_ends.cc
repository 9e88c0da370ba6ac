// The rule that keeps the products' 16-byte reads inside their operands' pages
// (csrc/tdg_check.h: page_stop, chunk_stop, stops_each), against every read of
// stacks of small matrices.  Host only; the addresses are made up.
#include <stdint.h>
#include <stdio.h>

#include <random>
#include <set>

#include "tdg_check.h"

using namespace tdg;

// Reads of 16-byte pieces that leave the pages of the matrices' own bytes, where
// pieces that end past their matrix's stop are not read whole.
static long outside(uint64_t p, int64_t rows, int64_t cols, int64_t ld, int64_t count, int64_t stride, bool each) {
    std::set<uint64_t> pages;
    for (int64_t g = 0; g < count; g++) {
        const uint64_t first = p + g * stride * 2, last = first + ((rows - 1) * ld + cols) * 2 - 1;
        for (uint64_t page = first >> 12; page <= last >> 12; page++) pages.insert(page);
    }
    const uint64_t whole = chunk_stop((const void *)p, rows, cols, ld, count, stride);
    long bad = 0;
    for (int64_t g = 0; g < count; g++) {
        const uint64_t at = p + g * stride * 2;
        const uint64_t stop = each ? page_stop(at + (rows - 1) * ld * 2, cols) : whole;
        for (int64_t r = 0; r < rows; r++)
            for (int64_t c = 0; c < cols; c += 8) {
                const uint64_t piece = at + (r * ld + c) * 2;
                if (piece + 16 <= stop && !(pages.count(piece >> 12) && pages.count((piece + 15) >> 12))) bad++;
            }
    }
    return bad;
}

int main() {
    std::mt19937_64 rng(5);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    long cases = 0, apart = 0, one_stop_leaves = 0;
    for (int i = 0; i < 200000; i++) {
        const int64_t rows = pick(1, 12), cols = pick(1, 40), ld = cols + pick(0, 1) * pick(0, 12), count = pick(1, 5);
        const int64_t span = (rows - 1) * ld + cols;
        // apart by anything, or so that a page ends with (or near) each matrix
        int64_t stride = span + pick(0, 2) * pick(0, 3000);
        if (pick(0, 2) == 0) stride = (span + 2047) / 2048 * 2048 + 2048 * pick(0, 2);
        uint64_t p = ((uint64_t)1 << 40) + 2 * pick(0, 4096);
        if (pick(0, 1)) p = ((uint64_t)1 << 40) + (1 << 20) - span * 2 + 2 * pick(-8, 8);
        const bool each = stops_each(rows, cols, ld, count, stride);
        if (const long bad = outside(p, rows, cols, ld, count, stride, each)) {
            printf("%ld reads leave: p %llx rows %ld cols %ld ld %ld count %ld stride %ld\n", bad, (unsigned long long)p,
                   (long)rows, (long)cols, (long)ld, (long)count, (long)stride);
            return 1;
        }
        cases++;
        apart += each;
        one_stop_leaves += each && outside(p, rows, cols, ld, count, stride, false) > 0;
    }
    // the cases that need it are among those drawn
    if (apart < 1000 || one_stop_leaves < 100) return 2;
    printf("page ends passed: %ld cases, %ld with a stop each, %ld that one stop would not keep in\n", cases, apart,
           one_stop_leaves);
    return 0;
}
