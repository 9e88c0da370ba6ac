// Rows that a grid does not hold, taken one piece after the other
// (csrc/tdg_check.h: grid_dim, next_start): every piece of 16 or 32 rows is
// taken once and none lies outside, up to the largest number of rows.  Host
// only, with signed overflow trapped.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "tdg_check.h"

using namespace tdg;

// Pieces taken by all workgroups; -1 where one starts outside [0, rows).
static int64_t taken(int64_t rows, int height) {
    const int grid = (int)grid_dim(ceil_quot(rows, height)), step = grid * height, end = (int)rows;
    int64_t n = 0;
    for (int z = 0; z < grid; z++) {
        int turn = 0;
        for (int at = z * height; at < end; at = next_start(at, end, step), turn++, n++)
            if (at < 0 || at != z * (int64_t)height + turn * (int64_t)step) return -1;
    }
    return n;
}

int main() {
    const int64_t sizes[] = {0, 1, 15, 16, 17, 33, 65535 * 16 - 1, 65535 * 16, 65535 * 16 + 1, 65535 * 32 + 1,
                             5000000, ((int64_t)1 << 31) - 65535 * 32 - 1, 2145386528, 2145386529, kMaxSize - 1,
                             kMaxSize};
    for (const int height : {16, 32})
        for (const int64_t rows : sizes)
            if (const int64_t n = taken(rows, height); n != ceil_quot(rows, height)) {
                printf("%ld rows, %d to a piece: %ld pieces of %ld\n", (long)rows, height, (long)n,
                       (long)ceil_quot(rows, height));
                return 1;
            }
    // any start and step: never past the end, never past 2^31
    for (const int end : {1, 100, (int)kMaxSize, INT32_MAX})
        for (const int step : {1, 31, 65535 * 32, INT32_MAX})
            for (const int back : {1, 30, 100}) {
                const int at = end > back ? end - back : 0, next = next_start(at, end, step);
                if (next <= at || next > end || (next < end && next != at + step)) return 2;
            }
    printf("row steps passed\n");
    return 0;
}
