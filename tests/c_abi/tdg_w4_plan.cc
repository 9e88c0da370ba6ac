// Which kernel products with 4-bit weights run (csrc/tdg_w4_plan.h): a line of
// standard input, "rows groups N K group lda", gives a line with its name.
#include <stdio.h>

#include "tdg_w4_plan.h"

int main() {
    static const char *const names[tdg::W4_KERNELS] = {
        "few 1 1 16", "few 1 1 8", "few 1 2 8", "few 1 4 8", "few 2 4 8",
        "tile 128 512", "tile 64 256", "tile 64 128", "tile 32 128", "tile 32 64"};
    long rows, groups, N, K, group, lda;
    while (scanf("%ld %ld %ld %ld %ld %ld", &rows, &groups, &N, &K, &group, &lda) == 6)
        printf("%s\n", names[tdg::w4_kernel({rows, groups, N, K, group, lda})]);
    return 0;
}
