// How the layer of experts is cut (csrc/tdg_layer_plan.h): a line of standard
// input, "tokens top_k experts cols inner", gives a line with its kernels and
// parts.  "sweep" as the argument gives the lines that a wide sweep of sizes
// meets, once each, with the first size that gives it.
#include <stdio.h>
#include <string.h>

#include <initializer_list>
#include <set>
#include <string>

#include "tdg_layer_plan.h"

static std::string cut(long tokens, long top_k, long experts, long cols, long inner) {
    const tdg::LayerPlan p = tdg::layer_plan(tokens, top_k, experts, cols, inner);
    char line[80];
    snprintf(line, sizeof line, "up %s %d down %s %d%s", !inner ? "none" : p.thin_up ? "thin" : p.two_tiles ? "two" : "one",
             (int)p.parts, p.thin_down ? "thin" : p.narrow ? "narrow" : "wide", (int)p.parts_z, inner ? "" : " no inner");
    return line;
}

int main(int argc, char **argv) {
    long t, k, e, c, i;
    if (argc > 1 && !strcmp(argv[1], "sweep")) {
        std::set<std::string> seen;
        for (long tokens : {1, 2, 3, 4, 5, 8, 13, 16, 20, 27, 33, 40, 50, 64})
            for (long top_k : {1, 2, 3, 4, 6, 8, 16, 32})
                for (long experts : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 128, 256, 1024})
                    for (long cols : {1, 7, 8, 63, 128, 500, 511, 512, 700, 1000, 1023, 1024, 1500, 2048, 2050, 3000, 4096,
                                      6000, 8192, 16384})
                        for (long inner : {0, 1, 7, 8, 64, 128, 129, 255, 256, 384, 500, 511, 512, 700, 768, 1000, 1024,
                                           1500, 2048, 4096, 8192, 16384}) {
                            const std::string line = cut(tokens, top_k, experts, cols, inner);
                            if (seen.insert(line).second)
                                printf("%s: %ld %ld %ld %ld %ld\n", line.c_str(), tokens, top_k, experts, cols, inner);
                        }
        return 0;
    }
    while (scanf("%ld %ld %ld %ld %ld", &t, &k, &e, &c, &i) == 5) puts(cut(t, k, e, c, i).c_str());
    return 0;
}
