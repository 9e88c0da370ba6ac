// tdg_layer_plan.h -- how the layer of experts for a few tokens is cut, a function
// of its sizes alone, as its workspace is.  Nothing here calls HIP.
#pragma once

#include "tdg_check.h"

namespace tdg {

inline int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

inline int64_t at_most(int64_t n, int64_t most) { return n < most ? n : most; }

struct LayerPlan {
    int64_t slots, up_x, parts, down_x, parts_z, piece;
    bool thin_up, thin_down, narrow;  // matrices below 8 columns; 64 instead of 128 columns of down to a workgroup
    bool two_tiles;                   // two row tiles to a workgroup of up
    uint64_t z_at, bytes;
};

inline LayerPlan layer_plan(int64_t tokens, int64_t top_k, int64_t experts, int64_t cols, int64_t inner) {
    LayerPlan p;
    const int64_t entries = tokens * top_k;
    p.slots = entries < experts ? entries : experts;
    // down: 128 columns and eight waves, k in two parts below 512 workgroups; 64
    // columns and sixteen waves below 192 (us, 128 whole / 128 in two / 64 whole /
    // 64 in two: 16 tokens, 1024 workgroups of 128, 50.7 / 51.4 / 56 / 65; 33
    // tokens of 8 experts, 256, 22.3 / 20.2 / 23.3 / -; one token, 128, 10.9 / 9.3 /
    // 8.5 / 9.7; 2 experts of 4096 x 4096, 64, - / 27 / 28 / 17).
    p.thin_down = cols < 8;
    const int64_t wide = ceil_quot(cols, 128) * p.slots;
    p.narrow = !p.thin_down && wide < 192;
    p.down_x = ceil_quot(cols, p.thin_down ? 16 : p.narrow ? 64 : 128);
    p.parts_z = p.thin_down ? 1 : at_most(wide < 96 || (wide >= 192 && wide < 512) ? 2 : 1, inner / 256);
    if (p.parts_z < 1) p.parts_z = 1;
    // A CU takes about 35 GB/s from L2, so the weights need most CUs: k is cut in
    // two or four where there are few workgroups (us, 1 / 2 / 4 parts: one token, 8
    // experts of 2048 x 2 768, 48 workgroups, 17.3 / 12.5 / 11.4; two tokens, 96, 21
    // / 18.7 / 21; 33 tokens, 8 experts of 4095 x 2 1001, 64, - / 33.8 / 32.9), if LDS
    // holds what down then joins.
    p.thin_up = inner < 8;
    p.up_x = ceil_quot(inner, p.thin_up ? 16 : 128);
    // Two row tiles where many experts have more than one (us, one / two: 64
    // tokens, 2 of 8 experts, 146 / 99; 8 of 64 experts 107.8 / 104.5; 33 tokens, 2
    // of 8, 32.9 / 36.6).
    p.two_tiles = !p.thin_up && entries > 10 * p.slots;
    const int64_t wgs = p.up_x * p.slots, waves = p.narrow ? 16 : 8;
    p.piece = ceil_quot(ceil_quot(inner, 16), waves * p.parts_z) * 16 * at_most(entries, 16);
    p.parts = wgs > 96 || cols < 512 || p.piece * waves * 4 > 40 * 1024 ? 1 : wgs > 64 || cols < 1024 ? 2 : 4;
    p.z_at = (uint64_t)(entries * up4(inner) * 4 * (p.parts > 1 ? 2 * p.parts : 1));
    p.bytes = p.z_at + (uint64_t)(p.parts_z * entries * up4(cols) * 4);
    return p;
}

}  // namespace tdg
