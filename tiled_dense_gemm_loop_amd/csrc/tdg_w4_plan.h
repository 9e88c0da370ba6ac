// tdg_w4_plan.h -- which kernel a product with 4-bit weights runs, a function of
// its sizes alone.  Nothing here calls HIP.
#pragma once

#include "tdg_check.h"

namespace tdg {

// k_w4_few<MT, CT, waves> (16 MT rows, 16 CT columns) and k_w4_tile<MT, CT, waves>
// (16 MT rows, 16 CT columns for each wave).
enum W4Kernel {
    W4_FEW_1_1_16,
    W4_FEW_1_1_8,
    W4_FEW_1_2_8,
    W4_FEW_1_4_8,
    W4_FEW_2_4_8,
    W4_TILE_128_512,
    W4_TILE_64_256,
    W4_TILE_64_128,
    W4_TILE_32_128,
    W4_TILE_32_64,
    W4_KERNELS
};

struct W4Size {
    int64_t rows, groups;  // 0: all rows have one matrix
    int64_t N, K, group, lda;

    // Groups that can have rows.
    int64_t live() const { return !groups ? 1 : groups < rows ? groups : rows; }
    // Tiles of bm x bn that the product is expected to have: half a row tile for each
    // group that can have rows, beside those that the rows fill.
    int64_t tiles(int64_t bm, int64_t bn) const {
        const int64_t high = groups ? rows / bm + live() / 2 : ceil_quot(rows, bm);
        return (high > live() ? high : live()) * ceil_quot(N, bn);
    }
};

inline W4Kernel w4_kernel(const W4Size &p) {
    const int64_t live = p.live(), blocks = ceil_quot(p.K, 128);
    // Pieces of 16 rows by 16 columns.
    const int64_t pieces = (p.groups ? live : ceil_quot(p.rows, 16)) * ceil_quot(p.N, 16);
    // The DMA's lanes reach a tile's rows with 32-bit byte offsets.
    const bool far = p.lda > (int64_t)UINT32_MAX / 2 / 128 - 256;
    // Few rows: as many columns to a workgroup as leave one or two to a CU (us,
    // 16 / 32 / 64 columns: 16 x 4096 x 4096, 256 pieces, 6.6 / 7.2 / -; 24 rows,
    // 512, 9.7 / 7.5 / 8.7; 64 rows, 1024, 15.0 / 12.2 / 9.2; 1 x 16384 x 4096,
    // 1024, - / 10.6 / 10.2); then two row tiles (128 rows, 2048: 15.7 with one,
    // 13.7 with two, 32 x 64 tiles from LDS 16.1; 192 rows: 21.0, 24.8, 18.8; 32
    // x 16384 x 4096, 2048: 16.9, 15.0, 21).  Groups of rows: up to 8 to a
    // group (32 groups of 2048 x 2048, 200 rows: 17.9, tiles 19.2; 400: 22.6, 19.6).
    const bool short_groups = p.rows <= 8 * live;
    if (far || blocks == 0 || (p.groups ? short_groups : p.rows <= 32 || pieces <= 2048)) {
        // 16 waves where k is long or so few rows that their loads do not count
        // (us, 8 / 16 waves: 1 x 4096 x 4096 4.9 / 4.3, 1 x 512 x 8192 6.7 / 5.4, 16 x
        // 4096 x 4096 6.6 / 6.9).
        if (pieces <= 384) return (p.rows <= 4 || blocks >= 64) && !p.groups ? W4_FEW_1_1_16 : W4_FEW_1_1_8;
        if (pieces <= 640) return W4_FEW_1_2_8;
        if (pieces <= 1280 || p.rows <= 16 || (p.groups && short_groups)) return W4_FEW_1_4_8;
        return W4_FEW_2_4_8;
    }
    // Tiles.  128 x 512, one to a CU, where its rounds of 256 are full (us, against
    // 64 x 256: 4096 x 4096 x 4096, 256 tiles, 121 / 138; 3000 x 11008 x 2048, 528,
    // 174 / 150; 16 groups of 1024 rows, 4096 x 4096, 1088 588 / 585).  Shorter
    // groups' scales ask for more registers than there are (4096 x 8192 x 4096, groups
    // of 64: 302 / 302, of 32: 471 / 351).
    const int64_t large = p.tiles(128, 512);
    if (large * 100 > ceil_quot(large, 256) * 256 * 85 && p.rows >= 1024 * live && p.group % 128 == 0)
        return W4_TILE_128_512;
    // A few rows of each group: 32 x 128, or 64 wide (us, against 64 x 128 / 32 x 64:
    // 32 groups of 2048 x 2048, 600 rows 20.3, 25.2 / 21.4; 1000 rows 25.4, 26.1 /
    // 30.1; 2000 rows -, 32.7 / -; 9 groups of 1537 x 1000, 333 rows 8.6, 9.7 / 7.9).
    if (p.rows <= 40 * live) return p.tiles(32, 128) >= 256 ? W4_TILE_32_128 : W4_TILE_32_64;
    // 64 x 256, two to a CU (us, against 64 x 128: 2048 x 4096 x 4096, 512 tiles, 73
    // / 80; 1536 rows, 384, 64 / 60; 1024 rows, 256, 44 / 42); 64 x 128, three to a
    // CU, against 32 x 64 (512 rows, 256 tiles: 29 / 30; 192 rows, 96: 26 / 19).
    if (p.tiles(64, 256) > 416) return W4_TILE_64_256;
    if (p.tiles(64, 128) >= 256) return W4_TILE_64_128;
    return W4_TILE_32_64;
}

}  // namespace tdg
