// tdg_grouped.hip -- host side of the products whose rows pick their weights:
// gemm_f16f32_grouped, _nt and _tn.
#include "tdg_grouped.hpp"

#include "tdg_check.h"
#include "tdg_internal.h"

namespace {

using tdg::GroupedArgs;

constexpr int64_t kMaxGroups = 1024;

// Arguments of the three products: `rows` rows of A; NN / NT: a K-long sum per
// row and N columns; TN: an M x N product per group.
int grouped_args_ok(int lay, int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N, int64_t K,
                    const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b, const void *C,
                    int64_t ldc, int64_t stride_c) {
    if (groups < 0 || groups > kMaxGroups || !tdg::size_ok(rows) || !tdg::size_ok(M) || !tdg::size_ok(N) ||
        !tdg::size_ok(K))
        return TDG_ERR_INVALID_ARG;
    if (groups > 0 && (!offsets || !tdg::aligned_to(offsets, 4))) return TDG_ERR_INVALID_ARG;
    const uint64_t off_len = groups > 0 ? (uint64_t)(groups + 1) * 4 : 0;
    uint64_t a_len, b_len, c_len;
    if (lay == tdg::LAY_TN) {
        if (!tdg::matrix_ok(A, rows, M, lda, 2) || !tdg::matrix_ok(B, rows, N, ldb, 2) ||
            !tdg::stack_ok(C, groups, stride_c, M, N, ldc, 4, true))
            return TDG_ERR_INVALID_ARG;
        a_len = tdg::span_bytes(rows, M, lda, 2);
        b_len = tdg::span_bytes(rows, N, ldb, 2);
        c_len = tdg::span_bytes(M, N, ldc, 4, groups, stride_c);
    } else {
        const int64_t br = lay == tdg::LAY_NN ? K : N, bc = lay == tdg::LAY_NN ? N : K;
        if (!tdg::matrix_ok(A, rows, K, lda, 2) || !tdg::stack_ok(B, groups, stride_b, br, bc, ldb, 2, false) ||
            !tdg::matrix_ok(C, rows, N, ldc, 4))
            return TDG_ERR_INVALID_ARG;
        a_len = tdg::span_bytes(rows, K, lda, 2);
        b_len = tdg::span_bytes(br, bc, ldb, 2, groups, stride_b);
        c_len = tdg::span_bytes(rows, N, ldc, 4);
    }
    if (!tdg::aligned_to(A, 2) || !tdg::aligned_to(B, 2) || !tdg::aligned_to(C, 4)) return TDG_ERR_INVALID_ARG;
    if (tdg::overlaps(C, c_len, A, a_len) || tdg::overlaps(C, c_len, B, b_len) ||
        tdg::overlaps(C, c_len, offsets, off_len))
        return TDG_ERR_INVALID_ARG;
    return TDG_OK;
}

struct Variant {
    const void *fn;
    int bm, bn, threads;
    int most_wgs;  // workgroups that are launched at most (they take several tiles)
};

#define TDG_BY_LAYOUT(KERNEL, ...)                                              \
    (lay == tdg::LAY_NN   ? (const void *)&tdg::KERNEL<tdg::LAY_NN, __VA_ARGS__> \
     : lay == tdg::LAY_NT ? (const void *)&tdg::KERNEL<tdg::LAY_NT, __VA_ARGS__> \
                          : (const void *)&tdg::KERNEL<tdg::LAY_TN, __VA_ARGS__>)

Variant choose(int lay, int64_t groups, int64_t rows, int64_t M, int64_t N, int64_t lda, int64_t ldb,
               bool a_stops, bool b_stops) {
    const bool tn = lay == tdg::LAY_TN;
    // The DMA's lanes reach a tile's rows with 32-bit byte offsets.  Where
    // an operand's rows lie at one k each and its last chunk must not be copied
    // (a_stops, b_stops), the rows have to be long enough for no other row's
    // chunk to reach as far.
    const int64_t far = (int64_t)UINT32_MAX / 2 / 256 - 256;
    const bool thin = (tn && lda < 8 && a_stops) || (lay != tdg::LAY_NT && ldb < 8 && b_stops);
    if (thin || lda > far || ldb > far) return {TDG_BY_LAYOUT(tdg_grouped_any, 128, 128, 2, 2), 128, 128, 256, INT32_MAX};
    // Tiles that the product is expected to have: half a row tile more per
    // group that can have rows than the rows fill, one at the least.
    const int64_t live = groups < rows ? groups : rows;
    auto tiles = [&](int64_t b) {
        int64_t high = rows / b + live / 2;
        if (high < live) high = live;
        return (tn ? groups * tdg::ceil_quot(M, b) : high) * tdg::ceil_quot(N, b);
    };
    const int64_t t256 = tiles(256), t128 = tiles(128);
    // Rounds of workgroups, in tenths of one of 256 x 256 tiles (256 at a time).
    // A round of 128 x 128 tiles with two buffers has two for each CU, 512, and
    // takes 0.6 of that: half the operations at 0.84 of the rate.  A last round
    // of few large tiles is cut in two (not TN's), and takes 0.7.
    const int64_t rest = t256 % 256;
    const int64_t large = t256 / 256 * 10 + (rest == 0 ? 0 : !tn && t256 > 256 && rest <= 128 ? 7 : 10);
    const int64_t small = tdg::ceil_quot(t128, 512) * 6;
    // So 256 x 256 where its rounds are the shorter ones and the groups have
    // the rows for it (us, 256 / 128 wide; NN 4096 rows, 4 groups of 2048 x 2048,
    // 144 tiles: 49 / 56; of 2048 x 1792, 126 tiles: 47 / 38; TN 14815 rows, 9
    // groups of 1480 x 1216, 270 tiles: 98 / 85; NN 16384 rows, 16 groups of 4096
    // x 4096: 564 / 668; 4096 rows, 32 groups of 2048 x 2048: 102 / 97).
    if (large <= small && (tn || rows >= 192 * live))
        return tn ? Variant{(const void *)&tdg::tdg_grouped_tn_loop<256, 256, 2, 4, 2>, 256, 256, 512, 256}
                  : Variant{lay == tdg::LAY_NN ? (const void *)&tdg::tdg_grouped_cut<tdg::LAY_NN>
                                               : (const void *)&tdg::tdg_grouped_cut<tdg::LAY_NT>,
                            256, 256, 512, INT32_MAX};
    // A few rows of each group are bound by reading B from HBM: 32 x 256 spends
    // the copies in flight on B and reads 512 bytes of a row of it, where the
    // tiles fill half of the CUs (us against the rules below; 64 rows, 32
    // groups, 2048 x 2048: 41 / 45; 128 rows, 128 groups, 4096 x 1536: 157 /
    // 171; with 16 rows a group too many groups need two: 68 / 52).
    if (lay == tdg::LAY_NN && rows <= 8 * live && live * tdg::ceil_quot(N, 256) >= 128)
        return {(const void *)&tdg::tdg_grouped_ring<tdg::LAY_NN, 32, 256, 1, 4, 4>, 32, 256, 256, INT32_MAX};
    // Otherwise 64 x 64 for few rows, down to one tile that reads B (8 rows, 64
    // groups of 2048 x 1408, 64 / 128 wide: 11 / 17), and where NT reads whole
    // rows of B, a narrow tile more of each at a time (512 rows, 32 groups of
    // 2048 x 2048: 58 / 69); NN's many groups do better with 128 x 128 (52 / 56).
    const bool few = !tn && rows <= 16 * live;
    if (t128 > 256 && !(few && lay == tdg::LAY_NT))
        return {TDG_BY_LAYOUT(tdg_grouped_ring, 128, 128, 2, 2, 2), 128, 128, 256, INT32_MAX};
    // And 64 x 64, of which a CU holds two, for products that it can do in one
    // round (64 wide / 128 wide with four buffers, one to a CU: NN 6144 rows, 6
    // groups of 2048 x 384, 153 large tiles: 24 / 20; 4096 rows, 8 groups, 108:
    // 16 / 19; TN 16384 rows, 1536 x 1536, 144: 167 / 109; 8192 rows, 8 groups
    // of 512 x 512, 128: 14 / 16).
    if (t128 > 128 && !few) return {TDG_BY_LAYOUT(tdg_grouped_ring, 128, 128, 2, 2, 4), 128, 128, 256, INT32_MAX};
    return {TDG_BY_LAYOUT(tdg_grouped_ring, 64, 64, 2, 2, 4), 64, 64, 256, INT32_MAX};
}

int run_grouped(int lay, int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N, int64_t K,
                const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b, void *C, int64_t ldc,
                int64_t stride_c, void *stream) {
    int rc = grouped_args_ok(lay, groups, offsets, rows, M, N, K, A, lda, B, ldb, stride_b, C, ldc, stride_c);
    if (rc != TDG_OK) return rc;
    if (groups == 0 || N == 0 || (lay == tdg::LAY_TN ? M == 0 : rows == 0)) return TDG_OK;

    GroupedArgs a;
    const bool tn = lay == tdg::LAY_TN;
    a.a_stop = tdg::chunk_stop(A, rows, tn ? M : K, lda);
    const int64_t br = lay == tdg::LAY_NN ? K : N, bc = lay == tdg::LAY_NN ? N : K;  // of a group's B
    a.b_stop = tn ? tdg::chunk_stop(B, rows, N, ldb) : tdg::chunk_stop(B, br, bc, ldb, groups, stride_b);
    a.b_each = !tn && tdg::stops_each(br, bc, ldb, groups, stride_b);
    const Variant v = choose(lay, groups, rows, M, N, lda, ldb, a.a_stop != tdg::kNoStop,
                             a.b_each || a.b_stop != tdg::kNoStop);
    a.A = (const unsigned char *)A, a.B = (const unsigned char *)B, a.C = (unsigned char *)C;
    a.lda = lda * 2, a.ldb = ldb * 2, a.ldc = ldc * 4;
    a.stride_b = stride_b * 2, a.stride_c = stride_c * 4;
    a.offsets = offsets;
    a.groups = (int)groups, a.rows = (int)rows, a.M = (int)M, a.N = (int)N, a.K = (int)K;
    a.tiles_m = (int)tdg::ceil_quot(M, v.bm), a.tiles_n = (int)tdg::ceil_quot(N, v.bn);
    // A and B fit in half of the 256 MB memory-side cache, and C is much larger.
    const uint64_t in_bytes = (uint64_t)rows * (uint64_t)(M + N) * 2, out_bytes = (uint64_t)groups * M * N * 4;
    a.warm = in_bytes <= (128u << 20) && out_bytes / 4 >= in_bytes;
    a.flags = tdg::debug_flags_now();
    // Most row tiles: every group can end inside a tile, and needs a row for
    // it.
    const int64_t row_tiles = lay == tdg::LAY_TN ? groups * a.tiles_m
                                                 : rows / v.bm + (groups < rows ? groups : rows);
    if (row_tiles > INT32_MAX / a.tiles_n) return TDG_ERR_UNSUPPORTED;
    // (And up to 16 tiles of each XCD can be cut in two.)
    int64_t grid = tdg::ceil_quot(row_tiles * a.tiles_n, 8) * 8 + 8 * 16;
    if (grid > INT32_MAX - 65536) return TDG_ERR_UNSUPPORTED;
    a.tiles_most = (int)grid;
    if (grid > v.most_wgs) grid = v.most_wgs;
    if (grid > (int64_t)UINT32_MAX / v.threads) return TDG_ERR_UNSUPPORTED;
    rc = tdg::device_check();
    if (rc != TDG_OK) return rc;
    void *kargs[] = {&a};
    if (hipLaunchKernel(v.fn, dim3((unsigned)grid), dim3((unsigned)v.threads), kargs, 0, (hipStream_t)stream) != hipSuccess)
        return TDG_ERR_LAUNCH;
    if (hipGetLastError() != hipSuccess) return TDG_ERR_LAUNCH;
    return TDG_OK;
}

}  // namespace

extern "C" {

int gemm_f16f32_grouped(int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K, const uint16_t *A,
                        int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b, float *C, int64_t ldc,
                        void *stream) {
    return run_grouped(tdg::LAY_NN, groups, offsets, M, 0, N, K, A, lda, B, ldb, stride_b, C, ldc, 0, stream);
}

int gemm_f16f32_grouped_nt(int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K,
                           const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b,
                           float *C, int64_t ldc, void *stream) {
    return run_grouped(tdg::LAY_NT, groups, offsets, M, 0, N, K, A, lda, B, ldb, stride_b, C, ldc, 0, stream);
}

int gemm_f16f32_grouped_tn(int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N,
                           const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, float *C, int64_t ldc,
                           int64_t stride_c, void *stream) {
    return run_grouped(tdg::LAY_TN, groups, offsets, rows, M, N, 0, A, lda, B, ldb, 0, C, ldc, stride_c, stream);
}

}  // extern "C"
