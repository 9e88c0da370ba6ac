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

int run_grouped(int lay, int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N, int64_t K,
                const void *A, int64_t lda, const void *B, int64_t ldb, int64_t stride_b, void *C, int64_t ldc,
                int64_t stride_c, void *stream) {
    int rc = grouped_args_ok(lay, groups, offsets, rows, M, N, K, A, lda, B, ldb, stride_b, C, ldc, stride_c);
    if (rc != TDG_OK) return rc;
    if (groups == 0 || N == 0 || (lay == tdg::LAY_TN ? M == 0 : rows == 0)) return TDG_OK;

    constexpr int BM = 128, BN = 128, NT = 256;
    const void *fn = lay == tdg::LAY_NN   ? (const void *)&tdg::tdg_grouped_any<tdg::LAY_NN, BM, BN, 2, 2>
                     : lay == tdg::LAY_NT ? (const void *)&tdg::tdg_grouped_any<tdg::LAY_NT, BM, BN, 2, 2>
                                          : (const void *)&tdg::tdg_grouped_any<tdg::LAY_TN, BM, BN, 2, 2>;
    GroupedArgs a;
    a.A = (const unsigned char *)A, a.B = (const unsigned char *)B, a.C = (unsigned char *)C;
    a.lda = lda * 2, a.ldb = ldb * 2, a.ldc = ldc * 4;
    a.stride_b = stride_b * 2, a.stride_c = stride_c * 4;
    a.offsets = offsets;
    a.groups = (int)groups, a.rows = (int)rows, a.M = (int)M, a.N = (int)N, a.K = (int)K;
    a.tiles_m = (int)tdg::ceil_quot(M, BM), a.tiles_n = (int)tdg::ceil_quot(N, BN);
    // Most tiles: every group can end inside a tile, and needs a row for it.
    const int64_t row_tiles = lay == tdg::LAY_TN ? groups * a.tiles_m
                                                 : rows / BM + (groups < rows ? groups : rows);
    if (row_tiles > INT32_MAX / a.tiles_n) return TDG_ERR_UNSUPPORTED;
    const int64_t grid = tdg::ceil_quot(row_tiles * a.tiles_n, 8) * 8;
    if (grid > (int64_t)UINT32_MAX / NT) return TDG_ERR_UNSUPPORTED;
    rc = tdg::device_check();
    if (rc != TDG_OK) return rc;
    void *kargs[] = {&a};
    if (hipLaunchKernel(fn, dim3((unsigned)grid), dim3(NT), kargs, 0, (hipStream_t)stream) != hipSuccess)
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
