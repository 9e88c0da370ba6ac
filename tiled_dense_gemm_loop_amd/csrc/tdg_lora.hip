// tdg_lora.hip -- a shared projection with low-rank adapters of many requests
// beside it: C[t] = A[t] . B + scale[a] * (A[t] . down[a]) . up[a], where
// a = adapter[t], and the second term is left out where a is not in
// [0, adapters).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tdg_check.h"
#include "tdg_internal.h"
#include "tdgemm.h"

namespace {

struct LoraArgs {
    const _Float16 *A, *down, *up;
    const int32_t *adapter;
    const float *scale;
    float *C, *low;  // low: M x rank, the rows' products with their down
    int64_t lda, ldc, ld_down, stride_down, ld_up, stride_up;
    int M, N, K, adapters, rank;
};

constexpr int THREADS = 256;

// low[t][c]: 32 columns by 8 slices of K per workgroup.
__global__ void __launch_bounds__(THREADS) k_lora_low(LoraArgs p) {
    __shared__ float part[8][32];
    const int t = blockIdx.x, c = blockIdx.y * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    const int a = p.adapter[t];
    if ((unsigned)a >= (unsigned)p.adapters) return;
    const _Float16 *x = p.A + (int64_t)t * p.lda, *d = p.down + a * p.stride_down;
    float sum = 0.0f;
    if (c < p.rank)
        for (int k = slice; k < p.K; k += 8) sum = fmaf((float)x[k], (float)d[(int64_t)k * p.ld_down + c], sum);
    part[slice][threadIdx.x & 31] = sum;
    __syncthreads();
    if (slice == 0 && c < p.rank) {
        float s = 0.0f;
        for (int i = 0; i < 8; i++) s += part[i][threadIdx.x & 31];
        p.low[(int64_t)t * p.rank + c] = s;
    }
}

// C[t][n] += scale * sum_c low[t][c] * up[c][n].
__global__ void __launch_bounds__(THREADS) k_lora_add(LoraArgs p) {
    const int t = blockIdx.x;
    const int64_t n = (int64_t)blockIdx.y * THREADS + threadIdx.x;
    const int a = p.adapter[t];
    if ((unsigned)a >= (unsigned)p.adapters || n >= p.N) return;
    const _Float16 *u = p.up + a * p.stride_up + n;
    const float *low = p.low + (int64_t)t * p.rank;
    float sum = 0.0f;
    for (int c = 0; c < p.rank; c++) sum = fmaf(low[c], (float)u[(int64_t)c * p.ld_up], sum);
    float *dst = p.C + (int64_t)t * p.ldc + n;
    *dst = fmaf(p.scale ? p.scale[a] : 1.0f, sum, *dst);
}

int launch(const void *fn, dim3 grid, LoraArgs *args, void *stream) {
    void *kargs[] = {args};
    if (hipLaunchKernel(fn, grid, dim3(THREADS), kargs, 0, (hipStream_t)stream) != hipSuccess) return TDG_ERR_LAUNCH;
    if (hipGetLastError() != hipSuccess) return TDG_ERR_LAUNCH;
    return TDG_OK;
}

bool sizes_ok(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank) {
    return tdg::size_ok(M) && tdg::size_ok(N) && tdg::size_ok(K) && tdg::size_ok(adapters) && rank >= 0 &&
           rank <= TDG_LORA_MAX_RANK;
}

}  // namespace

extern "C" {

int tdg_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank, size_t *bytes) {
    if (!bytes || !sizes_ok(M, N, K, adapters, rank)) return TDG_ERR_INVALID_ARG;
    *bytes = (size_t)M * (size_t)rank * sizeof(float);
    return TDG_OK;
}

int gemm_f16f32_lora(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, const uint16_t *B,
                     int64_t ldb, int64_t adapters, int64_t rank, const uint16_t *down, int64_t ld_down,
                     int64_t stride_down, const uint16_t *up, int64_t ld_up, int64_t stride_up,
                     const int32_t *adapter, const float *scale, float *C, int64_t ldc, void *workspace,
                     size_t workspace_bytes, void *stream) {
    size_t need = 0;
    if (tdg_lora_workspace(M, N, K, adapters, rank, &need) != TDG_OK) return TDG_ERR_INVALID_ARG;
    int rc = tdg::validate_gemm(TDG_DTYPE_F16F32, M, N, K, A, lda, B, ldb, C, ldc);
    if (rc != TDG_OK) return rc;
    if (!tdg::stack_ok(down, adapters, stride_down, K, rank, ld_down, 2, false) ||
        !tdg::stack_ok(up, adapters, stride_up, rank, N, ld_up, 2, false))
        return TDG_ERR_INVALID_ARG;
    if (!tdg::aligned_to(A, 2) || !tdg::aligned_to(B, 2) || !tdg::aligned_to(down, 2) || !tdg::aligned_to(up, 2) ||
        !tdg::aligned_to(C, 4) || !tdg::aligned_to(adapter, 4) || !tdg::aligned_to(scale, 4))
        return TDG_ERR_INVALID_ARG;
    const bool side = adapters > 0 && rank > 0 && K > 0 && M > 0 && N > 0;
    if (side && !adapter) return TDG_ERR_INVALID_ARG;
    const uint64_t c_len = tdg::span_bytes(M, N, ldc, 4);
    const void *in[6] = {A, B, down, up, adapter, scale};
    const uint64_t in_len[6] = {tdg::span_bytes(M, K, lda, 2), tdg::span_bytes(K, N, ldb, 2),
                                tdg::span_bytes(K, rank, ld_down, 2, adapters, stride_down),
                                tdg::span_bytes(rank, N, ld_up, 2, adapters, stride_up), (uint64_t)M * 4,
                                (uint64_t)adapters * 4};
    if (side && need && (!workspace || workspace_bytes < need || !tdg::aligned_to(workspace, 16)))
        return TDG_ERR_INVALID_ARG;
    for (int i = 0; i < 6; i++)
        if (tdg::overlaps(C, c_len, in[i], in_len[i]) || (side && tdg::overlaps(workspace, need, in[i], in_len[i])))
            return TDG_ERR_INVALID_ARG;
    if (side && tdg::overlaps(workspace, need, C, c_len)) return TDG_ERR_INVALID_ARG;
    if (side && (M > (int64_t)UINT32_MAX / THREADS || tdg::ceil_quot(N, THREADS) > 65535))
        return TDG_ERR_UNSUPPORTED;

    rc = gemm_f16f32_pipelined(M, N, K, A, lda, B, ldb, C, ldc, stream);
    if (rc != TDG_OK || !side) return rc;
    LoraArgs p;
    p.A = (const _Float16 *)A, p.down = (const _Float16 *)down, p.up = (const _Float16 *)up;
    p.adapter = adapter, p.scale = scale, p.C = C, p.low = (float *)workspace;
    p.lda = lda, p.ldc = ldc, p.ld_down = ld_down, p.stride_down = stride_down, p.ld_up = ld_up;
    p.stride_up = stride_up;
    p.M = (int)M, p.N = (int)N, p.K = (int)K, p.adapters = (int)adapters, p.rank = (int)rank;
    rc = launch((const void *)&k_lora_low, dim3((unsigned)M, (unsigned)tdg::ceil_quot(rank, 32)), &p, stream);
    if (rc != TDG_OK) return rc;
    return launch((const void *)&k_lora_add, dim3((unsigned)M, (unsigned)tdg::ceil_quot(N, THREADS)), &p, stream);
}

}  // extern "C"
