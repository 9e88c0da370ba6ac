// tdg_lora.hip -- a shared projection with low-rank adapters of many requests
// beside it: C[t] = A[t] . B + scale[a] * (A[t] . down[a]) . up[a], where
// a = adapter[t], and the second term is left out where a is not in
// [0, adapters).
//
// Two launches.  The first makes low[t] = A[t] . down[a], a thin product that
// K is cut for so that it fills the chip; its parts are summed where they are
// read.  The second makes C:
//   * many rows (k_lora_main): the shared product's tiles, and on each wave's
//     32-row blocks low . up on the matrix cores, one pass per distinct
//     adapter of the block, added to the accumulators of that adapter's rows
//     alone: C is written once, and no row sees another's adapter;
//   * few rows: the shared product is bound by reading B, and has too few
//     tiles to do it at full rate.  Its parts over K are made in the first
//     launch beside low's, and the second (k_lora_join) sums them and adds
//     low . up in FP32.
// On the matrix cores low goes in as two FP16 parts, high and rest, of the row
// scaled by a power of two to just under 2^14: 21 bits or more at any size.
#include "tdg_grouped.hpp"

#include "tdg_check.h"
#include "tdg_internal.h"

namespace {

using namespace tdg;

struct LoraArgs {
    const unsigned char *A, *B, *down, *up;
    const int32_t *adapter;
    const float *scale;
    float *C;
    float *part;  // parts x M x N: the shared product over slices of K (few rows)
    float *low;   // low_parts x M x rank
    int64_t lda, ldb, ldc, ld_down, stride_down, ld_up, stride_up;  // bytes
    int M, N, K, adapters, rank;
    int row_tiles, col_tiles;           // of the shared product
    int parts, k_per_part;              // K tiles of each slice
    int low_parts, low_k_per_part;
    int low_cols, low_lanes;            // blocks of the rank; workgroups that share a row tile's adapters
    int shared_wgs;                     // workgroups on the shared product
    int flags;
};

// Which adapter a row has, -1 for none.
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int row) {
    const int a = row < p.M ? p.adapter[row] : -1;
    return (unsigned)a < (unsigned)p.adapters ? a : -1;
}

// The first launch: tiles of the shared product over a slice of K (few rows
// only), and of low.  A tile of low belongs to BM <= 64 rows; its workgroups
// take the distinct adapters among those rows in turn, each a whole product of
// which the adapter's own rows are kept.
template <class E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void lora_parts(const LoraArgs &p, unsigned char *smem) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    poison_lds<E::SMEM, E::NT>(p.flags, smem);
    f32x16 acc[E::MI][E::NI];
    int b = blockIdx.x;
    if (b < p.shared_wgs) {
        // XCD b % 8 takes a run of tiles, rows first: B's tile is read once
        // into its L2 for all row tiles.
        const int per = (p.shared_wgs + 7) >> 3;
        b = (b & 7) * per + (b >> 3);
        if (b >= p.row_tiles * p.col_tiles * p.parts) return;
        const int tm = b % p.row_tiles, rest = b / p.row_tiles;
        const int tn = rest % p.col_tiles, part = rest / p.col_tiles;
        const int k_lo = part * p.k_per_part * 64, k_hi = min(p.K, k_lo + p.k_per_part * 64);
        clear_acc(acc);
        E::run(p.A, p.lda, p.B, p.ldb, tm * BM, p.M, tn * BN, p.N, k_lo, k_hi, smem, acc);
        store_tile<E::MI, E::NI>((unsigned char *)(p.part + (int64_t)part * p.M * p.N), (int64_t)p.N * 4,
                                 tm * BM + wm * E::WTM, p.M, tn * BN + wn * E::WTN, p.N, acc);
        return;
    }
    b -= p.shared_wgs;
    const int turn = b % p.low_lanes;
    b /= p.low_lanes;
    const int tc = b % p.low_cols;
    b /= p.low_cols;
    const int part = b % p.low_parts, row0 = b / p.low_parts * BM;
    const int k_lo = part * p.low_k_per_part * 64, k_hi = min(p.K, k_lo + p.low_k_per_part * 64);
    float *low = p.low + (int64_t)part * p.M * p.rank;
    const int id = adapter_of(p, lane < BM ? row0 + lane : p.M);
    unsigned long long left = __ballot(id >= 0);
    bool first = true;
    for (int n = 0; left; n++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffsll(left) - 1));
        const unsigned long long mine = __ballot(id == a);
        left &= ~mine;
        if (n % p.low_lanes != turn) continue;
        if (!first) __syncthreads();  // every wave is done with the LDS of the product before
        first = false;
        clear_acc(acc);
        E::run(p.A, p.lda, p.down + (int64_t)a * p.stride_down, p.ld_down, row0, p.M, tc * BN, p.rank, k_lo, k_hi,
               smem, acc);
#pragma unroll
        for (int mi = 0; mi < E::MI; mi++)
#pragma unroll
            for (int ni = 0; ni < E::NI; ni++) {
                const int c = tc * BN + wn * E::WTN + ni * 32 + (lane & 31);
#pragma unroll
                for (int v = 0; v < 16; v++) {
                    const int r = wm * E::WTM + mi * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
                    if ((mine >> r) & 1 && c < p.rank) low[(int64_t)(row0 + r) * p.rank + c] = acc[mi][ni][v];
                }
            }
    }
}

template <int BM, int BN, int WM, int WN, int STAGES>
__global__ void __launch_bounds__(WM *WN * 64, 1) k_lora_parts_ring(LoraArgs p) {
    typedef GroupedRing<LAY_NN, BM, BN, WM, WN, STAGES> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    lora_parts<E, BM, BN, WM, WN>(p, smem);
}
template <int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM *WN * 64, 1) k_lora_parts_any(LoraArgs p) {
    typedef GroupedAny<LAY_NN, BM, BN, WM, WN> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    lora_parts<E, BM, BN, WM, WN>(p, smem);
}

// low[row][c .. c + 7], summed over its parts; zero past the rank.
__device__ __forceinline__ void load_low(const LoraArgs &p, int row, int c, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = 0.0f;
    for (int i = 0; i < p.low_parts; i++) {
        const float *q = p.low + ((int64_t)i * p.M + row) * p.rank + c;
        if (c + 8 <= p.rank) {
            typedef float f32x4_ua __attribute__((ext_vector_type(4), aligned(4)));
            const f32x4_ua x = *(const f32x4_ua *)q, y = *(const f32x4_ua *)(q + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += x[e], v[4 + e] += y[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (c + e < p.rank) v[e] += q[e];
        }
    }
}

// acc += scale * low . up for the wave's rows from row0 and columns from col0.
// The columns of up[a] that the wave needs are staged in its own part of LDS
// (no barrier), 64 of the rank at a time.
template <int MI, int NI>
__device__ __forceinline__ void add_adapters(const LoraArgs &p, int row0, int col0, unsigned char *lds,
                                             f32x16 (&acc)[MI][NI]) {
    typedef Image<false, NI * 32> IU;  // 64 of the rank by the wave's columns
    const int lane = threadIdx.x & 63;
    int staged = -1, staged_c = 0;
#pragma unroll
    for (int mi = 0; mi < MI; mi++) {
        const int row = row0 + mi * 32 + (lane & 31);
        const int id = adapter_of(p, row);
        uint32_t left = (uint32_t)__ballot(id >= 0);  // both halves of the wave hold the same rows
        while (left) {
            const int a = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffs(left) - 1));
            const uint32_t mine = (uint32_t)__ballot(id == a);
            left &= ~mine;
            // the row's power of two: its largest finite |low| below 2^14
            float most = 0.0f;
            for (int c = (lane >> 5) * 8; c < p.rank; c += 16) {
                float v[8];
                load_low(p, min(row, p.M - 1), c, v);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float m = fabsf(v[e]);
                    most = m <= 3.402823466e38f ? fmaxf(most, m) : most;
                }
            }
            most = fmaxf(most, __shfl_xor(most, 32));
            const int ex = most > 0.0f ? ilogbf(most) - 13 : 0;
            f32x16 sum[NI];
#pragma unroll
            for (int ni = 0; ni < NI; ni++) sum[ni] = f32x16{};
            for (int c0 = 0; c0 < p.rank; c0 += 64) {
                if (staged != a || staged_c != c0) {
                    const unsigned char *up = p.up + (int64_t)a * p.stride_up;
#pragma unroll
                    for (int i = 0; i < IU::CHUNKS / 64; i++) {
                        const int q = i * 64 + lane, r = q / IU::CPR, c = ((q % IU::CPR) ^ IU::swz(r)) * 8;
                        lds_write16(lds + q * 16, load_chunk(up, p.ld_up, c0 + r, p.rank, col0 + c, p.N));
                    }
                    staged = a, staged_c = c0;
                    __builtin_amdgcn_wave_barrier();
                }
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    if (c0 + s * 16 >= p.rank) break;
                    float v[8];
                    load_low(p, min(row, p.M - 1), c0 + s * 16 + (lane >> 5) * 8, v);
                    f16x8 hi, rest;
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const float x = ldexpf(v[e], -ex);
                        hi[e] = (_Float16)x;
                        const float d = x - (float)hi[e];
                        rest[e] = fabsf(x) <= 65504.0f ? (_Float16)d : (_Float16)0.0f;  // not finite: all in hi
                    }
#pragma unroll
                    for (int ni = 0; ni < NI; ni++) {
                        const u32x4 u = IU::read(lds, lane, ni * 32, s);
                        sum[ni] = Mfma<DT_F16>::mac_sub(__builtin_bit_cast(u32x4, hi), u, sum[ni], 0);
                        sum[ni] = Mfma<DT_F16>::mac_sub(__builtin_bit_cast(u32x4, rest), u, sum[ni], 0);
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
            const float scale = p.scale ? p.scale[a] : 1.0f;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int r = (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
                const int e = __shfl(ex, r);
                if ((mine >> r) & 1) {
#pragma unroll
                    for (int ni = 0; ni < NI; ni++) acc[mi][ni][v] += scale * ldexpf(sum[ni][v], e);
                }
            }
        }
    }
}

// The second launch for many rows: the shared product's tiles with the
// adapters added to the accumulators.
template <class E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void lora_main(const LoraArgs &p, unsigned char *smem) {
    static_assert(E::SMEM >= WM * WN * Image<false, E::NI * 32>::BYTES, "LDS for up");
    const int total = p.row_tiles * p.col_tiles, per = (total + 7) >> 3;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
    int tm, tn;
    order_tile(id, p.row_tiles, p.col_tiles, tm, tn);
    poison_lds<E::SMEM, E::NT>(p.flags, smem);
    f32x16 acc[E::MI][E::NI];
    clear_acc(acc);
    E::run(p.A, p.lda, p.B, p.ldb, tm * BM, p.M, tn * BN, p.N, 0, p.K, smem, acc);
    __syncthreads();  // every wave is done with the tiles in LDS
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = tm * BM + (wave % WM) * E::WTM, col0 = tn * BN + (wave / WM) * E::WTN;
    add_adapters<E::MI, E::NI>(p, row0, col0, smem + wave * Image<false, E::NI * 32>::BYTES, acc);
    store_tile<E::MI, E::NI>((unsigned char *)p.C, p.ldc, row0, p.M, col0, p.N, acc);
}

template <int BM, int BN, int WM, int WN, int STAGES>
__global__ void __launch_bounds__(WM *WN * 64, 1) k_lora_main_ring(LoraArgs p) {
    typedef GroupedRing<LAY_NN, BM, BN, WM, WN, STAGES> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    lora_main<E, BM, BN, WM, WN>(p, smem);
}
template <int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM *WN * 64, 1) k_lora_main_any(LoraArgs p) {
    typedef GroupedAny<LAY_NN, BM, BN, WM, WN> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    lora_main<E, BM, BN, WM, WN>(p, smem);
}

// The second launch for few rows: C[t][n] = the shared product's parts, in
// order, and scale * sum_c low[t][c] * up[c][n].  A thread owns V columns of
// JOIN_ROWS rows; neighbouring rows with the same adapter share up's loads.
constexpr int JOIN_THREADS = 256, JOIN_ROWS = 4;

template <int V>
__global__ void __launch_bounds__(JOIN_THREADS) k_lora_join(LoraArgs p) {
    __shared__ float low[JOIN_ROWS][TDG_LORA_MAX_RANK];
    const int t0 = blockIdx.x * JOIN_ROWS, tid = threadIdx.x;
    const int64_t n = ((int64_t)blockIdx.y * JOIN_THREADS + tid) * V;
    int id[JOIN_ROWS];
#pragma unroll
    for (int j = 0; j < JOIN_ROWS; j++) {
        id[j] = __builtin_amdgcn_readfirstlane(adapter_of(p, t0 + j));
        if (id[j] >= 0)
            for (int c = tid; c < p.rank; c += JOIN_THREADS) {
                float s = 0.0f;
                for (int i = 0; i < p.low_parts; i++) s += p.low[((int64_t)i * p.M + t0 + j) * p.rank + c];
                low[j][c] = s;
            }
    }
    __syncthreads();
    if (n >= p.N) return;
    typedef float fv __attribute__((ext_vector_type(V), aligned(4)));
    typedef _Float16 hv __attribute__((ext_vector_type(V), aligned(2)));
    fv sum[JOIN_ROWS];
#pragma unroll
    for (int j = 0; j < JOIN_ROWS; j++) {
        fv s = {};
        if (t0 + j < p.M)
            for (int i = 0; i < p.parts; i++) s += *(const fv *)(p.part + ((int64_t)i * p.M + t0 + j) * p.N + n);
        sum[j] = s;
    }
    fv side[JOIN_ROWS] = {};
    for (int c = 0; c < p.rank; c++) {
        fv u = {};
#pragma unroll
        for (int j = 0; j < JOIN_ROWS; j++) {
            if (id[j] < 0) continue;
            if (j == 0 || id[j] != id[j - 1]) {
                const hv h = *(const hv *)(p.up + (int64_t)id[j] * p.stride_up + (int64_t)c * p.ld_up + n * 2);
#pragma unroll
                for (int q = 0; q < V; q++) u[q] = (float)h[q];
            }
#pragma unroll
            for (int q = 0; q < V; q++) side[j][q] = fmaf(low[j][c], u[q], side[j][q]);
        }
    }
#pragma unroll
    for (int j = 0; j < JOIN_ROWS; j++) {
        if (t0 + j >= p.M) continue;
        if (id[j] >= 0) {
            const float scale = p.scale ? p.scale[id[j]] : 1.0f;
#pragma unroll
            for (int q = 0; q < V; q++) sum[j][q] = fmaf(scale, side[j][q], sum[j][q]);
        }
        *(fv *)((unsigned char *)p.C + (int64_t)(t0 + j) * p.ldc + n * 4) = sum[j];
    }
}

// ------------------------------------------------------------------ host side

int launch(const void *fn, dim3 grid, int threads, LoraArgs *args, void *stream) {
    void *kargs[] = {args};
    if (hipLaunchKernel(fn, grid, dim3((unsigned)threads), kargs, 0, (hipStream_t)stream) != hipSuccess)
        return TDG_ERR_LAUNCH;
    if (hipGetLastError() != hipSuccess) return TDG_ERR_LAUNCH;
    return TDG_OK;
}

bool sizes_ok(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank) {
    return size_ok(M) && size_ok(N) && size_ok(K) && size_ok(adapters) && rank >= 0 && rank <= TDG_LORA_MAX_RANK;
}

// How the work is cut; a function of the sizes alone, as the workspace is.
struct Plan {
    bool few;             // few rows: parts of the shared product and a join
    int bm;               // row tile of the first launch
    int64_t parts, k_per_part, low_parts, low_k_per_part;
    uint64_t low_at, bytes;  // workspace: parts, then low
};

constexpr int64_t kFewRows = 256;

Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t rank) {
    Plan p = {};
    const int64_t kt = ceil_quot(K, 64);
    p.few = M <= kFewRows;
    p.bm = M <= 32 ? 32 : 64;
    const int64_t row_tiles = ceil_quot(M, p.bm);
    auto cut = [&](int64_t tiles, int64_t want, int64_t *parts, int64_t *per) {
        int64_t n = ceil_quot(want, tiles > 0 ? tiles : 1);
        n = n > 8 ? 8 : n;                       // the parts are read again
        n = n * 4 > kt ? (kt + 3) / 4 : n;       // a slice is four K tiles or more
        n = n < 1 ? 1 : n;
        *per = ceil_quot(kt, n);
        *parts = *per > 0 ? ceil_quot(kt, *per) : 1;
    };
    if (p.few) cut(row_tiles * ceil_quot(N, 64), 512, &p.parts, &p.k_per_part);
    cut(row_tiles * ceil_quot(rank, 64), 256, &p.low_parts, &p.low_k_per_part);
    p.low_at = p.few ? (uint64_t)p.parts * M * N * 4 : 0;
    p.low_at = (p.low_at + 15) / 16 * 16;
    p.bytes = p.low_at + (uint64_t)p.low_parts * M * rank * 4;
    return p;
}

}  // namespace

extern "C" {

int tdg_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank, size_t *bytes) {
    if (!bytes || !sizes_ok(M, N, K, adapters, rank)) return TDG_ERR_INVALID_ARG;
    const bool side = adapters > 0 && rank > 0 && K > 0 && M > 0 && N > 0;
    *bytes = side ? (size_t)make_plan(M, N, K, rank).bytes : 0;
    return TDG_OK;
}

int gemm_f16f32_lora(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, const uint16_t *B,
                     int64_t ldb, int64_t adapters, int64_t rank, const uint16_t *down, int64_t ld_down,
                     int64_t stride_down, const uint16_t *up, int64_t ld_up, int64_t stride_up,
                     const int32_t *adapter, const float *scale, float *C, int64_t ldc, void *workspace,
                     size_t workspace_bytes, void *stream) {
    size_t need = 0;
    if (tdg_lora_workspace(M, N, K, adapters, rank, &need) != TDG_OK) return TDG_ERR_INVALID_ARG;
    int rc = validate_gemm(TDG_DTYPE_F16F32, M, N, K, A, lda, B, ldb, C, ldc);
    if (rc != TDG_OK) return rc;
    if (!stack_ok(down, adapters, stride_down, K, rank, ld_down, 2, false) ||
        !stack_ok(up, adapters, stride_up, rank, N, ld_up, 2, false))
        return TDG_ERR_INVALID_ARG;
    if (!aligned_to(A, 2) || !aligned_to(B, 2) || !aligned_to(down, 2) || !aligned_to(up, 2) || !aligned_to(C, 4) ||
        !aligned_to(adapter, 4) || !aligned_to(scale, 4))
        return TDG_ERR_INVALID_ARG;
    const bool side = adapters > 0 && rank > 0 && K > 0 && M > 0 && N > 0;
    if (side && !adapter) return TDG_ERR_INVALID_ARG;
    const uint64_t c_len = span_bytes(M, N, ldc, 4);
    const void *in[6] = {A, B, down, up, adapter, scale};
    const uint64_t in_len[6] = {span_bytes(M, K, lda, 2), span_bytes(K, N, ldb, 2),
                                span_bytes(K, rank, ld_down, 2, adapters, stride_down),
                                span_bytes(rank, N, ld_up, 2, adapters, stride_up), (uint64_t)M * 4,
                                (uint64_t)adapters * 4};
    if (side && need && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16)))
        return TDG_ERR_INVALID_ARG;
    for (int i = 0; i < 6; i++)
        if (overlaps(C, c_len, in[i], in_len[i]) || (side && overlaps(workspace, need, in[i], in_len[i])))
            return TDG_ERR_INVALID_ARG;
    if (side && overlaps(workspace, need, C, c_len)) return TDG_ERR_INVALID_ARG;
    if (!side) return gemm_f16f32_pipelined(M, N, K, A, lda, B, ldb, C, ldc, stream);

    const Plan plan = make_plan(M, N, K, rank);
    LoraArgs p;
    p.A = (const unsigned char *)A, p.B = (const unsigned char *)B;
    p.down = (const unsigned char *)down, p.up = (const unsigned char *)up;
    p.adapter = adapter, p.scale = scale, p.C = C;
    p.part = (float *)workspace, p.low = (float *)((unsigned char *)workspace + plan.low_at);
    p.lda = lda * 2, p.ldb = ldb * 2, p.ldc = ldc * 4;
    p.ld_down = ld_down * 2, p.stride_down = stride_down * 2, p.ld_up = ld_up * 2, p.stride_up = stride_up * 2;
    p.M = (int)M, p.N = (int)N, p.K = (int)K, p.adapters = (int)adapters, p.rank = (int)rank;
    p.flags = debug_flags_now();
    p.parts = (int)plan.parts, p.k_per_part = (int)plan.k_per_part;
    p.low_parts = (int)plan.low_parts, p.low_k_per_part = (int)plan.low_k_per_part;
    // The DMA copies whole 16-byte chunks and reaches a tile's rows with
    // 32-bit byte offsets.
    const int64_t far = (int64_t)UINT32_MAX / 2 / 256 - 256;
    const bool near = lda <= far && ldb <= far && ld_down <= far;
    const bool ring = near && K % 8 == 0 && N % 8 == 0 && rank % 8 == 0;
    const bool ring_main = near && K % 8 == 0 && N % 8 == 0;

    const int64_t low_tiles = ceil_quot(M, plan.bm);
    p.low_cols = (int)ceil_quot(rank, 64);
    p.low_lanes = low_tiles >= 64 ? 4 : plan.bm;
    p.row_tiles = (int)low_tiles, p.col_tiles = (int)ceil_quot(N, 64);
    const int64_t shared = plan.few ? ceil_quot(low_tiles * p.col_tiles * plan.parts, 8) * 8 : 0;
    const int64_t wgs = shared + low_tiles * plan.low_parts * p.low_cols * p.low_lanes;
    if (wgs > (int64_t)UINT32_MAX / 256 || ceil_quot(M, 64) > INT32_MAX / 8 / ceil_quot(N, 64) ||
        ceil_quot(N, JOIN_THREADS) > 65535)
        return TDG_ERR_UNSUPPORTED;
    p.shared_wgs = (int)shared;
    rc = device_check();
    if (rc != TDG_OK) return rc;
    const void *fn;
    if (plan.bm == 32)
        fn = ring ? (const void *)&k_lora_parts_ring<32, 64, 1, 2, 4> : (const void *)&k_lora_parts_any<32, 64, 1, 2>;
    else
        fn = ring ? (const void *)&k_lora_parts_ring<64, 64, 2, 2, 4> : (const void *)&k_lora_parts_any<64, 64, 2, 2>;
    rc = launch(fn, dim3((unsigned)wgs), plan.bm == 32 ? 128 : 256, &p, stream);
    if (rc != TDG_OK) return rc;
    if (plan.few) {
        const bool v4 = N % 4 == 0;
        fn = v4 ? (const void *)&k_lora_join<4> : (const void *)&k_lora_join<1>;
        return launch(fn, dim3((unsigned)ceil_quot(M, JOIN_ROWS), (unsigned)ceil_quot(N, JOIN_THREADS * (v4 ? 4 : 1))),
                      JOIN_THREADS, &p, stream);
    }
    const bool big = ring_main && ceil_quot(M, 256) * ceil_quot(N, 256) >= 128;
    const int bt = big ? 256 : 128;
    p.row_tiles = (int)ceil_quot(M, bt), p.col_tiles = (int)ceil_quot(N, bt);
    const int64_t grid = ceil_quot((int64_t)p.row_tiles * p.col_tiles, 8) * 8;
    fn = big         ? (const void *)&k_lora_main_ring<256, 256, 2, 4, 2>
         : ring_main ? (const void *)&k_lora_main_ring<128, 128, 2, 2, 2>
                     : (const void *)&k_lora_main_any<128, 128, 2, 2>;
    return launch(fn, dim3((unsigned)grid), big ? 512 : 256, &p, stream);
}

}  // extern "C"
