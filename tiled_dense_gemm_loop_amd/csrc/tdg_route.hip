// tdg_route.hip -- rows sorted by expert and back: the plan, the dispatch,
// the weighted combine and the combine's gradient.
//
// T tokens choose top_k experts each; entry e = t * top_k + j is token t's
// j-th choice.  The plan is a stable counting sort of the kept entries (those
// with an id in [0, E)) by expert:
//   slot(e)  = offsets[id(e)] + #{e' < e : id(e') = id(e)},   -1 when dropped,
//   order[slot(e)] = e,   offsets[g] = #{kept e : id(e) < g}.
// The rows then move by slot, token by token, so that a token's row is read
// (dispatch) or written (combine) once however many experts it has:
//   dispatch  out[slot(t, j)] = x[t]
//   combine   y[t] = sum_j w[t][j] * z[slot(t, j)]              (j ascending, FP32)
//   gradient  dz[slot(t, j)] = w[t][j] * dy[t],  dw[t][j] = <dy[t], z[slot(t, j)]>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tdg_check.h"
#include "tdg_internal.h"
#include "tdgemm.h"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_ua __attribute__((ext_vector_type(4), aligned(1)));  // any byte alignment
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f16x4 f16x4_ua __attribute__((aligned(2)));
typedef f16x8 f16x8_ua __attribute__((aligned(2)));
typedef f32x4 f32x4_ua __attribute__((aligned(4)));

// ------------------------------------------------------------------ the plan

constexpr int MAX_EXPERTS = 1024;
constexpr int PLAN_THREADS = 1024;
// Up to PLAN_ALONE entries one workgroup does it all (7.9 us for 4096, as two
// launches take); above, 1024 or 2048 entries per workgroup, or more where
// that would be over PLAN_BLOCKS (us for 16000 and 65536 entries of 64
// experts: 8.5 and 9.5 by 1024, 9.3 and 9.7 by 2048, 10.9 and 11.4 by 4096;
// for 262144: 13.3, 11.8, 12.5).
constexpr int PLAN_ALONE = 4096, PLAN_BLOCKS = 256;

struct RouteArgs {
    const int32_t *ids;
    int64_t ld_ids;
    int32_t *offsets, *order, *slots;
    int32_t *counts;  // blocks x experts (more than one workgroup)
    int entries, top_k, experts, per_block, blocks;
};

__device__ __forceinline__ int entry_id(const RouteArgs &a, int e) {
    if (a.ld_ids == a.top_k) return a.ids[e];
    const int t = e / a.top_k;
    return a.ids[(int64_t)t * a.ld_ids + (e - t * a.top_k)];
}

// First of two launches for many entries: each workgroup counts its entries
// per expert.
__global__ void __launch_bounds__(PLAN_THREADS) k_route_count(RouteArgs a) {
    __shared__ int cnt[MAX_EXPERTS];
    const int tid = threadIdx.x;
    for (int e = tid; e < a.experts; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * a.per_block, hi = min(a.entries, lo + a.per_block);
    for (int e = lo + tid; e < hi; e += blockDim.x) {
        const int id = entry_id(a, e);
        if ((unsigned)id < (unsigned)a.experts) atomicAdd(&cnt[id], 1);
    }
    __syncthreads();
    for (int e = tid; e < a.experts; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.experts + e] = cnt[e];
}

// The sort itself.  A workgroup owns a run of entries and each of its waves a
// run of those, so (wave, lane) order is entry order.  Ranks inside a wave
// come from ballots over the bits of the id: the lanes with the same id are
// found without any data-dependent order, so the plan is the same every time.
__global__ void __launch_bounds__(PLAN_THREADS) k_route_place(RouteArgs a) {
    extern __shared__ int lds[];
    const int E = a.experts, tid = threadIdx.x, nt = blockDim.x;
    const int waves = nt >> 6, lane = tid & 63, wave = tid >> 6;
    int *cnt = lds;              // waves x E: entries of the wave, then its next slot
    int *total = cnt + waves * E;  // E: all entries of the expert, then its first slot
    int *before = total + E;     // E: those of earlier workgroups
    int *wsum = before + E;      // waves + 1
    for (int i = tid; i < (waves + 2) * E; i += nt) cnt[i] = 0;
    __syncthreads();

    const int per_wave = ((a.per_block + waves * 64 - 1) / (waves * 64)) * 64;
    const int b_lo = blockIdx.x * a.per_block, b_hi = min(a.entries, b_lo + a.per_block);
    const int w_lo = min(b_hi, b_lo + wave * per_wave), w_hi = min(b_hi, w_lo + per_wave);
    for (int e = w_lo + lane; e < w_hi; e += 64) {
        const int id = entry_id(a, e);
        if ((unsigned)id < (unsigned)E) atomicAdd(&cnt[wave * E + id], 1);
    }
    if (a.blocks > 1) {
        // column sums of the counts of all workgroups, and of the earlier ones
        const int groups = max(1, nt / E);
        const int g = tid / E, e0 = tid - g * E;
        if (g < groups) {
            for (int e = e0; e < E; e += (groups == 1 ? nt : E)) {
                int all = 0, pre = 0;
                for (int b = g; b < a.blocks; b += groups) {
                    const int c = a.counts[(int64_t)b * E + e];
                    all += c;
                    if (b < (int)blockIdx.x) pre += c;
                }
                atomicAdd(&total[e], all);
                atomicAdd(&before[e], pre);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += nt) {
        int run = 0;
        for (int w = 0; w < waves; w++) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        if (a.blocks == 1) total[e] = run;
    }
    __syncthreads();
    // exclusive sum over the experts, a run of them per thread
    const int per = (E + nt - 1) / nt;
    const int e_lo = min(E, tid * per), e_hi = min(E, e_lo + per);
    int mine = 0;
    for (int e = e_lo; e < e_hi; e++) mine += total[e];
    int incl = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(incl, d);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int start = incl - mine;
    for (int w = 0; w < wave; w++) start += wsum[w];
    int kept = 0;
    for (int w = 0; w < waves; w++) kept += wsum[w];
    for (int e = e_lo; e < e_hi; e++) {
        const int c = total[e];
        total[e] = start;
        if (blockIdx.x == 0) a.offsets[e] = start;
        start += c;
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[E] = kept;
    __syncthreads();
    for (int i = tid; i < waves * E; i += nt) {
        const int e = i % E;
        cnt[i] += total[e] + before[e];
    }
    __syncthreads();

    int bits = 0;
    while ((1 << bits) < E) bits++;
    for (int e0 = w_lo; e0 < w_hi; e0 += 64) {
        const int e = e0 + lane;
        const int id = e < w_hi ? entry_id(a, e) : -1;
        const bool ok = (unsigned)id < (unsigned)E;
        unsigned long long same = __ballot(ok);
        for (int b = 0; b < bits; b++) {
            const bool one = (id >> b) & 1;
            const unsigned long long m = __ballot(one);
            same &= one ? m : ~m;
        }
        int slot = -1;
        int first = 0;
        if (ok) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int leader = __ffsll((unsigned long long)same) - 1;
            if (lane == leader) first = atomicAdd(&cnt[wave * E + id], __popcll(same));
            slot = __shfl(first, leader) + rank;
            a.order[slot] = e;
        }
        if (e < w_hi) a.slots[e] = slot;
    }
    // the order's tail, behind the last kept entry
    for (int64_t i = (int64_t)kept + (int64_t)blockIdx.x * nt + tid; i < a.entries; i += (int64_t)gridDim.x * nt)
        a.order[i] = -1;
}

// ------------------------------------------------------------------ row movement

constexpr int ROW_THREADS = 256;

// Rows of `units` 16-byte (or, for the last, shorter) pieces.  A workgroup is
// ROW_THREADS / tx token rows of tx threads, and covers tx pieces of each; tx
// is the power of two that covers a row, at most ROW_THREADS, and long rows
// are cut into `segs` segments, so that a few tokens still spread over many
// CUs.  A token's segments are neighbours in the grid: with all tokens' first
// segments together, rows whose length is a power of two keep a part of the
// memory channels busy at a time (4096 tokens, 4 rows of 16 KiB each: dispatch
// 79 us against 72, combine 96 against 72).  Rows off the 16-byte grid are the
// other way round (rows 4 bytes shorter: combine 84 us with the segments
// apart, 91 with them together; dispatch of 8191 FP16 columns 89 and 97).
// Pieces start at any byte address: the chip runs in unaligned-access mode.
struct RowsArgs {
    const unsigned char *tok;  // token rows read (dispatch: x, gradient: dy)
    const unsigned char *row;  // sorted rows read (z)
    unsigned char *tok_out;    // combine: y
    unsigned char *row_out;    // dispatch: out, gradient: dz
    int64_t ld_tok, ld_row, ld_out;  // bytes
    const int32_t *slots;
    const float *w;
    int64_t ld_w;
    float *dw;
    int64_t ld_dw;
    int tokens, top_k, cols, rows;
    int tx_log2, segs;
    int apart;  // a token's segments lie apart in the grid
};

// The block of token rows (x) and the segment (y) of this workgroup.
__device__ __forceinline__ int2 row_block(const RowsArgs &a) {
    const int per = a.apart ? gridDim.x / a.segs : a.segs;
    const int q = blockIdx.x / per, r = blockIdx.x - q * per;
    return a.apart ? make_int2(r, q) : make_int2(q, r);
}

template <int ES>
__global__ void __launch_bounds__(ROW_THREADS) k_rows_dispatch(RowsArgs a) {
    const int tx = 1 << a.tx_log2;
    const int2 at = row_block(a);
    const int t = at.x * (ROW_THREADS >> a.tx_log2) + (threadIdx.x >> a.tx_log2);
    if (t >= a.tokens) return;
    constexpr int EPC = 16 / ES;
    const int64_t col = ((int64_t)at.y * tx + (threadIdx.x & (tx - 1))) * EPC;
    if (col >= a.cols) return;
    const unsigned char *src = a.tok + (int64_t)t * a.ld_tok + col * ES;
    const int32_t *slots = a.slots + (int64_t)t * a.top_k;
    if (col + EPC <= a.cols) {
        const u32x4 v = *(const u32x4_ua *)src;
        for (int j = 0; j < a.top_k; j++) {
            const int s = slots[j];
            if ((unsigned)s < (unsigned)a.rows) *(u32x4_ua *)(a.row_out + (int64_t)s * a.ld_out + col * ES) = v;
        }
    } else {
        typedef typename std::conditional<ES == 2, uint16_t, uint32_t>::type T;
        for (int j = 0; j < a.top_k; j++) {
            const int s = slots[j];
            if ((unsigned)s >= (unsigned)a.rows) continue;
            T *dst = (T *)(a.row_out + (int64_t)s * a.ld_out);
            for (int64_t c = col; c < a.cols; c++) dst[c] = ((const T *)(a.tok + (int64_t)t * a.ld_tok))[c];
        }
    }
}

// What is loaded, and not used, in place of a row that is not there.
static __device__ __attribute__((aligned(16))) const uint32_t no_row[8] = {};

// V consecutive elements as floats, and back (rounded to nearest even).
template <typename T, int V>
__device__ __forceinline__ void load_v(const unsigned char *p, float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            const f32x4 x = *(const f32x4_ua *)(p + 4 * q);
            v[q] = x[0], v[q + 1] = x[1], v[q + 2] = x[2], v[q + 3] = x[3];
        }
    } else if constexpr (V == 8) {
        const f16x8 x = *(const f16x8_ua *)p;
#pragma unroll
        for (int q = 0; q < 8; q++) v[q] = (float)x[q];
    } else {
        const f16x4 x = *(const f16x4_ua *)p;
#pragma unroll
        for (int q = 0; q < 4; q++) v[q] = (float)x[q];
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(unsigned char *p, const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int q = 0; q < V; q += 4) *(f32x4_ua *)(p + 4 * q) = f32x4{v[q], v[q + 1], v[q + 2], v[q + 3]};
    } else if constexpr (V == 8) {
        f16x8 x;
#pragma unroll
        for (int q = 0; q < 8; q++) x[q] = (_Float16)v[q];
        *(f16x8_ua *)p = x;
    } else {
        f16x4 x;
#pragma unroll
        for (int q = 0; q < 4; q++) x[q] = (_Float16)v[q];
        *(f16x4_ua *)p = x;
    }
}

// Sorted rows of type Z, token rows of type Y.  A thread owns 16 bytes of the
// sorted rows (4 FP32 or 8 FP16 columns).  The sum is kept in FP32, in the
// order of j, and rounded once.
template <typename Z, typename Y>
__global__ void __launch_bounds__(ROW_THREADS) k_rows_combine(RowsArgs a) {
    constexpr int V = 16 / sizeof(Z);
    const int tx = 1 << a.tx_log2;
    const int2 at = row_block(a);
    const int t = at.x * (ROW_THREADS >> a.tx_log2) + (threadIdx.x >> a.tx_log2);
    if (t >= a.tokens) return;
    const int64_t col = ((int64_t)at.y * tx + (threadIdx.x & (tx - 1))) * V;
    if (col >= a.cols) return;
    const int32_t *slots = a.slots + (int64_t)t * a.top_k;
    const float *w = a.w ? a.w + (int64_t)t * a.ld_w : nullptr;
    unsigned char *dst = a.tok_out + (int64_t)t * a.ld_tok + col * sizeof(Y);
    const unsigned char *none = (const unsigned char *)no_row;
    if (col + V <= a.cols) {
        float acc[V] = {};
        // Four rows' loads go out together: one at a time, the loads in flight
        // on the chip are too few for HBM's rate.
        for (int j0 = 0; j0 < a.top_k; j0 += 4) {
            int s[4];
            float wj[4], z[4][V];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                s[j] = j0 + j < a.top_k ? slots[j0 + j] : -1;
                wj[j] = w && j0 + j < a.top_k ? w[j0 + j] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
                load_v<Z, V>((unsigned)s[j] < (unsigned)a.rows ? a.row + (int64_t)s[j] * a.ld_row + col * sizeof(Z) : none,
                             z[j]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if ((unsigned)s[j] >= (unsigned)a.rows) continue;
#pragma unroll
                for (int q = 0; q < V; q++) acc[q] = fmaf(wj[j], z[j][q], acc[q]);
            }
        }
        store_v<Y, V>(dst, acc);
    } else {
        for (int c = (int)col; c < a.cols; c++) {
            float acc = 0.0f;
            for (int j = 0; j < a.top_k; j++) {
                const int s = slots[j];
                if ((unsigned)s >= (unsigned)a.rows) continue;
                acc = fmaf(w ? w[j] : 1.0f, (float)((const Z *)(a.row + (int64_t)s * a.ld_row))[c], acc);
            }
            ((Y *)(a.tok_out + (int64_t)t * a.ld_tok))[c] = (Y)acc;
        }
    }
}

// A token and a group of J choices belong to 1 << tx_log2 threads, one to four
// waves: dy's row is read once for the J rows of z and dz, and the J dot
// products are reduced in a fixed order (columns by thread, lanes by a
// butterfly, waves in order).  Short rows take the fewest waves that cover them.
template <typename Z, typename Y, int J>
__global__ void __launch_bounds__(ROW_THREADS) k_rows_combine_grad(RowsArgs a) {
    constexpr int V = 16 / sizeof(Z);
    __shared__ float part[J][ROW_THREADS / 64];
    const int tx = 1 << a.tx_log2, tid = threadIdx.x & (tx - 1);
    const int t_all = blockIdx.x * (ROW_THREADS >> a.tx_log2) + (threadIdx.x >> a.tx_log2);
    const bool on = t_all < a.tokens;
    const int t = on ? t_all : 0, j0 = blockIdx.y * J;
    const int nj = on ? min(J, a.top_k - j0) : 0;
    const unsigned char *dy = a.tok + (int64_t)t * a.ld_tok;
    int slot[J];
    float w[J], dot[J];
#pragma unroll
    for (int j = 0; j < J; j++) {
        slot[j] = j < nj ? a.slots[(int64_t)t * a.top_k + j0 + j] : -1;
        if ((unsigned)slot[j] >= (unsigned)a.rows) slot[j] = -1;
        w[j] = slot[j] >= 0 && a.w ? a.w[(int64_t)t * a.ld_w + j0 + j] : 1.0f;
        dot[j] = 0.0f;
    }
    // Neighbouring tokens start in different segments of their rows: see above.
    const int segs = on ? (a.cols + tx * V - 1) / (tx * V) : 0;
    int seg = segs > 0 ? t % segs : 0;
    for (int i = 0; i < segs; i++, seg = seg + 1 == segs ? 0 : seg + 1) {
        const int64_t col = ((int64_t)seg * tx + tid) * V;
        if (col >= a.cols) continue;
        if (col + V <= a.cols) {
            float g[V];
            load_v<Y, V>(dy + col * sizeof(Y), g);
            float z[J][V];
#pragma unroll
            for (int j = 0; j < J; j++)
                load_v<Z, V>(slot[j] >= 0 ? a.row + (int64_t)slot[j] * a.ld_row + col * sizeof(Z)
                                          : (const unsigned char *)no_row,
                             z[j]);
#pragma unroll
            for (int j = 0; j < J; j++) {
                if (slot[j] < 0) continue;
#pragma unroll
                for (int q = 0; q < V; q++) {
                    dot[j] = fmaf(g[q], z[j][q], dot[j]);
                    z[j][q] = w[j] * g[q];
                }
                store_v<Z, V>(a.row_out + (int64_t)slot[j] * a.ld_out + col * sizeof(Z), z[j]);
            }
        } else {
            for (int c = (int)col; c < a.cols; c++) {
                const float g = (float)((const Y *)dy)[c];
#pragma unroll
                for (int j = 0; j < J; j++) {
                    if (slot[j] < 0) continue;
                    dot[j] = fmaf(g, (float)((const Z *)(a.row + (int64_t)slot[j] * a.ld_row))[c], dot[j]);
                    ((Z *)(a.row_out + (int64_t)slot[j] * a.ld_out))[c] = (Z)(w[j] * g);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < J; j++) {
        for (int d = 32; d > 0; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
        if ((threadIdx.x & 63) == 0) part[j][threadIdx.x >> 6] = dot[j];
    }
    __syncthreads();
    if (tid < nj) {
        float s = 0.0f;
        for (int i = 0; i < tx >> 6; i++) s += part[tid][(threadIdx.x - tid) / 64 + i];
        a.dw[(int64_t)t * a.ld_dw + j0 + tid] = s;
    }
}

// ------------------------------------------------------------------ host side

int launch(const void *fn, dim3 grid, int threads, size_t lds, void *args, void *stream) {
    void *kargs[] = {args};
    if (hipLaunchKernel(fn, grid, dim3((unsigned)threads), kargs, lds, (hipStream_t)stream) != hipSuccess)
        return TDG_ERR_LAUNCH;
    if (hipGetLastError() != hipSuccess) return TDG_ERR_LAUNCH;
    return TDG_OK;
}

// At most 2^30 entries: the plan forms (first entry + run length) in 32 bits.
constexpr int64_t kMaxEntries = (int64_t)1 << 30;
bool entries_ok(int64_t tokens, int64_t top_k) {
    return tokens >= 0 && tokens <= kMaxEntries && top_k >= 1 && top_k <= kMaxEntries &&
           (tokens == 0 || top_k <= kMaxEntries / tokens);
}

// HIP counts a launch's threads in 32 bits.
bool grid_ok(int64_t blocks, int64_t threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

bool elem_ok(int e) { return e == TDG_ELEM_F16 || e == TDG_ELEM_F32; }
int64_t elem_bytes(int e) { return e == TDG_ELEM_F16 ? 2 : 4; }

// Threads along a row, as a power of two, and the grid.
bool rows_grid(int64_t tokens, int64_t cols, int per_thread, RowsArgs *a, dim3 *grid) {
    const int64_t units = tdg::ceil_quot(cols, per_thread);
    int lg = 0;
    while ((1 << lg) < ROW_THREADS && (1 << lg) < units) lg++;
    const int64_t segs = tdg::ceil_quot(units, (int64_t)1 << lg);
    const int64_t blocks = tdg::ceil_quot(tokens, ROW_THREADS >> lg) * segs;
    if (!grid_ok(blocks, ROW_THREADS)) return false;
    a->tx_log2 = lg, a->segs = (int)segs;
    a->apart = (((uintptr_t)a->row | (uintptr_t)a->row_out | (uint64_t)a->ld_row | (uint64_t)a->ld_out) & 15) != 0;
    *grid = dim3((unsigned)blocks);
    return true;
}

void plan_split(int64_t entries, int *per_block, int *blocks) {
    if (entries <= PLAN_ALONE) {
        *per_block = entries > 0 ? (int)entries : 1;
        *blocks = 1;
        return;
    }
    int64_t per = entries <= 16384 ? 1024 : 2048;
    if (tdg::ceil_quot(entries, per) > PLAN_BLOCKS)
        per = tdg::ceil_quot(tdg::ceil_quot(entries, PLAN_BLOCKS), 64) * 64;
    *per_block = (int)per;
    *blocks = entries > 0 ? (int)tdg::ceil_quot(entries, per) : 1;
}

}  // namespace

extern "C" {

int tdg_route_workspace(int64_t tokens, int64_t top_k, int64_t experts, size_t *bytes) {
    if (!bytes || !entries_ok(tokens, top_k) || experts < 1 || experts > MAX_EXPERTS) return TDG_ERR_INVALID_ARG;
    int per_block, blocks;
    plan_split(tokens * top_k, &per_block, &blocks);
    *bytes = blocks > 1 ? (size_t)blocks * (size_t)experts * sizeof(int32_t) : 0;
    return TDG_OK;
}

int tdg_route_plan(int64_t tokens, int64_t top_k, int64_t experts, const int32_t *ids, int64_t ld_ids,
                   int32_t *offsets, int32_t *order, int32_t *slots, void *workspace, size_t workspace_bytes,
                   void *stream) {
    size_t need = 0;
    if (tdg_route_workspace(tokens, top_k, experts, &need) != TDG_OK) return TDG_ERR_INVALID_ARG;
    const int64_t n = tokens * top_k;
    if (!tdg::matrix_ok(ids, tokens, top_k, ld_ids, 4) || !offsets || (n > 0 && (!order || !slots)))
        return TDG_ERR_INVALID_ARG;
    if (!tdg::aligned_to(ids, 4) || !tdg::aligned_to(offsets, 4) || !tdg::aligned_to(order, 4) ||
        !tdg::aligned_to(slots, 4))
        return TDG_ERR_INVALID_ARG;
    if (need && (!workspace || workspace_bytes < need || !tdg::aligned_to(workspace, 4))) return TDG_ERR_INVALID_ARG;
    const void *out[4] = {offsets, order, slots, workspace};
    const uint64_t len[4] = {(uint64_t)(experts + 1) * 4, (uint64_t)n * 4, (uint64_t)n * 4, (uint64_t)need};
    const uint64_t ids_len = tdg::span_bytes(tokens, top_k, ld_ids, 4);
    for (int i = 0; i < 4; i++) {
        if (tdg::overlaps(out[i], len[i], ids, ids_len)) return TDG_ERR_INVALID_ARG;
        for (int j = 0; j < i; j++)
            if (tdg::overlaps(out[i], len[i], out[j], len[j])) return TDG_ERR_INVALID_ARG;
    }
    const int rc = tdg::device_check();
    if (rc != TDG_OK) return rc;
    RouteArgs a;
    a.ids = ids, a.ld_ids = ld_ids, a.offsets = offsets, a.order = order, a.slots = slots;
    a.counts = (int32_t *)workspace;
    a.entries = (int)n, a.top_k = (int)top_k, a.experts = (int)experts;
    plan_split(n, &a.per_block, &a.blocks);
    if (a.blocks > 1) {
        const int rc2 = launch((const void *)&k_route_count, dim3((unsigned)a.blocks), PLAN_THREADS, 0, &a, stream);
        if (rc2 != TDG_OK) return rc2;
    }
    // one counter per wave and expert: 8 waves keep 1024 experts within 64 KiB
    const int threads = n <= 256 ? 256 : experts > 512 ? 512 : PLAN_THREADS;
    const size_t lds = ((size_t)(threads / 64 + 2) * experts + threads / 64 + 1) * sizeof(int);
    return launch((const void *)&k_route_place, dim3((unsigned)a.blocks), threads, lds, &a, stream);
}

int tdg_rows_dispatch(int elem, int64_t tokens, int64_t top_k, int64_t cols, const void *x, int64_t ldx,
                      const int32_t *slots, int64_t rows, void *out, int64_t ldo, void *stream) {
    if (!elem_ok(elem) || !entries_ok(tokens, top_k) || !tdg::size_ok(cols) || !tdg::size_ok(rows))
        return TDG_ERR_INVALID_ARG;
    const int64_t es = elem_bytes(elem);
    if (!tdg::matrix_ok(x, tokens, cols, ldx, es) || !tdg::matrix_ok(out, rows, cols, ldo, es) ||
        (tokens > 0 && !slots))
        return TDG_ERR_INVALID_ARG;
    const uint64_t out_len = tdg::span_bytes(rows, cols, ldo, es);
    if (tdg::overlaps(out, out_len, x, tdg::span_bytes(tokens, cols, ldx, es)) ||
        tdg::overlaps(out, out_len, slots, (uint64_t)(tokens * top_k) * 4))
        return TDG_ERR_INVALID_ARG;
    if (!tdg::aligned_to(x, es) || !tdg::aligned_to(out, es) || !tdg::aligned_to(slots, 4)) return TDG_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0 || rows == 0) return TDG_OK;
    RowsArgs a = {};
    a.tok = (const unsigned char *)x, a.row_out = (unsigned char *)out;
    a.ld_tok = ldx * es, a.ld_out = ldo * es, a.slots = slots;
    a.tokens = (int)tokens, a.top_k = (int)top_k, a.cols = (int)cols, a.rows = (int)rows;
    dim3 grid;
    if (!rows_grid(tokens, cols, (int)(16 / es), &a, &grid)) return TDG_ERR_UNSUPPORTED;
    const int rc = tdg::device_check();
    if (rc != TDG_OK) return rc;
    const void *fn = elem == TDG_ELEM_F16 ? (const void *)&k_rows_dispatch<2> : (const void *)&k_rows_dispatch<4>;
    return launch(fn, grid, ROW_THREADS, 0, &a, stream);
}

int tdg_rows_combine(int row_elem, int token_elem, int64_t tokens, int64_t top_k, int64_t cols, const void *z,
                     int64_t ldz, int64_t rows, const int32_t *slots, const float *weights, int64_t ld_weights,
                     void *y, int64_t ldy, void *stream) {
    if (!elem_ok(row_elem) || !elem_ok(token_elem) || !entries_ok(tokens, top_k) || !tdg::size_ok(cols) ||
        !tdg::size_ok(rows))
        return TDG_ERR_INVALID_ARG;
    const int64_t zs = elem_bytes(row_elem), ys = elem_bytes(token_elem);
    if (!tdg::matrix_ok(z, rows, cols, ldz, zs) || !tdg::matrix_ok(y, tokens, cols, ldy, ys) ||
        (weights && !tdg::matrix_ok(weights, tokens, top_k, ld_weights, 4)) || (tokens > 0 && !slots))
        return TDG_ERR_INVALID_ARG;
    const uint64_t y_len = tdg::span_bytes(tokens, cols, ldy, ys);
    if (tdg::overlaps(y, y_len, z, tdg::span_bytes(rows, cols, ldz, zs)) ||
        tdg::overlaps(y, y_len, slots, (uint64_t)(tokens * top_k) * 4) ||
        tdg::overlaps(y, y_len, weights, tdg::span_bytes(tokens, top_k, ld_weights, 4)))
        return TDG_ERR_INVALID_ARG;
    if (!tdg::aligned_to(z, zs) || !tdg::aligned_to(y, ys) || !tdg::aligned_to(slots, 4) ||
        !tdg::aligned_to(weights, 4))
        return TDG_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return TDG_OK;
    RowsArgs a = {};
    a.row = (const unsigned char *)z, a.tok_out = (unsigned char *)y;
    a.ld_row = ldz * zs, a.ld_tok = ldy * ys, a.slots = slots, a.w = weights, a.ld_w = ld_weights;
    a.tokens = (int)tokens, a.top_k = (int)top_k, a.cols = (int)cols, a.rows = (int)rows;
    dim3 grid;
    if (!rows_grid(tokens, cols, (int)(16 / zs), &a, &grid)) return TDG_ERR_UNSUPPORTED;
    const int rc = tdg::device_check();
    if (rc != TDG_OK) return rc;
    const void *fn;
    if (row_elem == TDG_ELEM_F16)
        fn = token_elem == TDG_ELEM_F16 ? (const void *)&k_rows_combine<_Float16, _Float16>
                                        : (const void *)&k_rows_combine<_Float16, float>;
    else
        fn = token_elem == TDG_ELEM_F16 ? (const void *)&k_rows_combine<float, _Float16>
                                        : (const void *)&k_rows_combine<float, float>;
    return launch(fn, grid, ROW_THREADS, 0, &a, stream);
}

int tdg_rows_combine_grad(int row_elem, int token_elem, int64_t tokens, int64_t top_k, int64_t cols,
                          const void *dy, int64_t ldy, const void *z, int64_t ldz, int64_t rows,
                          const int32_t *slots, const float *weights, int64_t ld_weights, void *dz, int64_t lddz,
                          float *dweights, int64_t ld_dweights, void *stream) {
    if (!elem_ok(row_elem) || !elem_ok(token_elem) || !entries_ok(tokens, top_k) || !tdg::size_ok(cols) ||
        !tdg::size_ok(rows))
        return TDG_ERR_INVALID_ARG;
    const int64_t zs = elem_bytes(row_elem), ys = elem_bytes(token_elem);
    if (!tdg::matrix_ok(dy, tokens, cols, ldy, ys) || !tdg::matrix_ok(z, rows, cols, ldz, zs) ||
        !tdg::matrix_ok(dz, rows, cols, lddz, zs) ||
        (weights && !tdg::matrix_ok(weights, tokens, top_k, ld_weights, 4)) ||
        !tdg::matrix_ok(dweights, tokens, top_k, ld_dweights, 4) || (tokens > 0 && !slots))
        return TDG_ERR_INVALID_ARG;
    const void *in[4] = {dy, z, slots, weights};
    const uint64_t in_len[4] = {tdg::span_bytes(tokens, cols, ldy, ys), tdg::span_bytes(rows, cols, ldz, zs),
                                (uint64_t)(tokens * top_k) * 4, tdg::span_bytes(tokens, top_k, ld_weights, 4)};
    const uint64_t dz_len = tdg::span_bytes(rows, cols, lddz, zs);
    const uint64_t dw_len = tdg::span_bytes(tokens, top_k, ld_dweights, 4);
    for (int i = 0; i < 4; i++)
        if (tdg::overlaps(dz, dz_len, in[i], in_len[i]) || tdg::overlaps(dweights, dw_len, in[i], in_len[i]))
            return TDG_ERR_INVALID_ARG;
    if (tdg::overlaps(dz, dz_len, dweights, dw_len)) return TDG_ERR_INVALID_ARG;
    if (!tdg::aligned_to(z, zs) || !tdg::aligned_to(dz, zs) || !tdg::aligned_to(dy, ys) ||
        !tdg::aligned_to(slots, 4) || !tdg::aligned_to(weights, 4) || !tdg::aligned_to(dweights, 4))
        return TDG_ERR_INVALID_ARG;
    if (tokens == 0) return TDG_OK;
    RowsArgs a = {};
    a.tok = (const unsigned char *)dy, a.row = (const unsigned char *)z, a.row_out = (unsigned char *)dz;
    a.ld_tok = ldy * ys, a.ld_row = ldz * zs, a.ld_out = lddz * zs, a.slots = slots;
    a.w = weights, a.ld_w = ld_weights, a.dw = dweights, a.ld_dw = ld_dweights;
    a.tokens = (int)tokens, a.top_k = (int)top_k, a.cols = (int)cols, a.rows = (int)rows;
    const int J = top_k >= 5 ? 8 : top_k >= 3 ? 4 : top_k >= 2 ? 2 : 1;
    const int64_t gy = tdg::ceil_quot(top_k, J);
    // (12601 tokens x 8 rows of 177 FP16 columns: 62 us with a workgroup to
    // each token.)
    const int64_t units = tdg::ceil_quot(cols, 16 / zs);
    a.tx_log2 = units <= 64 ? 6 : units <= 128 ? 7 : 8;
    const int64_t gx = tdg::ceil_quot(tokens, ROW_THREADS >> a.tx_log2);
    if (gy > 65535 || !grid_ok(gx, ROW_THREADS)) return TDG_ERR_UNSUPPORTED;
    const int rc = tdg::device_check();
    if (rc != TDG_OK) return rc;
#define TDG_GRAD(Z, Y)                                                       \
    (J == 8   ? (const void *)&k_rows_combine_grad<Z, Y, 8>                  \
     : J == 4 ? (const void *)&k_rows_combine_grad<Z, Y, 4>                  \
     : J == 2 ? (const void *)&k_rows_combine_grad<Z, Y, 2>                  \
              : (const void *)&k_rows_combine_grad<Z, Y, 1>)
    const void *fn = row_elem == TDG_ELEM_F16
                         ? (token_elem == TDG_ELEM_F16 ? TDG_GRAD(_Float16, _Float16) : TDG_GRAD(_Float16, float))
                         : (token_elem == TDG_ELEM_F16 ? TDG_GRAD(float, _Float16) : TDG_GRAD(float, float));
#undef TDG_GRAD
    return launch(fn, dim3((unsigned)gx, (unsigned)gy), ROW_THREADS, 0, &a, stream);
}

}  // extern "C"
