// tdg_layer.hip -- a whole layer of experts for a few tokens:
//   y[t] = sum over j of w[t][j] * (h[t][j] . down[e]),   e = ids[t][j],
//   h[t][j] = silu(x[t] . gate[e]) * (x[t] . up[e]),      silu(g) = g / (1 + exp(-g)),
// where gate[e] and up[e] are the left and the right half of one matrix.
//
// A few tokens read every weight of the experts that they pick and use each for
// a few rows, so the layer is bound by reading them, and by the launches and
// waits around that.  Weights go from memory to registers as they lie (rows of
// k, a lane takes neighbouring columns) and from there to the matrix cores.  A
// workgroup works for one expert: it finds the expert's entries (e = t * top_k
// + j) among the ids by itself, so that nothing is sorted before.
//   * k_layer_up: FP16 products of x, FP32 sums; h in FP32 to the workspace.
//   * k_layer_down: z = h . down with h as it is, on the FP32 matrix instructions:
//     up to 16 rows at a time keep about the pace of reading the weights.
//   * k_layer_join: y from the tokens' rows of z, in the order of j, rounded once.
// Rows of a tile belong to one expert alone, so no token meets a weight of an
// expert that it did not pick, whatever that holds.
#include "tdg_kernels.hpp"

#include "tdg_check.h"
#include "tdg_internal.h"
#include "tdg_layer_plan.h"

namespace {

using namespace tdg;

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int MAX_ENTRIES = TDG_LAYER_MAX_TOKENS * TDG_LAYER_MAX_TOP_K;

struct LayerArgs {
    const unsigned char *x, *up, *down;
    const int32_t *ids;
    const float *weights;  // NULL: 1
    unsigned char *y;
    // The workspace.  One part of k in the up product: h, entries x ld_h; more:
    // parts x entries x 2 x ld_h sums of gate and up.  z: parts_z x entries x ld_z.
    float *h, *z;
    int64_t ldx, ld_up, stride_up, ld_down, stride_down, ldy;     // bytes
    int64_t ld_ids, ld_weights;                                   // elements
    int64_t ld_h, ld_z;                                           // elements, multiples of 4
    int top_k, experts, cols, inner, entries;
    int parts, parts_z;  // workgroups that share k: grid.z of the up and of the down product
    int piece;           // elements of h that a wave of down joins in LDS
};

__device__ __forceinline__ int id_of(const LayerArgs &p, int entry) {
    const int t = entry / p.top_k;
    return entry < p.entries ? p.ids[t * p.ld_ids + (entry - t * p.top_k)] : -1;
}

// The entries of the workgroup's expert, in order.  Where there are no more
// entries than experts, workgroup `slot` works for the expert of entry `slot`,
// if that is the first entry that names it; else for expert `slot`.
struct Mine {
    int expert, count;
};

__device__ __forceinline__ Mine find_entries(const LayerArgs &p, int slot, int *list) {
    const int lane = threadIdx.x & 63;
    const bool by_entry = p.entries <= p.experts;
    int id = id_of(p, lane);
    Mine m = {by_entry ? id_of(p, slot) : slot, 0};
    m.expert = __builtin_amdgcn_readfirstlane(m.expert);
    if ((unsigned)m.expert >= (unsigned)p.experts) return m;
    for (int base = 0; base < p.entries; base += 64) {  // (every wave: the same values to the same places)
        if (base) id = id_of(p, base + lane);
        const bool hit = id == m.expert;
        const unsigned long long hits = __ballot(hit);
        if (hit) list[m.count + __popcll(hits & ((1ull << lane) - 1))] = base + lane;
        if (by_entry && m.count == 0 && hits && base + __ffsll((long long)hits) - 1 < slot) return m;  // not the first
        m.count += __popcll(hits);
    }
    return m;
}

// V neighbouring FP16 elements at any alignment.
template <int V>
struct Halves {
    typedef _Float16 vec __attribute__((ext_vector_type(V)));
    typedef vec vec_ua __attribute__((aligned(2)));
};
template <>
struct Halves<1> {
    typedef _Float16 vec;
    typedef _Float16 vec_ua;
};

template <int V>
__device__ __forceinline__ typename Halves<V>::vec load_halves(const unsigned char *p) {
    return *(const typename Halves<V>::vec_ua *)p;
}

template <int V>
__device__ __forceinline__ _Float16 element(typename Halves<V>::vec v, int i) {
    if constexpr (V == 1) return v;
    else return v[i];
}

// V neighbouring elements of N rows of a matrix from row k on; rows from K on,
// which the caller's `cut` says there may be, are zeros.
template <int V, int N>
__device__ __forceinline__ void load_rows(typename Halves<V>::vec (&w)[N], const unsigned char *base, int64_t ld, int k,
                                          int K, bool cut) {
#pragma unroll
    for (int e = 0; e < N; e++) {
        if (!cut || k + e < K) w[e] = load_halves<V>(base + (int64_t)(k + e) * ld);
        else w[e] = typename Halves<V>::vec{};
    }
}

// silu(g) * u.  Below -87 exp(-g) nears FP32's largest value, and from -88.8 on the
// quotient would be 0: there 1 + exp(-g) is exp(-g) to the last bit, and g * exp(g)
// * u is formed with a root of exp(g) on each side, so that it stays until it is
// itself too small for FP32.
__device__ __forceinline__ float gated(float g, float u) {
    const bool low = g < -87.0f;
    const float e = expf(low ? 0.5f * g : -g);
    return low ? g * e * (u * e) : g / (1.0f + e) * u;
}

// Sums the waves' parts of one accumulator row, in order.
template <int NW, int SIDES, int N>
__device__ __forceinline__ float join_waves(const float (&part)[NW][SIDES][N], int side, int e) {
    float sum = part[0][side][e];
#pragma unroll
    for (int w = 1; w < NW; w++) sum += part[w][side][e];
    return sum;
}

// A workgroup has 16 V columns of gate and up and all of k, of which each wave
// takes a part, 32 at a time: lane l loads V columns from 16 V (l % 16) on, at
// k = 8 (l / 16) .. + 7.
template <int MT, int V, int NW>
__global__ void __launch_bounds__(NW * 64) k_layer_up(LayerArgs p) {
    __shared__ int list[MAX_ENTRIES];
    __shared__ float part[NW][2][V * 64];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Mine mine = find_entries(p, blockIdx.y, list);
    if (mine.count == 0) return;
    typedef typename Halves<V>::vec vec;
    const int want = ((int)blockIdx.x * 16 + c) * V, n = min(want, p.inner - V);
    const unsigned char *gate = p.up + mine.expert * p.stride_up + (int64_t)n * 2, *up = gate + (int64_t)p.inner * 2;
    const int steps = (p.cols + 31) / 32, runs = NW * p.parts, run = (int)blockIdx.z * NW + wave;
    const int s0 = (int)((int64_t)steps * run / runs), s1 = (int)((int64_t)steps * (run + 1) / runs);
    __syncthreads();
    for (int r0 = 0; r0 < mine.count; r0 += 16 * MT) {
        const unsigned char *x[MT];  // a lane behind the last row takes that one: its sums are not stored
#pragma unroll
        for (int i = 0; i < MT; i++)
            x[i] = p.x + (int64_t)(list[min(r0 + i * 16 + c, mine.count - 1)] / p.top_k) * p.ldx;
        f32x4 acc[2][V][MT] = {};
        for (int s = s0; s < s1; s++) {
            const int k = s * 32 + q * 8;
            const bool cut = s * 32 + 32 > p.cols;
            vec g[8], u[8];
            load_rows<V, 8>(g, gate, p.ld_up, k, p.cols, cut);
            load_rows<V, 8>(u, up, p.ld_up, k, p.cols, cut);
            f16x8 a[MT];
#pragma unroll
            for (int i = 0; i < MT; i++) {
                if (!cut || k + 8 <= p.cols) {
                    a[i] = __builtin_bit_cast(f16x8, load16_global(x[i] + (int64_t)k * 2));
                } else {
                    a[i] = f16x8{};
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (k + e < p.cols) a[i][e] = *(const _Float16 *)(x[i] + (int64_t)(k + e) * 2);
                }
            }
#pragma unroll
            for (int v = 0; v < V; v++) {
                f16x8 bg, bu;
#pragma unroll
                for (int e = 0; e < 8; e++) bg[e] = element<V>(g[e], v), bu[e] = element<V>(u[e], v);
#pragma unroll
                for (int i = 0; i < MT; i++) {
                    acc[0][v][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i], bg, acc[0][v][i], 0, 0, 0);
                    acc[1][v][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i], bu, acc[1][v][i], 0, 0, 0);
                }
            }
        }
        // Lane l has rows 4 (l / 16) .. + 3 of column l % 16; a round joins one
        // row of each.
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                if (r0 + i * 16 + r >= mine.count) continue;
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; v++) {
                    part[wave][0][v * 64 + lane] = acc[0][v][i][r];
                    part[wave][1][v * 64 + lane] = acc[1][v][i][r];
                }
                __syncthreads();
                for (int e = tid; e < V * 64; e += NW * 64) {  // (e % 64 == lane)
                    const int row = r0 + i * 16 + q * 4 + r;
                    if (row >= mine.count || want >= p.inner) continue;
                    const float sg = join_waves(part, 0, e), su = join_waves(part, 1, e);
                    if (p.parts == 1) {
                        p.h[list[row] * p.ld_h + n + (e >> 6)] = gated(sg, su);
                    } else {
                        float *out = p.h + ((int64_t)blockIdx.z * p.entries + list[row]) * 2 * p.ld_h + n + (e >> 6);
                        out[0] = sg, out[p.ld_h] = su;
                    }
                }
            }
    }
}

// A wave's piece of h from the parts of gate and up, k = k0 .. k0 + len - 1 of
// `count` rows, to LDS: each element once for the wave, not once for each lane
// and column that it is multiplied with.  Zeros from the end of k on.  A lane
// takes W neighbours: four where there are many, or its gates follow each other
// for nothing (one token: 9.8 us with one, 10.7 with four; 33 tokens 27.8, 26.8).
template <int PARTS, int W>
__device__ __forceinline__ void join_h(const LayerArgs &p, const int *list, int count, int k0, int len, int lane,
                                       float *piece) {
    typedef float vec __attribute__((ext_vector_type(W)));
    for (int e = lane * W; e < count * len; e += 64 * W) {
        const int r = e / len, k = k0 + (e - r * len);
        vec v = {};
        if (k < p.inner) {  // (rows are whole pieces of four)
            const float *at = p.h + list[r] * 2 * p.ld_h + k;
            vec g[PARTS], u[PARTS];
#pragma unroll
            for (int i = 0; i < PARTS; i++) {
                const float *from = at + i * p.entries * 2 * p.ld_h;
                g[i] = *(const vec *)from, u[i] = *(const vec *)(from + p.ld_h);
            }
#pragma unroll
            for (int i = 1; i < PARTS; i++) g[0] += g[i], u[0] += u[i];
#pragma unroll
            for (int j = 0; j < W; j++) v[j] = k + j < p.inner ? gated(g[0][j], u[0][j]) : 0.0f;
        }
        *(vec *)(piece + e) = v;
    }
}

// y[t][n] from the token's rows of z; eight of them travel at a time.
template <typename T>
__device__ __forceinline__ void join_token(const LayerArgs &p, int t, int n) {
    constexpr int J = 8;
    const float *z = p.z + t * p.top_k * p.ld_z + n;
    float sum = 0.0f;
    for (int j0 = 0; j0 < p.top_k; j0 += J) {
        int id[J];
        float w[J], v[J];
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int at = min(j0 + j, p.top_k - 1);
            id[j] = j0 + j < p.top_k ? p.ids[t * p.ld_ids + at] : -1;
            w[j] = p.weights ? p.weights[t * p.ld_weights + at] : 1.0f;
            v[j] = z[at * p.ld_z];
        }
        for (int i = 1; i < p.parts_z; i++)
#pragma unroll
            for (int j = 0; j < J; j++) v[j] += z[(i * p.entries + min(j0 + j, p.top_k - 1)) * p.ld_z];
#pragma unroll
        for (int j = 0; j < J; j++)
            if ((unsigned)id[j] < (unsigned)p.experts) sum = fmaf(w[j], v[j], sum);
    }
    *(T *)(p.y + t * p.ldy + (int64_t)n * sizeof(T)) = (T)sum;
}

// The down product of up to 16 rows of an expert: a workgroup has 16 V columns,
// lane l loads V of them at k = 4 q .. + 3 of each 16, q = l / 16, and the e-th
// products take row e of those.  Without FOURS v_mfma_f32_16x16x4_f32, a
// product of 16 rows at the four k of the lane groups; with it four rows on
// v_mfma_f32_4x4x1_16b_f32, a quarter of its time: 16 blocks of four lanes' columns, each at its own lanes' k, so that a column's sum is spread
// over the four lane groups, and added at the end.  Most experts of a few tokens
// have four rows or fewer, and the time of 16 rows' products shows: it is as long
// as that of reading the weights (16 tokens, 8 of 64 experts, 2048 x 1024: 47 us
// without loads, 47 without products, 58.6 with both; with four rows' products 55;
// one token 10.3 and 8.0).
template <int V, int NW, int PARTS, bool FOURS>
__device__ __forceinline__ void down_rows(const LayerArgs &p, const unsigned char *down, const int *list, int rows,
                                          int want, int n, int s0, int s1, float *piece,
                                          float (&part)[NW][1][V * 64]) {
    constexpr bool JOIN = PARTS > 1;
    typedef typename Halves<V>::vec vec;
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto load = [&](vec (&w)[4], int s) {
        load_rows<V, 4>(w, down, p.ld_down, s * 16 + q * 4, p.inner, s * 16 + 16 > p.inner);
    };
    vec w[4];
    if constexpr (JOIN) {  // the first weights travel while h is joined
        if (s0 < s1) load(w, s0);
        const int len = (s1 - s0) * 16;
        if (rows * len > 256) join_h<PARTS, 4>(p, list, rows, s0 * 16, len, lane, piece);
        else join_h<PARTS, 1>(p, list, rows, s0 * 16, len, lane, piece);
        __builtin_amdgcn_wave_barrier();  // (the wave's own piece: no other wave reads it)
    }
    const int row = min(FOURS ? lane & 3 : c, rows - 1);  // (rows behind the last: not stored)
    const float *h = JOIN ? piece + row * (s1 - s0) * 16 - s0 * 16 : p.h + list[row] * p.ld_h;
    f32x4 acc[V] = {};
    for (int s = s0; s < s1; s++) {
        const int k = s * 16 + q * 4;
        // (Loads a step ahead: 63.6 us for 58.6 at 16 tokens, for the waves that their
        // registers cost.)
        if (!JOIN || s > s0) load(w, s);
        f32x4 a = {};
        if (JOIN || k < p.inner) a = *(const f32x4 *)(h + k);  // (rows are whole pieces of four)
        if (!JOIN && s * 16 + 16 > p.inner) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (k + e >= p.inner) a[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 4; e++)
#pragma unroll
            for (int v = 0; v < V; v++) {
                const float ae = a[e], be = (float)element<V>(w[e], v);
                if constexpr (FOURS) acc[v] = __builtin_amdgcn_mfma_f32_4x4x1f32(ae, be, acc[v], 0, 0, 0);
                else acc[v] = __builtin_amdgcn_mfma_f32_16x16x4f32(ae, be, acc[v], 0, 0, 0);
            }
    }
#pragma unroll
    for (int r = 0; r < 4; r++) {
        if (r >= rows) break;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; v++) part[wave][0][v * 64 + lane] = acc[v][r];
        __syncthreads();
        for (int e = tid; e < V * 64; e += NW * 64) {  // (e % 64 == lane)
            float sum = join_waves(part, 0, e);
            if constexpr (FOURS) sum += __shfl_xor(sum, 16), sum += __shfl_xor(sum, 32);
            const int at = FOURS ? r : q * 4 + r;
            if (at < rows && want < p.cols && (!FOURS || q == 0))
                p.z[((int64_t)blockIdx.z * p.entries + list[at]) * p.ld_z + n + (e >> 6)] = sum;
        }
    }
}

template <int V, int NW, int PARTS>
__global__ void __launch_bounds__(NW * 64) k_layer_down(LayerArgs p) {
    __shared__ int list[MAX_ENTRIES];
    __shared__ float part[NW][1][V * 64];
    extern __shared__ __attribute__((aligned(16))) float pieces[];  // PARTS > 1: a piece of h for each wave
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Mine mine = find_entries(p, blockIdx.y, list);
    if (mine.count == 0) return;
    const int want = ((int)blockIdx.x * 16 + (threadIdx.x & 15)) * V, n = min(want, p.cols - V);
    const unsigned char *down = p.down + mine.expert * p.stride_down + (int64_t)n * 2;
    const int steps = (p.inner + 15) / 16, runs = NW * p.parts_z, run = (int)blockIdx.z * NW + wave;
    const int s0 = (int)((int64_t)steps * run / runs), s1 = (int)((int64_t)steps * (run + 1) / runs);
    float *piece = PARTS > 1 ? pieces + wave * p.piece : nullptr;
    __syncthreads();
    for (int r0 = 0; r0 < mine.count; r0 += 16) {
        const int rows = min(16, mine.count - r0);
        if (rows <= 4) down_rows<V, NW, PARTS, true>(p, down, list + r0, rows, want, n, s0, s1, piece, part);
        else down_rows<V, NW, PARTS, false>(p, down, list + r0, rows, want, n, s0, s1, piece, part);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_layer_join(LayerArgs p) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n < p.cols) join_token<T>(p, blockIdx.y, n);
}

// ------------------------------------------------------------------ host side

bool sizes_ok(int64_t tokens, int64_t top_k, int64_t experts, int64_t cols, int64_t inner) {
    return tokens >= 0 && top_k >= 1 && experts >= 1 && experts <= 1024 && size_ok(tokens) && size_ok(top_k) &&
           size_ok(cols) && cols <= kMaxSize / 2 && size_ok(inner) && inner <= kMaxSize / 2;
}

int launch(const void *fn, dim3 grid, int threads, size_t lds, LayerArgs *args, void *stream) {
    void *kargs[] = {args};
    if (hipLaunchKernel(fn, grid, dim3((unsigned)threads), kargs, lds, (hipStream_t)stream) != hipSuccess)
        return TDG_ERR_LAUNCH;
    if (hipGetLastError() != hipSuccess) return TDG_ERR_LAUNCH;
    return TDG_OK;
}

}  // namespace

extern "C" {

int tdg_expert_layer_workspace(int64_t tokens, int64_t top_k, int64_t experts, int64_t cols, int64_t inner,
                               size_t *bytes) {
    if (!bytes || !sizes_ok(tokens, top_k, experts, cols, inner)) return TDG_ERR_INVALID_ARG;
    if (tokens > TDG_LAYER_MAX_TOKENS || top_k > TDG_LAYER_MAX_TOP_K) return TDG_ERR_UNSUPPORTED;
    *bytes = (size_t)layer_plan(tokens, top_k, experts, cols, inner).bytes;
    return TDG_OK;
}

int tdg_expert_layer(int out_elem, int64_t tokens, int64_t top_k, int64_t experts, int64_t cols, int64_t inner,
                     const uint16_t *x, int64_t ldx, const int32_t *ids, int64_t ld_ids, const float *weights,
                     int64_t ld_weights, const uint16_t *up, int64_t ld_up, int64_t stride_up, const uint16_t *down,
                     int64_t ld_down, int64_t stride_down, void *y, int64_t ldy, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (out_elem != TDG_ELEM_F16 && out_elem != TDG_ELEM_F32) return TDG_ERR_INVALID_ARG;
    const int64_t es = out_elem == TDG_ELEM_F16 ? 2 : 4;
    size_t need = 0;
    const int fits = tdg_expert_layer_workspace(tokens, top_k, experts, cols, inner, &need);
    if (fits == TDG_ERR_INVALID_ARG) return fits;
    if (!matrix_ok(x, tokens, cols, ldx, 2) || !matrix_ok(ids, tokens, top_k, ld_ids, 4) ||
        (weights && !matrix_ok(weights, tokens, top_k, ld_weights, 4)) ||
        !stack_ok(up, experts, stride_up, cols, 2 * inner, ld_up, 2, false) ||
        !stack_ok(down, experts, stride_down, inner, cols, ld_down, 2, false) || !matrix_ok(y, tokens, cols, ldy, es))
        return TDG_ERR_INVALID_ARG;
    if (!aligned_to(x, 2) || !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(up, 2) ||
        !aligned_to(down, 2) || !aligned_to(y, es))
        return TDG_ERR_INVALID_ARG;
    const void *in[5] = {x, ids, weights, up, down};
    const uint64_t in_len[5] = {span_bytes(tokens, cols, ldx, 2), span_bytes(tokens, top_k, ld_ids, 4),
                                span_bytes(tokens, top_k, ld_weights, 4),
                                span_bytes(cols, 2 * inner, ld_up, 2, experts, stride_up),
                                span_bytes(inner, cols, ld_down, 2, experts, stride_down)};
    const uint64_t y_len = span_bytes(tokens, cols, ldy, es);
    for (int i = 0; i < 5; i++)
        if (overlaps(y, y_len, in[i], in_len[i])) return TDG_ERR_INVALID_ARG;
    if (fits != TDG_OK) return fits;
    if (tokens == 0 || cols == 0) return TDG_OK;
    if (!workspace || workspace_bytes < need || !aligned_to(workspace, 16) || overlaps(workspace, need, y, y_len))
        return TDG_ERR_INVALID_ARG;
    for (int i = 0; i < 5; i++)
        if (overlaps(workspace, need, in[i], in_len[i])) return TDG_ERR_INVALID_ARG;

    const LayerPlan plan = layer_plan(tokens, top_k, experts, cols, inner);
    LayerArgs p;
    p.x = (const unsigned char *)x, p.up = (const unsigned char *)up, p.down = (const unsigned char *)down;
    p.ids = ids, p.weights = weights, p.y = (unsigned char *)y;
    p.entries = (int)(tokens * top_k);
    p.ld_h = up4(inner), p.ld_z = up4(cols);
    p.h = (float *)workspace, p.z = (float *)((unsigned char *)workspace + plan.z_at);
    p.ldx = ldx * 2, p.ld_up = ld_up * 2, p.stride_up = stride_up * 2, p.ld_down = ld_down * 2;
    p.stride_down = stride_down * 2, p.ldy = ldy * es, p.ld_ids = ld_ids, p.ld_weights = ld_weights;
    p.top_k = (int)top_k, p.experts = (int)experts, p.cols = (int)cols;
    p.inner = (int)inner;
    p.parts = (int)plan.parts, p.parts_z = (int)plan.parts_z, p.piece = (int)plan.piece;
    const int64_t join_x = ceil_quot(cols, 256), most = (int64_t)UINT32_MAX / 1024;
    if (plan.up_x * plan.slots * plan.parts > most || plan.down_x * plan.slots * plan.parts_z > most ||
        join_x * tokens > most)
        return TDG_ERR_UNSUPPORTED;
    int rc = device_check();
    if (rc != TDG_OK) return rc;
    if (inner > 0) {
        const void *fn = plan.thin_up     ? (const void *)&k_layer_up<2, 1, 8>
                         : plan.two_tiles ? (const void *)&k_layer_up<2, 8, 8>
                                          : (const void *)&k_layer_up<1, 8, 8>;
        rc = launch(fn, dim3((unsigned)plan.up_x, (unsigned)plan.slots, (unsigned)plan.parts), 512, 0, &p, stream);
        if (rc != TDG_OK) return rc;
    }
#define TDG_LAYER_DOWN(...)                                                  \
    (plan.parts == 1   ? (const void *)&k_layer_down<__VA_ARGS__, 1>         \
     : plan.parts == 2 ? (const void *)&k_layer_down<__VA_ARGS__, 2>         \
                       : (const void *)&k_layer_down<__VA_ARGS__, 4>)
    const void *fn = plan.thin_down ? (const void *)&k_layer_down<1, 8, 1>  // (with few columns k is not cut)
                     : plan.narrow  ? TDG_LAYER_DOWN(4, 16)
                                    : TDG_LAYER_DOWN(8, 8);
#undef TDG_LAYER_DOWN
    rc = launch(fn, dim3((unsigned)plan.down_x, (unsigned)plan.slots, (unsigned)plan.parts_z), plan.narrow ? 1024 : 512,
                p.parts > 1 ? (size_t)p.piece * 4 * (plan.narrow ? 16 : 8) : 0, &p, stream);
    if (rc != TDG_OK) return rc;
    return launch(es == 2 ? (const void *)&k_layer_join<_Float16> : (const void *)&k_layer_join<float>,
                  dim3((unsigned)join_x, (unsigned)tokens), 256, 0, &p, stream);
}

}  // extern "C"
