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
//   * k_layer_down: h stays FP32, on v_mfma_f32_16x16x4_f32, whose rate on up to
//     16 rows is still above that of reading the weights; z = h . down in FP32.
//   * k_layer_join: y from the tokens' rows of z, in the order of j, rounded once.
// Rows of a tile belong to one expert alone, so no token meets a weight of an
// expert that it did not pick, whatever that holds.
#include "tdg_kernels.hpp"

#include "tdg_check.h"
#include "tdg_internal.h"

namespace {

using namespace tdg;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int MAX_ENTRIES = TDG_LAYER_MAX_TOKENS * TDG_LAYER_MAX_TOP_K;
constexpr int WAVES = 8, THREADS = WAVES * 64;

struct LayerArgs {
    const unsigned char *x, *up, *down;
    const int32_t *ids;
    const float *weights;  // NULL: 1
    unsigned char *y;
    float *h, *z;                                                 // entries x ld_h, entries x ld_z
    int64_t ldx, ld_up, stride_up, ld_down, stride_down, ldy;     // bytes
    int64_t ld_ids, ld_weights;                                   // elements
    int64_t ld_h, ld_z;                                           // elements, multiples of 4
    int tokens, top_k, experts, cols, inner, entries;
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
    Mine m = {by_entry ? id_of(p, slot) : slot, 0};
    if ((unsigned)m.expert >= (unsigned)p.experts) return m;
    for (int base = 0; base < p.entries; base += 64) {  // (every wave: the same values to the same places)
        const bool hit = id_of(p, base + lane) == m.expert;
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

// Joins the waves' sums of one accumulator row: `sum` of V columns and the 64
// lanes, waves in order.
template <int V, int SIDES>
__device__ __forceinline__ float join_waves(const float (&part)[WAVES][SIDES][V * 64], int side, int e) {
    float sum = part[0][side][e];
#pragma unroll
    for (int w = 1; w < WAVES; w++) sum += part[w][side][e];
    return sum;
}

// A workgroup has 16 V columns of gate and up and all of k, of which each wave
// takes a part, 32 at a time: lane l loads V columns from 16 V (l % 16) on, at
// k = 8 (l / 16) .. + 7.
template <int MT, int V>
__global__ void __launch_bounds__(THREADS) k_layer_up(LayerArgs p) {
    __shared__ int list[MAX_ENTRIES];
    __shared__ float part[WAVES][2][V * 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, q = lane >> 4;
    const Mine mine = find_entries(p, blockIdx.y, list);
    if (mine.count == 0) return;
    typedef typename Halves<V>::vec vec;
    const int want = ((int)blockIdx.x * 16 + c) * V, n = min(want, p.inner - V);
    const unsigned char *gate = p.up + mine.expert * p.stride_up + (int64_t)n * 2, *up = gate + (int64_t)p.inner * 2;
    const int steps = (p.cols + 31) / 32, per = (steps + WAVES - 1) / WAVES;
    const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
    __syncthreads();
    for (int r0 = 0; r0 < mine.count; r0 += 16 * MT) {
        const unsigned char *x[MT];
#pragma unroll
        for (int i = 0; i < MT; i++) {
            const int r = r0 + i * 16 + c;
            x[i] = r < mine.count ? p.x + (int64_t)(list[r] / p.top_k) * p.ldx : nullptr;
        }
        f32x4 acc[2][V][MT] = {};
        for (int s = s0; s < s1; s++) {
            const int k = s * 32 + q * 8;
            vec g[8], u[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                g[e] = u[e] = vec{};
                if (k + e < p.cols) {
                    g[e] = load_halves<V>(gate + (int64_t)(k + e) * p.ld_up);
                    u[e] = load_halves<V>(up + (int64_t)(k + e) * p.ld_up);
                }
            }
            f16x8 a[MT];
#pragma unroll
            for (int i = 0; i < MT; i++) {
                a[i] = f16x8{};
                if (x[i] && k + 8 <= p.cols) {
                    a[i] = __builtin_bit_cast(f16x8, load16_global(x[i] + (int64_t)k * 2));
                } else if (x[i]) {
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
                for (int e = tid; e < V * 64; e += THREADS) {  // (e % 64 == lane)
                    const float sg = join_waves<V, 2>(part, 0, e), su = join_waves<V, 2>(part, 1, e);
                    const int row = r0 + i * 16 + q * 4 + r;
                    if (row < mine.count && want < p.inner)
                        p.h[list[row] * p.ld_h + n + (e >> 6)] = sg / (1.0f + expf(-sg)) * su;
                }
            }
    }
}

// A workgroup has 16 V columns of down; lane l loads V of them at k = 4 (l / 16)
// .. + 3, and the product's e-th step takes row e of each.
template <int MT, int V>
__global__ void __launch_bounds__(THREADS) k_layer_down(LayerArgs p) {
    __shared__ int list[MAX_ENTRIES];
    __shared__ float part[WAVES][1][V * 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, q = lane >> 4;
    const Mine mine = find_entries(p, blockIdx.y, list);
    if (mine.count == 0) return;
    typedef typename Halves<V>::vec vec;
    const int want = ((int)blockIdx.x * 16 + c) * V, n = min(want, p.cols - V);
    const unsigned char *down = p.down + mine.expert * p.stride_down + (int64_t)n * 2;
    const int steps = (p.inner + 15) / 16, per = (steps + WAVES - 1) / WAVES;
    const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
    __syncthreads();
    for (int r0 = 0; r0 < mine.count; r0 += 16 * MT) {
        const float *h[MT];
#pragma unroll
        for (int i = 0; i < MT; i++) {
            const int r = r0 + i * 16 + c;
            h[i] = r < mine.count ? p.h + list[r] * p.ld_h : nullptr;
        }
        f32x4 acc[V][MT] = {};
        for (int s = s0; s < s1; s++) {
            const int k = s * 16 + q * 4;
            vec w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                w[e] = vec{};
                if (k + e < p.inner) w[e] = load_halves<V>(down + (int64_t)(k + e) * p.ld_down);
            }
            f32x4 a[MT];
#pragma unroll
            for (int i = 0; i < MT; i++) {
                a[i] = f32x4{};
                if (h[i] && k < p.inner) a[i] = *(const f32x4 *)(h[i] + k);  // (rows end on 16 bytes)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (k + e >= p.inner) a[i][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 4; e++)
#pragma unroll
                for (int v = 0; v < V; v++) {
                    const float b = (float)element<V>(w[e], v);
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const float ae = a[i][e];
                        acc[v][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(ae, b, acc[v][i], 0, 0, 0);
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                if (r0 + i * 16 + r >= mine.count) continue;
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; v++) part[wave][0][v * 64 + lane] = acc[v][i][r];
                __syncthreads();
                for (int e = tid; e < V * 64; e += THREADS) {
                    const float sum = join_waves<V, 1>(part, 0, e);
                    const int row = r0 + i * 16 + q * 4 + r;
                    if (row < mine.count && want < p.cols) p.z[list[row] * p.ld_z + n + (e >> 6)] = sum;
                }
            }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_layer_join(LayerArgs p) {
    const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (n >= p.cols) return;
    float sum = 0.0f;
    for (int j = 0; j < p.top_k; j++) {
        if ((unsigned)p.ids[t * p.ld_ids + j] >= (unsigned)p.experts) continue;
        const float z = p.z[(t * p.top_k + j) * p.ld_z + n];
        sum = p.weights ? fmaf(p.weights[t * p.ld_weights + j], z, sum) : sum + z;
    }
    *(T *)(p.y + t * p.ldy + (int64_t)n * sizeof(T)) = (T)sum;
}

// ------------------------------------------------------------------ host side

bool sizes_ok(int64_t tokens, int64_t top_k, int64_t experts, int64_t cols, int64_t inner) {
    return tokens >= 0 && top_k >= 1 && experts >= 1 && experts <= 1024 && size_ok(tokens) && size_ok(top_k) &&
           size_ok(cols) && cols <= kMaxSize / 2 && size_ok(inner) && inner <= kMaxSize / 2;
}

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

int launch(const void *fn, dim3 grid, int threads, LayerArgs *args, void *stream) {
    void *kargs[] = {args};
    if (hipLaunchKernel(fn, grid, dim3((unsigned)threads), kargs, 0, (hipStream_t)stream) != hipSuccess)
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
    *bytes = (size_t)(tokens * top_k * (up4(inner) + up4(cols)) * 4);
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

    LayerArgs p;
    p.x = (const unsigned char *)x, p.up = (const unsigned char *)up, p.down = (const unsigned char *)down;
    p.ids = ids, p.weights = weights, p.y = (unsigned char *)y;
    p.entries = (int)(tokens * top_k);
    p.ld_h = up4(inner), p.ld_z = up4(cols);
    p.h = (float *)workspace, p.z = p.h + p.entries * p.ld_h;
    p.ldx = ldx * 2, p.ld_up = ld_up * 2, p.stride_up = stride_up * 2, p.ld_down = ld_down * 2;
    p.stride_down = stride_down * 2, p.ldy = ldy * es, p.ld_ids = ld_ids, p.ld_weights = ld_weights;
    p.tokens = (int)tokens, p.top_k = (int)top_k, p.experts = (int)experts, p.cols = (int)cols;
    p.inner = (int)inner;
    const int64_t slots = p.entries < experts ? p.entries : experts;
    const int vu = inner >= 8 ? 4 : 1, vd = cols >= 8 ? 8 : 1;
    const int64_t up_x = ceil_quot(inner, 16 * vu), down_x = ceil_quot(cols, 16 * vd), join_x = ceil_quot(cols, 256);
    const int64_t most = (int64_t)UINT32_MAX / THREADS;
    if (up_x * slots > most || down_x * slots > most || join_x * tokens > most) return TDG_ERR_UNSUPPORTED;
    int rc = device_check();
    if (rc != TDG_OK) return rc;
    if (inner > 0)
        rc = launch(vu == 4 ? (const void *)&k_layer_up<4, 4> : (const void *)&k_layer_up<4, 1>,
                    dim3((unsigned)up_x, (unsigned)slots), THREADS, &p, stream);
    if (rc != TDG_OK) return rc;
    rc = launch(vd == 8 ? (const void *)&k_layer_down<1, 8> : (const void *)&k_layer_down<1, 1>,
                dim3((unsigned)down_x, (unsigned)slots), THREADS, &p, stream);
    if (rc != TDG_OK) return rc;
    return launch(es == 2 ? (const void *)&k_layer_join<_Float16> : (const void *)&k_layer_join<float>,
                  dim3((unsigned)join_x, (unsigned)tokens), 256, &p, stream);
}

}  // extern "C"
