// tdg_w4.hip -- 4-bit weights with group scales: quantizing, reading back, and
// the products that multiply FP16 rows by them, for one matrix and for a stack
// of experts' matrices whose rows are sorted.
//
// A K x N matrix is kept as codes, 4 bits a weight, and for every `group`
// values of k of a column an FP16 scale s and a zero point z (8 where none are
// given); the weight is (code - z) * s.  The product is
//   C[m][n] = sum over groups G of s[G][n] * sum over k in G of A[m][k] * (code[k][n] - z[G][n]).
// code - z is a whole number of at most 255 and exact in FP16, so the matrix
// instructions multiply it as it is; the scale joins in FP32, once for each
// group's (or each 32 k's) sum: no weight is rounded.
//
// Codes are laid out for v_mfma_f32_16x16x32_f16, whose lane l takes column l %
// 16 at k = 8 (l / 16) .. + 7: a column's 128 k are 64 bytes, of which lane
// group q = l / 16 takes 16: the words of its k in each of four instructions.
// The nibbles of a word stand so that four masks give them in pairs, two
// neighbours in k in the halves of a register.
#include "tdg_grouped.hpp"

#include "tdg_check.h"
#include "tdg_internal.h"
#include "tdg_w4_plan.h"

namespace {

using namespace tdg;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int BLOCK = 128;  // k in one block of codes: 64 bytes of a column

// Strides in bytes; `codes`' row is a block of k.
struct Weights4 {
    const unsigned char *codes, *scales, *zeros;
    int64_t ld_codes, ld_scales, ld_zeros;              // between blocks, groups
    int64_t stride_codes, stride_scales, stride_zeros;  // between matrices
};

// Where bit 0 of k's nibble stands in its word, k = 0 .. 7.
__device__ __forceinline__ constexpr int nibble_at(int k) { return 4 * (k >> 1) + 16 * (k & 1); }

// ------------------------------------------------------------------ quantizing

struct QuantArgs {
    const unsigned char *W;
    int64_t ldw, stride_w;  // bytes
    Weights4 q;             // written
    int K, N, group;
    int run;  // neighbours that one XCD takes
};

struct Place {
    int x, y, z;
};

// The workgroup's place in its grid.  Workgroups are dealt round-robin to the 8
// XCDs; here each takes `run` neighbours of a row, so that a line that two of
// them share is read, or put together, in one L2.
__device__ __forceinline__ Place place_in_runs(uint32_t run) {
    if (run == 1) return {(int)blockIdx.x, (int)blockIdx.y, (int)blockIdx.z};
    const uint32_t total = gridDim.x * gridDim.y * gridDim.z, round = 8 * run;
    uint32_t id = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    const uint32_t in = id % round;
    if (id - in + round <= total) id += (in & 7) * run + (in >> 3) - in;  // (the last round stays as it is)
    const uint32_t row = id / gridDim.x, z = row / gridDim.y;
    return {(int)(id - row * gridDim.x), (int)(row - z * gridDim.y), (int)z};
}

struct ScaleZero {
    float s, r, z;  // r: 1 / s
};

// Scale and zero point of a group that holds values from lo to hi (symmetric:
// of a magnitude up to hi).  Each step is one correctly rounded FP32 operation.
template <bool ZEROS>
__device__ __forceinline__ ScaleZero scale_of(float lo, float hi) {
    const float s = (float)(_Float16)(ZEROS ? (hi - lo) / 15.0f : hi / 7.0f);
    if constexpr (!ZEROS) return {s, 1.0f / s, 8.0f};
    const float z = rintf(-lo / s);  // s == 0, or infinities: NaN may come out
    return {s, 1.0f / s, s > 0.0f && z >= 0.0f ? fminf(z, 15.0f) : 0.0f};
}

// The code of w: the nearest of the 16 values.  The quotient is w * r with one
// correction.  A quotient of two FP16 numbers that is half a whole number below
// 16 comes out exactly (the correction's own error is far below half a step),
// and any other lies at least 2^-13 from such a one: the code is that of the
// correctly rounded quotient.  NaN comes out for a scale of 0 or infinity and
// for a weight of NaN: the zero's code.
__device__ __forceinline__ uint32_t code_of(float w, ScaleZero g) {
    float q = w * g.r;
    q = rintf(fmaf(fmaf(-q, g.s, w), g.r, q));
    return (uint32_t)(q != q ? g.z : __builtin_amdgcn_fmed3f(q + g.z, 0.0f, 15.0f));
}

__device__ __forceinline__ float load_weight(const unsigned char *p) { return (float)*(const _Float16 *)p; }

template <bool ZEROS>
__device__ __forceinline__ void widen(float w, float &lo, float &hi) {  // (a NaN changes nothing)
    if constexpr (ZEROS) lo = fminf(lo, w), hi = fmaxf(hi, w);
    else hi = fmaxf(hi, fabsf(w));
}

template <bool ZEROS>
__device__ __forceinline__ void store_scale(const QuantArgs &a, int64_t e, int g, int n, ScaleZero v) {
    *(_Float16 *)(a.q.scales + e * a.q.stride_scales + g * a.q.ld_scales + (int64_t)n * 2) = (_Float16)v.s;
    if constexpr (ZEROS)
        *(unsigned char *)(a.q.zeros + e * a.q.stride_zeros + g * a.q.ld_zeros + n) = (unsigned char)v.z;
}

// Groups of G = 32, 64 or 128: one pass.  A workgroup has 64 columns of a block
// and each of its four waves 32 k of them, a column to a lane; LDS joins the
// waves' ranges, and puts the words of a column together, so that the codes leave
// as whole lines (4096 x 4096, groups of 128: 11.5 us; a thread with all 128 k of one
// column 14.8, of two 19.4; scales and codes in two passes, with two divisions, 54).
// Rows that start inside lines: runs of 8 places (8 of 1000 x 4095, groups of 64:
// 21.2 us, 24.4 without; rows of whole lines 11.8, and 11.4 without).
template <int G, bool ZEROS>
__global__ void __launch_bounds__(256) k_w4_quantize(QuantArgs a) {
    constexpr int PIECES = G / 32;             // waves that share a group
    __shared__ float low[4][64], high[4][64];
    __shared__ uint32_t words[64][17];         // (a column's 16; 17 spread over the banks)
    const Place at = place_in_runs(a.run);
    const int tid = threadIdx.x, lane = tid & 63, j = tid >> 6, b = at.y;
    const int n0 = at.x * 64, n = min(n0 + lane, a.N - 1);
    const int64_t e = at.z;
    const int k0 = b * BLOCK + 32 * j, left = a.K - k0;
    const unsigned char *w = a.W + e * a.stride_w + (int64_t)k0 * a.ldw + (int64_t)n * 2;
    _Float16 v[32];
    if (left >= 32) {
#pragma unroll
        for (int k = 0; k < 32; k++) v[k] = *(const _Float16 *)(w + k * a.ldw);
    } else {
#pragma unroll
        for (int k = 0; k < 32; k++) v[k] = k < left ? *(const _Float16 *)(w + k * a.ldw) : (_Float16)0.0f;
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; k++) widen<ZEROS>((float)v[k], lo, hi);
    if constexpr (PIECES > 1) {
        low[j][lane] = lo, high[j][lane] = hi;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const int of = j / PIECES * PIECES + i;
            lo = fminf(lo, low[of][lane]), hi = fmaxf(hi, high[of][lane]);
        }
    }
    const ScaleZero sz = scale_of<ZEROS>(lo, hi);
    if (j % PIECES == 0 && left > 0 && n0 + lane < a.N) store_scale<ZEROS>(a, e, k0 / G, n, sz);
#pragma unroll
    for (int q = 0; q < 4; q++) {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) word |= code_of((float)v[8 * q + i], sz) << nibble_at(i);
        if (left < 8 * q + 8) {  // no codes from the end of k on
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (8 * q + i >= left) word &= ~(15u << nibble_at(i));
        }
        words[lane][4 * q + j] = word;
    }
    __syncthreads();
    const int col = tid >> 2, q = tid & 3;
    if (n0 + col >= a.N) return;
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; i++) out[i] = words[col][4 * q + i];
    *(u32x4 *)(a.q.codes + e * a.q.stride_codes + b * a.q.ld_codes + (int64_t)n0 * 64 + tid * 16) = out;
}

// Scales of groups of any length: a workgroup has 64 columns of one group, its
// four waves every fourth k.
template <bool ZEROS>
__global__ void __launch_bounds__(256) k_w4_scales(QuantArgs a) {
    __shared__ float low[4][64], high[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = min((int)blockIdx.x * 64 + lane, a.N - 1), g = blockIdx.y;
    const int64_t e = blockIdx.z;
    const int k1 = (int)min((int64_t)a.K, (int64_t)(g + 1) * a.group);
    const unsigned char *w = a.W + e * a.stride_w + (int64_t)n * 2;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll 8
    for (int64_t k = (int64_t)g * a.group + wave; k < k1; k += 4) widen<ZEROS>(load_weight(w + k * a.ldw), lo, hi);
    low[wave][lane] = lo, high[wave][lane] = hi;
    __syncthreads();
    if (wave || (int)blockIdx.x * 64 + lane >= a.N) return;
    for (int i = 1; i < 4; i++) lo = fminf(lo, low[i][lane]), hi = fmaxf(hi, high[i][lane]);
    store_scale<ZEROS>(a, e, g, n, scale_of<ZEROS>(lo, hi));
}

// Codes under scales that are there: a thread has a column of a block.
template <bool ZEROS>
__global__ void __launch_bounds__(256) k_w4_codes(QuantArgs a) {
    const int n = blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
    const int64_t e = blockIdx.z;
    if (n >= a.N) return;
    const unsigned char *w = a.W + e * a.stride_w + (int64_t)b * BLOCK * a.ldw + (int64_t)n * 2;
    u32x4 word[4] = {};
#pragma unroll
    for (int j = 0; j < 4; j++) {  // 32 k: all in one group
        if (b * BLOCK + 32 * j >= a.K) break;
        const int g = (b * BLOCK + 32 * j) / a.group;
        ScaleZero v;
        v.s = load_weight(a.q.scales + e * a.q.stride_scales + g * a.q.ld_scales + (int64_t)n * 2);
        v.r = 1.0f / v.s;
        v.z = ZEROS ? (float)a.q.zeros[e * a.q.stride_zeros + g * a.q.ld_zeros + n] : 8.0f;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int k = 32 * j + 8 * q + i;
                if (b * BLOCK + k < a.K) bits |= code_of(load_weight(w + k * a.ldw), v) << nibble_at(i);
            }
            word[q][j] = bits;
        }
    }
    u32x4 *out = (u32x4 *)(a.q.codes + e * a.q.stride_codes + b * a.q.ld_codes + (int64_t)n * 64);
#pragma unroll
    for (int q = 0; q < 4; q++) out[q] = word[q];
}

// Weights from codes: a workgroup has 128 columns of a block, whose codes come
// as whole lines and turn in LDS, so that a thread has V columns by 64 / V k and
// a row's pieces are stored next to each other: 16 bytes to a lane, or 4 where
// rows of FP16 start at odd elements (V = 8 / 4 / 2: 4096 x 4096 8.0 / 8.1 / 8.8 us,
// in FP32 17.5 / 15.3 / 17.2; 8 of 1000 x 4095 20.0 / 17.5 / 15.1; a thread with all
// 128 k of two columns 11.2 and 16.2).  Places in runs of 8: 9.4 without.
template <typename T, bool ZEROS, int V>
__global__ void __launch_bounds__(256) k_w4_values(QuantArgs a) {
    constexpr int ACROSS = 128 / V, WORDS = 8 / V;  // threads to a row; words of 8 k to a thread's column
    typedef T vec __attribute__((ext_vector_type(V)));
    typedef vec vec_ua __attribute__((aligned(sizeof(T))));
    typedef _Float16 halves __attribute__((ext_vector_type(V)));
    typedef halves halves_ua __attribute__((aligned(2)));
    typedef unsigned char bytes __attribute__((ext_vector_type(V)));
    typedef bytes bytes_ua __attribute__((aligned(1)));
    __shared__ __attribute__((aligned(16))) uint32_t words[16][128 + 4];  // (4: the writes' banks)
    const Place at = place_in_runs(a.run);
    const int tid = threadIdx.x, n0 = at.x * 128, b = at.y;
    const int64_t e = at.z;
    const unsigned char *codes = a.q.codes + e * a.q.stride_codes + b * a.q.ld_codes;
    u32x4 in[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
        in[i] = *(const u32x4 *)(codes + (int64_t)min(n0 + 64 * i + (tid >> 2), a.N - 1) * 64 + (tid & 3) * 16);
    // The thread's columns from n on, k from k0 on: all in one group.
    const int c = tid % ACROSS * V, n = n0 + c, first = tid / ACROSS * WORDS, have = min(a.N - n, V);
    const int k0 = b * BLOCK + first * 8, left = a.K - k0, g = min(k0, a.K - 1) / a.group;
    const unsigned char *scales = a.q.scales + e * a.q.stride_scales + g * a.q.ld_scales + (int64_t)n * 2;
    const unsigned char *zeros = a.q.zeros + e * a.q.stride_zeros + g * a.q.ld_zeros + n;
    halves s = {};
    bytes z = {};
    if (have == V) {
        s = *(const halves_ua *)scales;
        if constexpr (ZEROS) z = *(const bytes_ua *)zeros;
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (v >= have) continue;
            s[v] = *(const _Float16 *)(scales + v * 2);
            if constexpr (ZEROS) z[v] = zeros[v];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) words[(tid & 3) * 4 + j][64 * i + (tid >> 2)] = in[i][j];
    __syncthreads();
    if (have <= 0) return;
    unsigned char *w = (unsigned char *)a.W + e * a.stride_w + (int64_t)k0 * a.ldw + (int64_t)n * sizeof(T);
#pragma unroll
    for (int u = 0; u < WORDS; u++) {
        uint32_t word[V];
#pragma unroll
        for (int v = 0; v < V; v++) word[v] = words[((first + u) & 3) * 4 + ((first + u) >> 2)][c + v];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (u * 8 + i >= left) return;
            vec out;
#pragma unroll
            for (int v = 0; v < V; v++)
                out[v] = (T)(((float)(word[v] >> nibble_at(i) & 15) - (ZEROS ? (float)z[v] : 8.0f)) * (float)s[v]);
            unsigned char *to = w + (u * 8 + i) * a.ldw;
            if (have == V) {
                *(vec_ua *)to = out;
            } else {
#pragma unroll
                for (int v = 0; v < V; v++)
                    if (v < have) *(T *)(to + v * sizeof(T)) = out[v];
            }
        }
    }
}

// ------------------------------------------------------------------ products

struct W4Args {
    const unsigned char *A;
    float *C;
    int64_t lda, ldc;  // bytes
    Weights4 w;
    const int32_t *offsets;  // groups of rows; NULL: all rows have the first matrix
    int row_groups, rows;
    int N, K, group, blocks;
    int tiles_m, tiles_n;  // k_w4_tile
    int flags;             // TDG_DEBUG_* bits
};

// Eight codes of a word, less the zero point, as FP16 in the order of k.  1024
// + q and 1024 + 16 q are FP16's bit patterns of nibbles set below its exponent;
// both differences are exact.
__device__ __forceinline__ f16x8 code_values(uint32_t word, f16x2 z1024, f16x2 z64) {
    const uint32_t high = word >> 8;
    uint32_t above = 0x64006400u;
    asm("" : "+v"(above));  // a register: and-or is one instruction, and takes no two literals
    f16x2 v[4];
    const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    v[0] = __builtin_bit_cast(f16x2, (word & 0x000f000fu) | above) - z1024;
    v[1] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (word & 0x00f000f0u) | above), sixteenth, -z64);
    v[2] = __builtin_bit_cast(f16x2, (high & 0x000f000fu) | above) - z1024;
    v[3] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (high & 0x00f000f0u) | above), sixteenth, -z64);
    return f16x8{v[0][0], v[0][1], v[1][0], v[1][1], v[2][0], v[2][1], v[3][0], v[3][1]};
}

// Few rows: a workgroup has 16 CT columns and up to 16 MT rows, and each of its
// NW waves a run of k's blocks, which LDS joins in order.  Rows, codes and scales
// go to registers as the matrix instructions take them; the waves share nothing
// but the rows.  The loads in flight are those of many waves: a wave that loads
// two or four blocks at a time, or the next one's codes early, holds so many
// registers that it loses more (1 x 4096 x 4096: 4.3 us with one block, 5.0 with
// two or four; 16 x 8192 x 8192: 13.1, 13.7, 14.3).
template <int MT, int CT, int NW, int SPAN, bool ZEROS>
__global__ void __launch_bounds__(NW * 64) k_w4_few(W4Args p) {
    constexpr int SCALES = 4 / SPAN;  // scales of a column in a block
    __shared__ float part[NW][CT * 4 * 64];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lo = 0, hi = p.rows;
    Weights4 w = p.w;
    if (p.offsets) {
        const int g = blockIdx.y;
        lo = min(max(p.offsets[g], 0), p.rows), hi = min(max(p.offsets[g + 1], 0), p.rows);
        w.codes += g * w.stride_codes, w.scales += g * w.stride_scales, w.zeros += g * w.stride_zeros;
    }
    const int per = (p.blocks + NW - 1) / NW;
    const int b0 = min(p.blocks, wave * per), b1 = min(p.blocks, b0 + per);
    int col[CT];
#pragma unroll
    for (int t = 0; t < CT; t++) col[t] = min((int)blockIdx.x * 16 * CT + t * 16 + c, p.N - 1);
    const int step = (int)gridDim.z * 16 * MT;
    for (int m0 = lo + (int)blockIdx.z * 16 * MT; m0 < hi; m0 = next_start(m0, hi, step)) {
        const unsigned char *row[MT];  // a lane behind the last row takes that one: its sums are not stored
#pragma unroll
        for (int i = 0; i < MT; i++) row[i] = p.A + (int64_t)min(m0 + i * 16 + c, hi - 1) * p.lda + q * 16;
        f32x4 acc[MT][CT] = {};
        for (int b = b0; b < b1; b++) {
            const int k = b * BLOCK;
            u32x4 word[CT];
            _Float16 scale[SCALES][CT];
            unsigned char zero[SCALES][CT];
            const unsigned char *code = w.codes + b * w.ld_codes + q * 16;
#pragma unroll
            for (int t = 0; t < CT; t++) word[t] = *(const u32x4 *)(code + (int64_t)col[t] * 64);
#pragma unroll
            for (int g = 0; g < SCALES; g++) {
                const int64_t at = min(k + g * 32 * SPAN, p.K - 1) / p.group;
#pragma unroll
                for (int t = 0; t < CT; t++) {
                    scale[g][t] = *(const _Float16 *)(w.scales + at * w.ld_scales + (int64_t)col[t] * 2);
                    if constexpr (ZEROS) zero[g][t] = w.zeros[at * w.ld_zeros + col[t]];
                }
            }
            f16x8 x[4][MT];
            if (k + BLOCK <= p.K) {
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int i = 0; i < MT; i++)
                        x[j][i] = __builtin_bit_cast(f16x8, load16_global(row[i] + (int64_t)(k + 32 * j) * 2));
            } else {  // the end of k cuts the block: zeros behind it
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const int have = p.K - k - 32 * j - 8 * q;
                        const unsigned char *at = row[i] + (int64_t)(k + 32 * j) * 2;
                        x[j][i] = f16x8{};
                        if (have >= 8) {
                            x[j][i] = __builtin_bit_cast(f16x8, load16_global(at));
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; e++)
                                if (e < have) x[j][i][e] = *(const _Float16 *)(at + e * 2);
                        }
                    }
            }
#pragma unroll
            for (int g = 0; g < SCALES; g++) {
                if (k + g * 32 * SPAN >= p.K) break;
#pragma unroll
                for (int t = 0; t < CT; t++) {
                    f16x2 z1024 = {(_Float16)1032.0f, (_Float16)1032.0f}, z64 = {(_Float16)72.0f, (_Float16)72.0f};
                    if constexpr (ZEROS) {
                        const float z = (float)zero[g][t];
                        z1024[0] = z1024[1] = (_Float16)(z + 1024.0f), z64[0] = z64[1] = (_Float16)(z + 64.0f);
                    }
                    f32x4 sum[MT] = {};
#pragma unroll
                    for (int j = g * SPAN; j < (g + 1) * SPAN; j++) {
                        const f16x8 v = code_values(word[t][j], z1024, z64);
#pragma unroll
                        for (int i = 0; i < MT; i++)
                            sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j][i], v, sum[i], 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < MT; i++)
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            acc[i][t][r] = fmaf((float)scale[g][t], sum[i][r], acc[i][t][r]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MT; i++) {
            if (m0 + i * 16 >= hi) break;
            __syncthreads();
#pragma unroll
            for (int t = 0; t < CT; t++)
#pragma unroll
                for (int r = 0; r < 4; r++) part[wave][(t * 4 + r) * 64 + lane] = acc[i][t][r];
            __syncthreads();
            for (int e = tid; e < CT * 256; e += NW * 64) {
                const int m = m0 + i * 16 + (e >> 4 & 3) * 4 + (e >> 6 & 3);
                const int n = (int)blockIdx.x * 16 * CT + (e >> 8) * 16 + (e & 15);
                if (m >= hi || n >= p.N) continue;
                float sum = part[0][e];
#pragma unroll
                for (int v = 1; v < NW; v++) sum += part[v][e];
                *(float *)((unsigned char *)p.C + (int64_t)m * p.ldc + (int64_t)n * 4) = sum;
            }
        }
    }
}

// Many rows: a workgroup has 16 MT rows and 16 CT columns for each of its waves,
// and every wave all the rows, so that no weight is unpacked twice in a
// workgroup.  Two LDS buffers are filled by the global-to-LDS DMA, one block of
// 128 k each: A's rows (256 bytes each, 16-byte pieces at piece ^ (row % 16)), the
// waves' codes (64 bytes a column, pieces at piece ^ (column / 4 % 4); both keep
// fragment reads free of bank conflicts), and their scales and zero points, a word
// for each column.  A block's codes become fragments in registers; then row by row
// of 16 the instructions of SPAN * 32 k run on a sum of their own, which joins the
// accumulators times the scale.  What bounds it: the copies' rate from L2, which
// tall and wide tiles spare, and the vector instructions that unpack and scale, so
// that tiles small enough for two or three workgroups to a CU do better than a
// third buffer (8192 rows, 16 matrices of 4096 x 4096, groups of
// 128: 64 x 256 tiles 291-310 us, 0.9 PFLOP/s, 128 x 256 with three buffers 319; groups
// of 64 326-338, the matrix cores busy for 44% of the time and vector instructions
// issued in 75%.  4096 x 8192 x 4096: 225-239 us, 1.2 PFLOP/s, the plain FP16 product's
// rate).
template <int MT_, int CT_, int WAVES_, int SPAN_, bool ZEROS_>
struct W4Tile {
    static constexpr int MT = MT_, CT = CT_, WAVES = WAVES_, SPAN = SPAN_;
    static constexpr bool ZEROS = ZEROS_;
    static constexpr int BM = 16 * MT, BN = 16 * CT * WAVES, THREADS = 64 * WAVES;
    static constexpr int ROWS = 4 * WAVES, COPIES = BM / ROWS;  // rows of A that all waves copy at once, how often
    static constexpr int SCALES = 4 / SPAN;                     // scales of a column in a block
    // One copy takes the words of 64 lanes: scales of 64 / (16 CT) groups.
    static constexpr int AT_ONCE = 4 / CT, SCALE_COPIES = (SCALES + AT_ONCE - 1) / AT_ONCE;
    static constexpr int A_BYTES = BM * 256, CODE_BYTES = CT * 1024, SCALE_BYTES = SCALE_COPIES * 256;
    static constexpr int WAVE_BYTES = CODE_BYTES + SCALE_BYTES * (ZEROS ? 2 : 1);
    static constexpr int STAGE = A_BYTES + WAVES * WAVE_BYTES;
    static_assert(BM % ROWS == 0 && ROWS % 16 == 0, "A's rows must split evenly, and their swizzle repeat");
    static_assert(2 * STAGE <= 160 * 1024, "two buffers");
};

// As copy_to_lds, 2 bytes (1 byte) from each lane's address to the word at m0 + 4 lane.
template <int BYTES>
__device__ __forceinline__ void copy_word_to_lds(const unsigned char *src, uint32_t m0) {
    static_assert(BYTES == 1 || BYTES == 2, "what a word is made of");
    if constexpr (BYTES == 2)
        asm volatile("s_nop 0\n\tglobal_load_lds_ushort %0, off" ::"v"((uint64_t)(uintptr_t)src), "{m0}"(m0) : "memory");
    else
        asm volatile("s_nop 0\n\tglobal_load_lds_ubyte %0, off" ::"v"((uint64_t)(uintptr_t)src), "{m0}"(m0) : "memory");
}

template <class T>
__device__ __forceinline__ void w4_tile(const W4Args &p, const Weights4 &w, int x0, int hi, int y0,
                                        unsigned char *smem) {
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lds = (uint32_t)(uintptr_t)(TDG_LDS unsigned char *)smem;
    const int n0 = y0 + wave * 16 * T::CT;
    // A's copies: rows ROWS i + tid / 16, of which the last one stands for all behind it.
    const int piece = (tid & 15) ^ (tid >> 4 & 15);
    uint32_t a_off[T::COPIES];
#pragma unroll
    for (int i = 0; i < T::COPIES; i++)
        a_off[i] = (uint32_t)((int64_t)min(i * T::ROWS + (tid >> 4), hi - 1 - x0) * p.lda + piece * 16);
    const unsigned char *a_base = p.A + (int64_t)x0 * p.lda;
    // Codes and scales: columns from n0 on; the last one stands for those behind it.
    const int first = min(n0, p.N - 1), last = p.N - 1 - first;
    uint32_t code_off[T::CT];
#pragma unroll
    for (int t = 0; t < T::CT; t++)
        code_off[t] = (uint32_t)(min(t * 16 + (lane >> 2), last) * 64 + (((lane & 3) ^ (lane >> 4)) << 4));
    const unsigned char *codes = w.codes + (int64_t)first * 64;
    // The lane's next scale: its column, k, and k counted from its group's start.
    int at_k[T::SCALE_COPIES], into[T::SCALE_COPIES];
    const unsigned char *scales[T::SCALE_COPIES], *zeros[T::SCALE_COPIES];
#pragma unroll
    for (int i = 0; i < T::SCALE_COPIES; i++) {
        at_k[i] = min(i * T::AT_ONCE + lane / (16 * T::CT), T::SCALES - 1) * 32 * T::SPAN;
        const int own = min(lane % (16 * T::CT), last), g = at_k[i] / p.group;
        into[i] = at_k[i] - g * p.group;
        scales[i] = w.scales + g * w.ld_scales + (int64_t)(first + own) * 2;
        if constexpr (T::ZEROS) zeros[i] = w.zeros + g * w.ld_zeros + first + own;
    }

    // (Blocks are copied in order: each moves codes, scales and zeros on.)
    auto issue = [&](int b) {
        const uint32_t at = lds + (uint32_t)(b & 1) * T::STAGE, mine = at + T::A_BYTES + wave * T::WAVE_BYTES;
        const unsigned char *base = a_base + (int64_t)b * 256;
        const int left = p.K - b * BLOCK;
        if (left >= BLOCK) {
#pragma unroll
            for (int i = 0; i < T::COPIES; i++) copy_to_lds(base, a_off[i], at + i * T::ROWS * 256 + wave * 1024);
        } else {
            // The last block, which the end of k cuts: pieces behind it are zeros,
            // and the one that it cuts is written element by element.
            const int have = left - piece * 8;
#pragma unroll
            for (int i = 0; i < T::COPIES; i++) {
                const unsigned char *src = base + a_off[i];
                if (have >= 8 || have <= 0) {
                    copy_to_lds(have > 0 ? (uint64_t)(uintptr_t)src : (uint64_t)(uintptr_t)tdg_zero16,
                                at + i * T::ROWS * 256 + wave * 1024);
                } else {
                    f16x8 v = {};
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (e < have) v[e] = *(const _Float16 *)(src + e * 2);
                    lds_write16(smem + (b & 1) * T::STAGE + i * T::ROWS * 256 + tid * 16, __builtin_bit_cast(u32x4, v));
                }
            }
        }
#pragma unroll
        for (int t = 0; t < T::CT; t++) copy_to_lds(codes, code_off[t], mine + t * 1024);
        codes += w.ld_codes;
#pragma unroll
        for (int i = 0; i < T::SCALE_COPIES; i++) {
            // (From the end of k on there are no groups: zeros.)
            const unsigned char *none = (const unsigned char *)tdg_zero16;
            copy_word_to_lds<2>(at_k[i] < p.K ? scales[i] : none, mine + T::CODE_BYTES + i * 256);
            if constexpr (T::ZEROS)
                copy_word_to_lds<1>(at_k[i] < p.K ? zeros[i] : none, mine + T::CODE_BYTES + T::SCALE_BYTES + i * 256);
            at_k[i] += BLOCK, into[i] += BLOCK;
#pragma unroll
            for (int j = 0; j < T::SCALES; j++) {  // on to the group that holds k of the next block
                const bool on = into[i] >= p.group;
                into[i] -= on ? p.group : 0;
                scales[i] += on ? w.ld_scales : 0;
                if constexpr (T::ZEROS) zeros[i] += on ? w.ld_zeros : 0;
            }
        }
    };

    f32x4 acc[T::MT][T::CT] = {};
    if (p.blocks > 0) issue(0);
    uint32_t a_at[4];
#pragma unroll
    for (int j = 0; j < 4; j++) a_at[j] = (uint32_t)(c * 256 + (((4 * j + q) ^ c) << 4));
    for (int b = 0; b < p.blocks; b++) {
        // Block b has landed, and nobody reads the other buffer any more.
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (b + 1 < p.blocks) issue(b + 1);
        const unsigned char *at = smem + (b & 1) * T::STAGE, *mine = at + T::A_BYTES + wave * T::WAVE_BYTES;
        f16x8 v[T::CT][4];
        float scale[T::CT][T::SCALES];
        u32x4 words[T::CT];
#pragma unroll
        for (int t = 0; t < T::CT; t++) words[t] = lds_read16(mine + t * 1024 + c * 64 + ((q ^ (c >> 2)) << 4));
#pragma unroll
        for (int t = 0; t < T::CT; t++) {
            const u32x4 word = words[t];
#pragma unroll
            for (int g = 0; g < T::SCALES; g++) {
                const uint32_t bits = *(const TDG_LDS uint32_t *)(mine + T::CODE_BYTES + ((g * T::CT + t) * 16 + c) * 4);
                scale[t][g] = (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
                asm("" : "+v"(scale[t][g]));  // converted once: not by each of the products that take it
                f16x2 z1024 = {(_Float16)1032.0f, (_Float16)1032.0f}, z64 = {(_Float16)72.0f, (_Float16)72.0f};
                if constexpr (T::ZEROS) {
                    const float z = (float)*(const TDG_LDS uint32_t *)(mine + T::CODE_BYTES + T::SCALE_BYTES +
                                                                       ((g * T::CT + t) * 16 + c) * 4);
                    z1024[0] = z1024[1] = (_Float16)(z + 1024.0f), z64[0] = z64[1] = (_Float16)(z + 64.0f);
                }
#pragma unroll
                for (int j = g * T::SPAN; j < (g + 1) * T::SPAN; j++) v[t][j] = code_values(word[j], z1024, z64);
            }
        }
#pragma unroll
        for (int i = 0; i < T::MT; i++) {
            f16x8 x[4];
#pragma unroll
            for (int j = 0; j < 4; j++) x[j] = __builtin_bit_cast(f16x8, lds_read16(at + i * 4096 + a_at[j]));
#pragma unroll
            for (int g = 0; g < T::SCALES; g++) {
                f32x4 sum[T::CT] = {};
#pragma unroll
                for (int j = g * T::SPAN; j < (g + 1) * T::SPAN; j++)
#pragma unroll
                    for (int t = 0; t < T::CT; t++)
                        sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j], v[t][j], sum[t], 0, 0, 0);
#pragma unroll
                for (int t = 0; t < T::CT; t++)
#pragma unroll
                    for (int r = 0; r < 4; r++) acc[i][t][r] = fmaf(scale[t][g], sum[t][r], acc[i][t][r]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < T::MT; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int m = x0 + i * 16 + q * 4 + r;
            if (m >= hi) continue;
            float *out = (float *)((unsigned char *)p.C + (int64_t)m * p.ldc) + n0 + c;
#pragma unroll
            for (int t = 0; t < T::CT; t++)
                if (n0 + t * 16 + c < p.N) out[t * 16] = acc[i][t][r];
        }
}

// (Registers for four waves to a SIMD: two workgroups of eight waves to a CU.)
template <int MT, int CT, int WAVES, int SPAN, bool ZEROS>
__global__ void __launch_bounds__(WAVES * 64, MT == 8 ? 2 : 4) k_w4_tile(W4Args p) {
    typedef W4Tile<MT, CT, WAVES, SPAN, ZEROS> T;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * T::STAGE];
    poison_lds<2 * T::STAGE, T::THREADS>(p.flags, smem);
    Weights4 w = p.w;
    if (!p.offsets) {
        int tm, tn;
        map_tile(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
        w4_tile<T>(p, w, tm * T::BM, p.rows, tn * T::BN, smem);
        return;
    }
    GroupedArgs a;
    a.offsets = p.offsets, a.groups = p.row_groups, a.rows = p.rows, a.tiles_n = p.tiles_n;
    const GroupedTile t = find_tile<LAY_NN, T::BM, false>(a, blockIdx.x);
    if (!t.ok) return;
    w.codes += t.g * w.stride_codes, w.scales += t.g * w.stride_scales, w.zeros += t.g * w.stride_zeros;
    w4_tile<T>(p, w, t.x0, t.hi, t.tn * T::BN, smem);
}

// ------------------------------------------------------------------ host side

int launch(const void *fn, dim3 grid, int threads, void *args, void *stream) {
    void *kargs[] = {args};
    if (hipLaunchKernel(fn, grid, dim3((unsigned)threads), kargs, 0, (hipStream_t)stream) != hipSuccess)
        return TDG_ERR_LAUNCH;
    if (hipGetLastError() != hipSuccess) return TDG_ERR_LAUNCH;
    return TDG_OK;
}

// A stack of 4-bit matrices as a caller names it, and its checks.
struct Named4 {
    int64_t count, K, N, group;
    const void *codes;
    int64_t ld_codes, stride_codes;
    const void *scales;
    int64_t ld_scales, stride_scales;
    const void *zeros;
    int64_t ld_zeros, stride_zeros;

    int64_t blocks() const { return ceil_quot(K, BLOCK); }
    int64_t groups() const { return ceil_quot(K, group); }
    bool ok(bool written) const {
        if (count < 0 || !size_ok(count) || !size_ok(K) || !size_ok(N) || group < 32 || group % 32 || !size_ok(group))
            return false;
        return stack_ok(codes, count, stride_codes, blocks(), N, ld_codes, 64, written) && aligned_to(codes, 16) &&
               stack_ok(scales, count, stride_scales, groups(), N, ld_scales, 2, written) && aligned_to(scales, 2) &&
               (!zeros || stack_ok(zeros, count, stride_zeros, groups(), N, ld_zeros, 1, written));
    }
    uint64_t bytes(int i) const {
        return i == 0   ? span_bytes(blocks(), N, ld_codes, 64, count, stride_codes)
               : i == 1 ? span_bytes(groups(), N, ld_scales, 2, count, stride_scales)
                        : span_bytes(groups(), N, ld_zeros, 1, count, stride_zeros);
    }
    const void *array(int i) const { return i == 0 ? codes : i == 1 ? scales : zeros; }
    bool apart_from(const void *p, uint64_t len) const {
        for (int i = 0; i < 3; i++)
            if (overlaps(array(i), bytes(i), p, len)) return false;
        return true;
    }
    Weights4 device() const {
        Weights4 w;
        w.codes = (const unsigned char *)codes, w.scales = (const unsigned char *)scales;
        w.zeros = (const unsigned char *)zeros;
        w.ld_codes = ld_codes * 64, w.ld_scales = ld_scales * 2, w.ld_zeros = ld_zeros;
        w.stride_codes = stride_codes * 64, w.stride_scales = stride_scales * 2, w.stride_zeros = stride_zeros;
        return w;
    }
};

QuantArgs quant_args(const Named4 &q, const void *W, int64_t ldw, int64_t stride_w, int64_t es) {
    QuantArgs a;
    a.W = (const unsigned char *)W, a.ldw = ldw * es, a.stride_w = stride_w * es, a.q = q.device();
    a.K = (int)q.K, a.N = (int)q.N, a.group = (int)q.group;
    return a;
}

bool grid_ok(const dim3 &g, int64_t threads) {
    return g.y <= 65535 && g.z <= 65535 && (uint64_t)g.x * g.y * g.z <= (uint64_t)UINT32_MAX / threads;
}

dim3 grid_of(int64_t x, int64_t y, int64_t z) {  // (what does not fit is refused by grid_ok)
    auto cap = [](int64_t v) { return (unsigned)(v < 65536 ? v : 65536); };
    return dim3((unsigned)x, cap(y), cap(z));
}

struct Variant4 {
    const void *fn;
    dim3 grid;
    int threads;
};

// The kernel of a shape for the group length and with or without zero points:
// a sum takes as many matrix instructions as the groups and blocks allow.
#define TDG_W4_SPAN(KERNEL, SPAN, ...) \
    (q.zeros ? (const void *)&KERNEL<__VA_ARGS__, SPAN, true> : (const void *)&KERNEL<__VA_ARGS__, SPAN, false>)
#define TDG_W4_FN(KERNEL, ...)                                \
    (q.group % 128 == 0  ? TDG_W4_SPAN(KERNEL, 4, __VA_ARGS__) \
     : q.group % 64 == 0 ? TDG_W4_SPAN(KERNEL, 2, __VA_ARGS__) \
                         : TDG_W4_SPAN(KERNEL, 1, __VA_ARGS__))

template <int MT, int CT, int NW>
Variant4 few(const W4Args &p, const Named4 &q) {
    const int64_t z = p.offsets ? 1 : grid_dim(ceil_quot(p.rows, 16 * MT));
    return {TDG_W4_FN(k_w4_few, MT, CT, NW), grid_of(ceil_quot(q.N, 16 * CT), p.row_groups, z), NW * 64};
}

template <class T>
Variant4 tiled(W4Args &p, const Named4 &q, int64_t live, const void *fn) {
    p.tiles_m = (int)ceil_quot(p.rows, T::BM), p.tiles_n = (int)ceil_quot(q.N, T::BN);
    // (Most tiles: every group can end inside one, and needs a row for it.)
    const int64_t most = p.offsets ? ceil_quot((p.rows / T::BM + live) * p.tiles_n, 8) * 8 : (int64_t)p.tiles_m * p.tiles_n;
    return {fn, dim3(most <= INT32_MAX - 65536 ? (unsigned)most : UINT32_MAX), T::THREADS};
}

template <int MT, int CT, int WAVES>
Variant4 tiled(W4Args &p, const Named4 &q, int64_t live) {
    return tiled<W4Tile<MT, CT, WAVES, 4, false>>(p, q, live, TDG_W4_FN(k_w4_tile, MT, CT, WAVES));
}

Variant4 choose(W4Args &p, const Named4 &q, int64_t lda) {
    const W4Size size = {p.rows, p.offsets ? p.row_groups : 0, q.N, q.K, q.group, lda};
    const int64_t live = size.live();
    switch (w4_kernel(size)) {
    case W4_FEW_1_1_16: return few<1, 1, 16>(p, q);
    case W4_FEW_1_1_8: return few<1, 1, 8>(p, q);
    case W4_FEW_1_2_8: return few<1, 2, 8>(p, q);
    case W4_FEW_1_4_8: return few<1, 4, 8>(p, q);
    case W4_FEW_2_4_8: return few<2, 4, 8>(p, q);
    case W4_TILE_128_512:  // (groups of whole blocks alone)
        return tiled<W4Tile<8, 4, 8, 4, false>>(p, q, live, TDG_W4_SPAN(k_w4_tile, 4, 8, 4, 8));
    case W4_TILE_64_256: return tiled<4, 2, 8>(p, q, live);
    case W4_TILE_64_128: return tiled<4, 1, 8>(p, q, live);
    case W4_TILE_32_128: return tiled<2, 2, 4>(p, q, live);
    default: return tiled<2, 1, 4>(p, q, live);
    }
}

int run_product(int64_t row_groups, const int32_t *offsets, int64_t M, const Named4 &q, const void *A, int64_t lda,
                float *C, int64_t ldc, void *stream) {
    if (!q.ok(false) || row_groups > 1024 || !size_ok(M) || !matrix_ok(A, M, q.K, lda, 2) ||
        !matrix_ok(C, M, q.N, ldc, 4) || !aligned_to(A, 2) || !aligned_to(C, 4) || !aligned_to(offsets, 4))
        return TDG_ERR_INVALID_ARG;
    const uint64_t c_len = span_bytes(M, q.N, ldc, 4);
    if (!q.apart_from(C, c_len) || overlaps(C, c_len, A, span_bytes(M, q.K, lda, 2)) ||
        (offsets && overlaps(C, c_len, offsets, (uint64_t)(row_groups + 1) * 4)))
        return TDG_ERR_INVALID_ARG;
    if (M == 0 || q.N == 0 || row_groups == 0) return TDG_OK;
    W4Args p;
    p.A = (const unsigned char *)A, p.C = C, p.lda = lda * 2, p.ldc = ldc * 4, p.w = q.device();
    p.offsets = offsets, p.row_groups = (int)row_groups, p.rows = (int)M;
    p.N = (int)q.N, p.K = (int)q.K, p.group = (int)q.group, p.blocks = (int)q.blocks();
    p.flags = debug_flags_now();
    const Variant4 v = choose(p, q, lda);
    if (!grid_ok(v.grid, v.threads)) return TDG_ERR_UNSUPPORTED;
    const int rc = device_check();
    if (rc != TDG_OK) return rc;
    return launch(v.fn, v.grid, v.threads, &p, stream);
}

}  // namespace

extern "C" {

int tdg_w4_quantize(int64_t count, int64_t K, int64_t N, int64_t group, const uint16_t *W, int64_t ldw,
                    int64_t stride_w, uint8_t *codes, int64_t ld_codes, int64_t stride_codes, uint16_t *scales,
                    int64_t ld_scales, int64_t stride_scales, uint8_t *zeros, int64_t ld_zeros, int64_t stride_zeros,
                    void *stream) {
    const Named4 q = {count, K, N, group, codes, ld_codes, stride_codes, scales, ld_scales, stride_scales,
                      zeros, ld_zeros, stride_zeros};
    if (!q.ok(true) || !stack_ok(W, count, stride_w, K, N, ldw, 2, false) || !aligned_to(W, 2) ||
        !q.apart_from(W, span_bytes(K, N, ldw, 2, count, stride_w)) || overlaps(codes, q.bytes(0), scales, q.bytes(1)) ||
        overlaps(codes, q.bytes(0), zeros, q.bytes(2)) || overlaps(scales, q.bytes(1), zeros, q.bytes(2)))
        return TDG_ERR_INVALID_ARG;
    if (count == 0 || K == 0 || N == 0) return TDG_OK;
    QuantArgs a = quant_args(q, W, ldw, stride_w, 2);
    const dim3 scale_grid = grid_of(ceil_quot(N, 64), q.groups(), count);
    const dim3 code_grid = grid_of(ceil_quot(N, 256), q.blocks(), count);
    const bool once = group == 32 || group == 64 || group == 128;
    const bool lines = aligned_to(W, 128) && ldw % 64 == 0 && (count == 1 || stride_w % 64 == 0);
    a.run = lines ? 1 : 8;
    const dim3 once_grid = grid_of(ceil_quot(N, 64), q.blocks(), count);
    if (once ? !grid_ok(once_grid, 256) : !grid_ok(scale_grid, 256) || !grid_ok(code_grid, 256)) return TDG_ERR_UNSUPPORTED;
    int rc = device_check();
    if (rc != TDG_OK) return rc;
#define TDG_W4_ONCE(G) (zeros ? (const void *)&k_w4_quantize<G, true> : (const void *)&k_w4_quantize<G, false>)
    if (once)
        return launch(group == 32 ? TDG_W4_ONCE(32) : group == 64 ? TDG_W4_ONCE(64) : TDG_W4_ONCE(128),
                      once_grid, 256, &a, stream);
#undef TDG_W4_ONCE
    rc = launch(zeros ? (const void *)&k_w4_scales<true> : (const void *)&k_w4_scales<false>, scale_grid, 256, &a,
                stream);
    if (rc != TDG_OK) return rc;
    return launch(zeros ? (const void *)&k_w4_codes<true> : (const void *)&k_w4_codes<false>, code_grid, 256, &a,
                  stream);
}

int tdg_w4_dequantize(int out_elem, int64_t count, int64_t K, int64_t N, int64_t group, const uint8_t *codes,
                      int64_t ld_codes, int64_t stride_codes, const uint16_t *scales, int64_t ld_scales,
                      int64_t stride_scales, const uint8_t *zeros, int64_t ld_zeros, int64_t stride_zeros, void *W,
                      int64_t ldw, int64_t stride_w, void *stream) {
    if (out_elem != TDG_ELEM_F16 && out_elem != TDG_ELEM_F32) return TDG_ERR_INVALID_ARG;
    const bool half = out_elem == TDG_ELEM_F16;
    const int64_t es = half ? 2 : 4;
    const Named4 q = {count, K, N, group, codes, ld_codes, stride_codes, scales, ld_scales, stride_scales,
                      zeros, ld_zeros, stride_zeros};
    if (!q.ok(false) || !stack_ok(W, count, stride_w, K, N, ldw, es, true) || !aligned_to(W, es) ||
        !q.apart_from(W, span_bytes(K, N, ldw, es, count, stride_w)))
        return TDG_ERR_INVALID_ARG;
    if (count == 0 || K == 0 || N == 0) return TDG_OK;
    QuantArgs a = quant_args(q, W, ldw, stride_w, es);
    const dim3 grid = grid_of(ceil_quot(N, 128), q.blocks(), count);
    if (!grid_ok(grid, 256)) return TDG_ERR_UNSUPPORTED;
    const int rc = device_check();
    if (rc != TDG_OK) return rc;
    a.run = 8;
    // FP16 rows that all start at multiples of 4 bytes.
    const bool even = aligned_to(W, 4) && ldw % 2 == 0 && (count == 1 || stride_w % 2 == 0);
#define TDG_W4_VALUES(T, V) (zeros ? (const void *)&k_w4_values<T, true, V> : (const void *)&k_w4_values<T, false, V>)
    const void *fn = !half ? TDG_W4_VALUES(float, 4) : even ? TDG_W4_VALUES(_Float16, 8) : TDG_W4_VALUES(_Float16, 2);
#undef TDG_W4_VALUES
    return launch(fn, grid, 256, &a, stream);
}

int gemm_f16w4f32(int64_t M, int64_t N, int64_t K, int64_t group, const uint16_t *A, int64_t lda,
                  const uint8_t *codes, int64_t ld_codes, const uint16_t *scales, int64_t ld_scales,
                  const uint8_t *zeros, int64_t ld_zeros, float *C, int64_t ldc, void *stream) {
    const Named4 q = {1, K, N, group, codes, ld_codes, 0, scales, ld_scales, 0, zeros, ld_zeros, 0};
    return run_product(1, nullptr, M, q, A, lda, C, ldc, stream);
}

int gemm_f16w4f32_grouped(int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K, int64_t group,
                          const uint16_t *A, int64_t lda, const uint8_t *codes, int64_t ld_codes,
                          int64_t stride_codes, const uint16_t *scales, int64_t ld_scales, int64_t stride_scales,
                          const uint8_t *zeros, int64_t ld_zeros, int64_t stride_zeros, float *C, int64_t ldc,
                          void *stream) {
    const Named4 q = {groups, K, N, group, codes, ld_codes, stride_codes, scales, ld_scales, stride_scales,
                      zeros, ld_zeros, stride_zeros};
    if (groups > 0 && !offsets) return TDG_ERR_INVALID_ARG;
    return run_product(groups, offsets, M, q, A, lda, C, ldc, stream);
}

}  // extern "C"
