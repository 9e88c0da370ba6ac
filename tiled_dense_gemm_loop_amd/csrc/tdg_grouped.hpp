// tdg_grouped.hpp -- products whose rows pick their own weights, on gfx950.
//
// A's rows are sorted by group; group g holds rows [offsets[g], offsets[g+1]),
// read on the device, so no call waits for the counts.  Three products, FP16
// in and FP32 out, as an expert layer and its gradients need them:
//   NN  C[i] = A[i] . B_g          A: rows x K, B_g: K x N       (forward)
//   NT  C[i] = A[i] . B_g^T        A: rows x K, B_g: N x K       (data gradient)
//   TN  C_g  = A[g]^T . B[g]       A: rows x M, B: rows x N      (weight gradient)
//
// Both operands are staged in LDS as they sit in memory, in one of two images
// of 64 k per tile, and read as MFMA fragments (v_mfma_f32_32x32x16_f16: lane
// l holds row or column l % 32, k = 8 (l / 32) .. + 7 of the step's 16):
//   rows of k (KC)     BX rows of 128 bytes, fragments by ds_read_b128;
//   rows at one k (RC) 64 rows of BX elements, fragments by two transposing
//                      ds_read_b64_tr_b16.
// NN takes (KC, RC), NT (KC, KC), TN (RC, RC).  The 16-byte-chunk swizzles are
// those of the plain product's tiles: fragment reads and chunk writes are free
// of bank conflicts.
#pragma once

#include "tdg_kernels.hpp"

namespace tdg {

enum { LAY_NN = 0, LAY_NT = 1, LAY_TN = 2 };

// Leading dimensions and strides in bytes.
struct GroupedArgs {
    const unsigned char *A, *B;
    unsigned char *C;
    int64_t lda, ldb, ldc;
    int64_t stride_b, stride_c;  // between groups (NN, NT: of B; TN: of C)
    const int32_t *offsets;      // groups + 1, on the device
    int groups;
    int rows;      // rows of A (TN: and of B; the groups cut the sum)
    int M, N, K;   // M: TN only (columns of A); K: NN and NT only
    int tiles_m;   // TN only: ceil(M / BM)
    int tiles_n;   // ceil(N / BN)
};

// One operand's LDS image: BX rows (or columns) of the product, 64 k.
template <bool KC, int BX>
struct Image {
    static constexpr int BYTES = BX * 128;
    static constexpr int CHUNKS = BYTES / 16;
    static constexpr int ROWB = KC ? 128 : BX * 2;  // bytes per image row
    static constexpr int CPR = ROWB / 16;           // chunks per image row
    static constexpr int RP = ROWB >= 256 ? 1 : 256 / ROWB;  // rows per 256-byte bank line
    static_assert(KC || RP <= 4, "a transposing read spans four k rows");
    // XOR on the chunk index of image row r.  KC: sixteen rows read at one
    // chunk land on sixteen bank slots.  RC: the four k rows of a transposing
    // read, four chunks each, land on distinct slots.
    __device__ static __forceinline__ int swz(int r) {
        return KC ? (r / RP) % CPR : ((r / RP) % (4 / RP)) * 4;
    }
    static_assert(KC || (4 / RP) * 4 <= CPR, "the swizzle must stay inside a row");
    // Offset of lane's fragment of k step s (16 k) and of the 32 rows or
    // columns from x0 on; RC takes the read at `h` = 0 and 1.
    __device__ static __forceinline__ uint32_t frag(int lane, int x0, int s, int h) {
        if (KC) {
            const int r = x0 + (lane & 31);
            return (uint32_t)(r * ROWB + (((2 * s + (lane >> 5)) ^ swz(r)) * 16));
        }
        const int k = s * 16 + (lane >> 5) * 8 + h * 4 + ((lane & 15) >> 2);
        const int byte = (x0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;
        return (uint32_t)(k * ROWB + (((byte >> 4) ^ swz(k)) << 4) + (byte & 15));
    }
    __device__ static __forceinline__ u32x4 read(const unsigned char *img, int lane, int x0, int s) {
        if constexpr (KC) return lds_read16(img + frag(lane, x0, s, 0));
        else return Mfma<DT_F16>::read_b(img + frag(lane, x0, s, 0), img + frag(lane, x0, s, 1));
    }
};

// Where a workgroup works: its group, the group's rows [lo, hi) and its tile.
struct GroupedTile {
    int g, lo, hi, tm, tn;
    bool ok;
};

__device__ static __forceinline__ int group_offset(const GroupedArgs &a, int g) {
    return min(max(a.offsets[g], 0), a.rows);
}

// Tile order inside a tiles_m x tiles_n block: groups of four tile rows, so
// that workgroups running together share A's and B's panels in L2.
__device__ static __forceinline__ void order_tile(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int per_group = 4 * tiles_n;
    const int first = id / per_group * 4;
    const int gm = min(tiles_m - first, 4);
    const int r = id - first * tiles_n;
    tm = first + r % gm;
    tn = r / gm;
}

// Workgroup -> tile.  Tiles are numbered group by group; workgroups are dealt
// round-robin to the 8 XCDs, so workgroup b takes tile (b % 8) * ceil(total / 8)
// + b / 8: every XCD works on a run of tiles and reads each group's B into its
// own L2 once.  For NN and NT the tile counts depend on the offsets: every
// wave sums them itself (64 lanes, a run of groups each), which costs less
// than a launch that would write them down.  The grid is sized for the most
// tiles that the rows can make; workgroups past the total end at once.
template <int LAY, int BM>
__device__ static __forceinline__ GroupedTile find_tile(const GroupedArgs &a) {
    GroupedTile t;
    t.ok = false;
    const int b = blockIdx.x;
    if constexpr (LAY == LAY_TN) {
        const int per_g = a.tiles_m * a.tiles_n;
        const int total = a.groups * per_g, per = (total + 7) >> 3;
        const int id = (b & 7) * per + (b >> 3);
        if ((b >> 3) >= per || id >= total) return t;
        t.g = id / per_g;
        order_tile(id - t.g * per_g, a.tiles_m, a.tiles_n, t.tm, t.tn);
        t.lo = group_offset(a, t.g);
        t.hi = max(t.lo, group_offset(a, t.g + 1));
        t.ok = true;
        return t;
    }
    const int lane = threadIdx.x & 63;
    const int run = (a.groups + 63) >> 6;
    const int g0 = min(a.groups, lane * run), g1 = min(a.groups, g0 + run);
    int mine = 0;
    if (g0 < g1) {
        int lo = group_offset(a, g0);
        for (int g = g0; g < g1; g++) {
            const int hi = group_offset(a, g + 1);
            mine += (max(hi - lo, 0) + BM - 1) / BM;
            lo = hi;
        }
    }
    int incl = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(incl, d);
        if (lane >= d) incl += up;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63) * a.tiles_n, per = (total + 7) >> 3;
    const int id = (b & 7) * per + (b >> 3);
    if ((b >> 3) >= per || id >= total) return t;
    const int row_tile = id / a.tiles_n;  // only to find the group: every group has whole runs of tiles_n
    const unsigned long long at = __ballot(incl > row_tile);
    const int owner = __builtin_amdgcn_readfirstlane(__ffsll(at) - 1);
    int first = __builtin_amdgcn_readlane(incl - mine, owner);  // row tiles before group g
    int g = min(a.groups, owner * run);
    int lo = group_offset(a, g), hi, tiles;
    for (;; g++) {
        hi = group_offset(a, g + 1);
        tiles = (max(hi - lo, 0) + BM - 1) / BM;
        if (row_tile < first + tiles || g + 1 >= a.groups) break;
        first += tiles;
        lo = hi;
    }
    t.g = g, t.lo = lo, t.hi = hi;
    // Offsets that do not ascend break the numbering; such a workgroup ends
    // here rather than work outside [lo, hi).
    const int local = id - first * a.tiles_n;
    if (local < 0 || local >= tiles * a.tiles_n) return t;
    order_tile(local, tiles, a.tiles_n, t.tm, t.tn);
    t.ok = true;
    return t;
}

// Accumulators -> C: lane l of a 32x32 block holds column l % 32 of rows
// 8 (v / 4) + 4 (l / 32) + v % 4.
template <int MI, int NI>
__device__ static __forceinline__ void store_tile(unsigned char *C, int64_t ldc, int row0, int row_end, int col0,
                                                  int col_end, const f32x16 (&acc)[MI][NI]) {
    const int lane = threadIdx.x & 63;
    const int rq = (lane >> 5) * 4;
    const bool inside = row0 + MI * 32 <= row_end && col0 + NI * 32 <= col_end;
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int ni = 0; ni < NI; ni++) {
            const int col = col0 + ni * 32 + (lane & 31);
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int row = row0 + mi * 32 + (v >> 2) * 8 + rq + (v & 3);
                if (inside || (row < row_end && col < col_end))
                    *(float *)(C + (int64_t)row * ldc + (int64_t)col * 4) = acc[mi][ni][v];
            }
        }
}

// Any sizes, strides and alignments: tiles go through registers, tile t+1
// loading while tile t is computed, two LDS buffers.  A 16-byte chunk that a
// row's end cuts is read element by element, so no byte outside an operand's
// rows is ever read; what lies outside is zero in LDS.
template <int LAY, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM *WN * 64, 1) tdg_grouped_any(GroupedArgs a) {
    typedef Image<LAY != LAY_TN, BM> IA;
    typedef Image<LAY == LAY_NT, BN> IB;
    constexpr int NT = WM * WN * 64;
    constexpr int CA = IA::CHUNKS / NT, CB = IB::CHUNKS / NT;
    static_assert(IA::CHUNKS % NT == 0 && IB::CHUNKS % NT == 0, "tile must split evenly over threads");
    constexpr int WTM = BM / WM, WTN = BN / WN, MI = WTM / 32, NI = WTN / 32;
    constexpr int STAGE = IA::BYTES + IB::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * STAGE];

    const GroupedTile t = find_tile<LAY, BM>(a);
    if (!t.ok) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    // The product's rows are x in [x0, x_end) of A, its columns y in [y0, N)
    // of B, its k in [k_lo, k_hi).
    const int x0 = LAY == LAY_TN ? t.tm * BM : t.lo + t.tm * BM, x_end = LAY == LAY_TN ? a.M : t.hi;
    const int y0 = t.tn * BN, y_end = a.N;
    const int k_lo = LAY == LAY_TN ? t.lo : 0, k_hi = LAY == LAY_TN ? t.hi : a.K;
    const unsigned char *A = a.A, *B = a.B + (LAY == LAY_TN ? 0 : (int64_t)t.g * a.stride_b);
    const int nt = (k_hi - k_lo + 63) / 64;

    auto load = [&](const unsigned char *P, int64_t ld, bool kc, int q, int cpr, int swz, int x, int x_hi,
                    int k0) -> u32x4 {
        const int r = q / cpr, c = ((q % cpr) ^ swz) * 8;
        const int row = kc ? x + r : k0 + r, row_hi = kc ? x_hi : k_hi;
        const int col = kc ? k0 + c : x + c, col_hi = kc ? k_hi : x_hi;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (row < row_hi && col < col_hi) {
            const unsigned char *p = P + (int64_t)row * ld + (int64_t)col * 2;
            const int left = col_hi - col;
            if (left >= 8) {
                v = load16_global(p);
            } else {
#pragma unroll
                for (int e = 0; e < 7; e++)
                    if (e < left) {
                        const uint32_t b = *(const TDG_GLOBAL uint16_t *)(p + 2 * e);
                        v[e / 2] |= b << (16 * (e & 1));
                    }
            }
        }
        return v;
    };
    u32x4 ra[CA], rb[CB];
    auto load_tile = [&](int kt) {
        const int k0 = k_lo + kt * 64;
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int q = i * NT + tid;
            ra[i] = load(A, a.lda, LAY != LAY_TN, q, IA::CPR, IA::swz(q / IA::CPR), x0, x_end, k0);
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int q = i * NT + tid;
            rb[i] = load(B, a.ldb, LAY == LAY_NT, q, IB::CPR, IB::swz(q / IB::CPR), y0, y_end, k0);
        }
    };
    auto store_lds = [&](unsigned char *st) {
#pragma unroll
        for (int i = 0; i < CA; i++) lds_write16(st + (i * NT + tid) * 16, ra[i]);
#pragma unroll
        for (int i = 0; i < CB; i++) lds_write16(st + IA::BYTES + (i * NT + tid) * 16, rb[i]);
    };

    f32x16 acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int ni = 0; ni < NI; ni++) acc[mi][ni] = f32x16{};
    if (nt > 0) {
        load_tile(0);
        store_lds(smem);
        __syncthreads();
        for (int kt = 0; kt < nt; kt++) {
            if (kt + 1 < nt) load_tile(kt + 1);
            const unsigned char *st = smem + (kt & 1) * STAGE;
#pragma unroll
            for (int s = 0; s < 4; s++) {
                u32x4 fa[MI], fb[NI];
#pragma unroll
                for (int mi = 0; mi < MI; mi++) fa[mi] = IA::read(st, lane, wm * WTM + mi * 32, s);
#pragma unroll
                for (int ni = 0; ni < NI; ni++) fb[ni] = IB::read(st + IA::BYTES, lane, wn * WTN + ni * 32, s);
#pragma unroll
                for (int mi = 0; mi < MI; mi++)
#pragma unroll
                    for (int ni = 0; ni < NI; ni++)
                        acc[mi][ni] = Mfma<DT_F16>::mac_sub(fa[mi], fb[ni], acc[mi][ni], 0);
            }
            if (kt + 1 < nt) {
                store_lds(smem + ((kt + 1) & 1) * STAGE);
                __syncthreads();
            }
        }
    }
    unsigned char *C = a.C + (LAY == LAY_TN ? (int64_t)t.g * a.stride_c : 0);
    store_tile<MI, NI>(C, a.ldc, x0 + wm * WTM, x_end, y0 + wn * WTN, y_end, acc);
}

}  // namespace tdg
