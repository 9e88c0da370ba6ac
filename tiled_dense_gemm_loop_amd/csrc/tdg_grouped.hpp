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

#include "tdg_check.h"
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
    int tiles_most;  // no tile has this number or a higher one
    uint64_t a_stop, b_stop;  // chunks end at this address or below (chunk_stop)
    int b_each;      // NN, NT: each group's B has a stop of its own (stops_each)
    int warm;        // read A and B once at the start (tdg_grouped_tn_loop)
    int flags;       // TDG_DEBUG_* bits
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

// threadIdx.x as a value of its own: in a loop over tiles, what is computed
// from it is computed again for each tile rather than kept in registers.
__device__ static __forceinline__ int thread_again() {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    return tid;
}

// Where a workgroup works: its group, the group's rows [lo, hi), the tile's
// first row (TN: column of A) and its column tile.
struct GroupedTile {
    int g, lo, hi, x0, tn;
    int half;  // -1: the whole tile; 0, 1: its left or right half (CUT)
    bool ok;
};

__device__ static __forceinline__ int group_offset(const GroupedArgs &a, int g) {
    // through the scalar cache: it does not touch the count of copies in flight
    typedef const int32_t __attribute__((address_space(4))) * Table;
    return min(max(((Table)(uintptr_t)a.offsets)[g], 0), a.rows);
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

// Workgroup b of a run of `total` tiles -> tile: workgroups are dealt round-
// robin to the 8 XCDs, so b takes tile (b % 8) * ceil(total / 8) + b / 8:
// every XCD works on a run of tiles and reads a group's B into its own L2 once.
// -1: none.
__device__ static __forceinline__ int xcd_tile(int b, int total) {
    const int per = (total + 7) >> 3, id = (b & 7) * per + (b >> 3);
    return (b >> 3) < per && id < total ? id : -1;
}

// The same where a CU holds one workgroup: when the last round of an XCD's 32
// CUs would have work for half of them or fewer, its tiles are cut in two,
// left and right.  `half`: -1 for a whole tile, else which half.
__device__ static __forceinline__ int xcd_tile_cut(int b, int total, int &half) {
    const int per = (total + 7) >> 3, last = per & 31, whole = last <= 16 ? per - last : per;
    int j = b >> 3;
    half = -1;
    if (j >= whole) {
        half = (j - whole) & 1;
        j = whole + ((j - whole) >> 1);
    }
    const int id = (b & 7) * per + j;
    return j < per && id < total ? id : -1;
}

// Workgroup -> tile.  Tiles are numbered group by group.  For NN and NT the
// tile counts depend on the offsets: every wave sums them itself (64 lanes, a
// run of groups each), which costs less than a launch that would write them
// down.  The grid is sized for the most tiles that the rows can make;
// workgroups past the total end at once.
template <int LAY, int BM, bool CUT>
__device__ static __forceinline__ GroupedTile find_tile(const GroupedArgs &a, int b) {
    GroupedTile t;
    t.ok = false;
    t.half = -1;
    if constexpr (LAY == LAY_TN) {
        const int per_g = a.tiles_m * a.tiles_n;
        const int id = xcd_tile(b, a.groups * per_g);
        if (id < 0) return t;
        t.g = id / per_g;
        int tm;
        order_tile(id - t.g * per_g, a.tiles_m, a.tiles_n, tm, t.tn);
        t.x0 = tm * BM;
        t.lo = group_offset(a, t.g);
        t.hi = max(t.lo, group_offset(a, t.g + 1));
        t.ok = true;
        return t;
    }
    const int lane = thread_again() & 63;
    const int run = (a.groups + 63) >> 6;
    const int g0 = min(a.groups, lane * run), g1 = min(a.groups, g0 + run);
    int mine = 0;  // row tiles of the lane's groups
    if (g0 < g1) {
        int lo = group_offset(a, g0);
        for (int g = g0; g < g1; g++) {
            const int hi = group_offset(a, g + 1), len = max(hi - lo, 0);
            mine += (len + BM - 1) / BM;
            lo = hi;
        }
    }
    int upto = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(upto, d);
        if (lane >= d) upto += up;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63) * a.tiles_n;
    const int id = CUT ? xcd_tile_cut(b, total, t.half) : xcd_tile(b, total);
    if (id < 0) return t;
    const int at = id / a.tiles_n;  // its row tile, counted over all groups
    const int owner = __builtin_amdgcn_readfirstlane(__ffsll(__ballot(upto > at)) - 1);
    int first = __builtin_amdgcn_readlane(upto - mine, owner);  // row tiles before group g
    int g = min(a.groups - 1, owner * run);
    int lo = group_offset(a, g), hi, tiles;
    for (;; g++) {
        hi = group_offset(a, g + 1);
        tiles = (max(hi - lo, 0) + BM - 1) / BM;
        if (at < first + tiles || g + 1 >= a.groups) break;
        first += tiles;
        lo = hi;
    }
    // Offsets that do not ascend break the numbering; such a workgroup ends
    // here rather than work outside [lo, hi).
    const int local = id - first * a.tiles_n;
    if (local < 0 || local >= tiles * a.tiles_n) return t;
    t.g = g, t.lo = lo, t.hi = hi;
    int tm;
    order_tile(local, tiles, a.tiles_n, tm, t.tn);
    t.x0 = lo + tm * BM;
    t.ok = true;
    return t;
}

// Accumulators -> C: lane l of a 32x32 block holds column l % 32 of rows
// 8 (v / 4) + 4 (l / 32) + v % 4.  Where C's rows are whole 128-byte lines the
// stores stream past the caches, which leaves those to A and B (8192 rows, 32
// groups, 2048 x 4000, TN: 377 us without, 258 with; 3999 columns, whose rows
// share lines: 487 without, 815 with).  Returns whether the tile was stored
// whole.
template <int MI, int NI>
__device__ static __forceinline__ bool store_tile(unsigned char *C, int64_t ldc, int row0, int row_end, int col0,
                                                  int col_end, const f32x16 (&acc)[MI][NI]) {
    const int lane = thread_again() & 63;
    const int rq = (lane >> 5) * 4;
    auto store = [&](auto masked, auto streaming) __attribute__((always_inline)) {
#pragma unroll
        for (int mi = 0; mi < MI; mi++)
#pragma unroll
            for (int ni = 0; ni < NI; ni++) {
                const int col = col0 + ni * 32 + (lane & 31);
#pragma unroll
                for (int v = 0; v < 16; v++) {
                    const int row = row0 + mi * 32 + (v >> 2) * 8 + rq + (v & 3);
                    if (decltype(masked)::value && (row >= row_end || col >= col_end)) continue;
                    float *p = (float *)(C + (int64_t)row * ldc + (int64_t)col * 4);
                    if constexpr (decltype(streaming)::value) __builtin_nontemporal_store(acc[mi][ni][v], p);
                    else *p = acc[mi][ni][v];
                }
            }
    };
    const bool inside = row0 + MI * 32 <= row_end && col0 + NI * 32 <= col_end;
    const bool lines = (((uintptr_t)C | (uint64_t)ldc) & 127) == 0;
    if (inside && lines) store(std::false_type{}, std::true_type{});
    else if (inside) store(std::false_type{}, std::false_type{});
    else store(std::true_type{}, std::false_type{});
    return inside;
}

// Where A's rows are: row x of the product at `off(x)` bytes from A.  RowsFrom:
// one after the other, row x0 at A itself; RowsBy: row x is A's row list[x].
struct RowsFrom {
    int x0;
    int64_t ld;
    __device__ __forceinline__ int64_t off(int x) const { return (int64_t)(x - x0) * ld; }
};
struct RowsBy {
    const int32_t *list;
    int64_t ld;
    __device__ __forceinline__ int64_t off(int x) const { return (int64_t)list[x] * ld; }
};

// One operand chunk of eight elements of the row at `row`, any size, stride
// and alignment: a whole chunk is one 16-byte load, one that the row's end
// cuts is read element by element, so no byte outside the rows is ever read;
// what lies outside is zero.
__device__ static __forceinline__ u32x4 load_chunk(const unsigned char *row, bool row_ok, int col, int col_end) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (row_ok && col < col_end) {
        const unsigned char *p = row + (int64_t)col * 2;
        const int left = col_end - col;
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
}

// Any sizes, strides and alignments: tiles go through registers, tile t+1
// loading while tile t is computed, two LDS buffers.
template <int LAY, int BM, int BN, int WM, int WN>
struct GroupedAny {
    typedef Image<LAY != LAY_TN, BM> IA;
    typedef Image<LAY == LAY_NT, BN> IB;
    static constexpr int NT = WM * WN * 64;
    static constexpr int CA = IA::CHUNKS / NT, CB = IB::CHUNKS / NT;
    static constexpr int WTM = BM / WM, WTN = BN / WN, MI = WTM / 32, NI = WTN / 32;
    static constexpr int STAGE = IA::BYTES + IB::BYTES, SMEM = 2 * STAGE;
    static_assert(IA::CHUNKS % NT == 0 && IB::CHUNKS % NT == 0, "tile must split evenly over threads");

    // acc += the tile's product over k in [k_lo, k_hi).  Rows (TN: columns) of
    // A from x0 to x_end, found by `rows` (TN: not used); columns (NT: rows)
    // of B from y0 to y_end.
    template <class Rows>
    __device__ static __forceinline__ void run(const unsigned char *A, int64_t lda, Rows rows,
                                               const unsigned char *B, int64_t ldb, int x0, int x_end, int y0,
                                               int y_end, int k_lo, int k_hi, uint64_t, uint64_t,
                                               unsigned char *smem, f32x16 (&acc)[MI][NI]) {
        const int nt = (k_hi - k_lo + 63) >> 6;
        if (nt <= 0) return;
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave % WM, wn = wave / WM;
        u32x4 ra[CA], rb[CB];
        auto load_tile = [&](int kt) {
            const int k0 = k_lo + kt * 64;
#pragma unroll
            for (int i = 0; i < CA; i++) {
                const int q = i * NT + tid, r = q / IA::CPR, c = ((q % IA::CPR) ^ IA::swz(r)) * 8;
                if (LAY == LAY_TN)
                    ra[i] = load_chunk(A + (int64_t)(k0 + r) * lda, k0 + r < k_hi, x0 + c, x_end);
                else
                    ra[i] = load_chunk(A + rows.off(min(x0 + r, x_end - 1)), x0 + r < x_end, k0 + c, k_hi);
            }
#pragma unroll
            for (int i = 0; i < CB; i++) {
                const int q = i * NT + tid, r = q / IB::CPR, c = ((q % IB::CPR) ^ IB::swz(r)) * 8;
                rb[i] = LAY == LAY_NT ? load_chunk(B + (int64_t)(y0 + r) * ldb, y0 + r < y_end, k0 + c, k_hi)
                                      : load_chunk(B + (int64_t)(k0 + r) * ldb, k0 + r < k_hi, y0 + c, y_end);
            }
        };
        auto store_lds = [&](unsigned char *st) {
#pragma unroll
            for (int i = 0; i < CA; i++) lds_write16(st + (i * NT + tid) * 16, ra[i]);
#pragma unroll
            for (int i = 0; i < CB; i++) lds_write16(st + IA::BYTES + (i * NT + tid) * 16, rb[i]);
        };
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
};

// Global-to-LDS DMA (global_load_lds_dwordx4, from any byte address), a ring
// of STAGES buffers with STAGES - 1 tiles in flight, fragments read three k
// steps ahead and the copies of a later tile spread over the MFMAs of two
// steps: the schedule of the plain product's direct loop.  Edges cost no test
// in the loop: a lane whose row or column lies past the tile's end copies the
// last one instead (it only feeds C elements that are not stored), and only
// the tile that the end of k cuts takes its chunks past that end from a block
// of zeros.  Chunks that start inside a row are copied whole: what they hold
// past a row's end feeds C elements that are not stored, or, where the row
// runs along k, is cleared in LDS.  Past an operand's last byte they read only
// within its 4 KiB page: where its last chunk would leave it (a_stop, b_stop),
// the last K tile takes that chunk from the block of zeros too, and its lane
// writes the elements to LDS once the tile has landed.  (A matrix of an even
// count of odd rows often ends with a page: 16384 rows, 16 groups of 4096 x 4095
// 625 us, through registers 1174; 64 rows, 32 groups of 2048 x 2047 45 and 245.)
template <int LAY, int BM, int BN, int WM, int WN, int STAGES>
struct GroupedRing {
    typedef Image<LAY != LAY_TN, BM> IA;
    typedef Image<LAY == LAY_NT, BN> IB;
    static constexpr int NT = WM * WN * 64;
    static constexpr int CA = IA::CHUNKS / NT, CB = IB::CHUNKS / NT, ND = CA + CB;
    static constexpr int WTM = BM / WM, WTN = BN / WN, MI = WTM / 32, NI = WTN / 32;
    static constexpr int STAGE = IA::BYTES + IB::BYTES, SMEM = STAGES * STAGE;
    static constexpr int A_STEP = NT / IA::CPR, B_STEP = NT / IB::CPR;  // image rows per chunk index
    static constexpr int AHEAD = STAGES - 1;
    static_assert(IA::CHUNKS % NT == 0 && IB::CHUNKS % NT == 0, "tile must split evenly over threads");
    static_assert(A_STEP % 16 == 0 || (LAY == LAY_TN && A_STEP % 4 == 0), "A swizzle must repeat");
    static_assert(B_STEP % 16 == 0 || (LAY != LAY_NT && B_STEP % 4 == 0), "B swizzle must repeat");
    static_assert(STAGES >= 2 && STAGES <= 4 && AHEAD * ND <= 63 && SMEM <= 160 * 1024, "ring");

    static constexpr bool AKC = LAY != LAY_TN, BKC = LAY == LAY_NT;
    static constexpr int FD = 3;                   // k steps that fragments are read ahead
    static constexpr int STORES = MI * NI * 16;    // store instructions of a whole tile, per wave

    // A tile's copies: per-lane byte offsets of the thread's chunks from the
    // tile's first row and k.  KC: one per chunk (the rows are clamped); RC:
    // one for all (the k rows advance with the wave-uniform base).
    uint32_t a_off[AKC ? CA : 1], b_off[BKC ? CB : 1];
    const unsigned char *a_base, *b_base;
    int64_t lda, ldb;
    int len, nt;       // k of the tile, and its K tiles
    uint64_t a_stop, b_stop;
    uint32_t lds_at;   // where the wave's first chunks go in the first buffer

    // As GroupedAny::run; here `rows` gives offsets below 2^32.
    template <class Rows>
    __device__ static __forceinline__ void run(const unsigned char *A, int64_t lda, Rows rows,
                                               const unsigned char *B, int64_t ldb, int x0, int x_end, int y0,
                                               int y_end, int k_lo, int k_hi, uint64_t a_stop, uint64_t b_stop,
                                               unsigned char *smem, f32x16 (&acc)[MI][NI]) {
        GroupedRing r;
        r.aim(A, lda, rows, B, ldb, x0, x_end, y0, y_end, k_lo, k_hi, a_stop, b_stop, smem);
        r.start();
        r.finish(smem, acc, false);
    }

    template <class Rows>
    __device__ __forceinline__ void aim(const unsigned char *A, int64_t lda_, Rows rows, const unsigned char *B,
                                        int64_t ldb_, int x0, int x_end, int y0, int y_end, int k_lo, int k_hi,
                                        uint64_t a_stop_, uint64_t b_stop_, unsigned char *smem) {
        lds_at = (uint32_t)(uintptr_t)(TDG_LDS unsigned char *)smem +
                 (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024u;
        lda = lda_, ldb = ldb_;
        a_stop = a_stop_, b_stop = b_stop_;
        len = k_hi - k_lo;
        nt = (len + 63) >> 6;
        if (nt <= 0) return;
        const int tid = thread_again();
        const int a_r = tid / IA::CPR, a_c = (tid % IA::CPR) ^ IA::swz(a_r);
        const int b_r = tid / IB::CPR, b_c = (tid % IB::CPR) ^ IB::swz(b_r);
#pragma unroll
        for (int i = 0; i < (AKC ? CA : 1); i++)
            a_off[i] = AKC ? (uint32_t)(rows.off(min(x0 + i * A_STEP + a_r, x_end - 1)) + a_c * 16)
                           : (uint32_t)(a_r * lda + min(a_c * 8, (x_end - 1 - x0) & ~7) * 2);
#pragma unroll
        for (int i = 0; i < (BKC ? CB : 1); i++)
            b_off[i] = BKC ? (uint32_t)(min(i * B_STEP + b_r, y_end - 1 - y0) * ldb + b_c * 16)
                           : (uint32_t)(b_r * ldb + min(b_c * 8, (y_end - 1 - y0) & ~7) * 2);
        a_base = A + (AKC ? (int64_t)k_lo * 2 : (int64_t)k_lo * lda + (int64_t)x0 * 2);
        b_base = B + (BKC ? (int64_t)y0 * ldb + (int64_t)k_lo * 2 : (int64_t)k_lo * ldb + (int64_t)y0 * 2);
    }

    __device__ static __forceinline__ uint32_t stage(int t) { return (uint32_t)((t % STAGES) * STAGE); }

    // Whether the last K tile needs looking after: the end of k cuts it, or an
    // operand's last chunk is kept off the DMA.
    __device__ __forceinline__ bool edge() const { return (a_stop & b_stop) != ~(uint64_t)0; }
    __device__ __forceinline__ bool cut() const { return (len & 63) != 0 || edge(); }

    // Where chunk set d (A's first, then B's) of K tile kt is.
    __device__ __forceinline__ const unsigned char *base_of(int kt, int d) const {
        const bool is_a = d < CA;
        const int i = is_a ? d : d - CA;
        return is_a ? a_base + (AKC ? (int64_t)kt * 128 : (int64_t)(kt * 64 + i * A_STEP) * lda)
                    : b_base + (BKC ? (int64_t)kt * 128 : (int64_t)(kt * 64 + i * B_STEP) * ldb);
    }
    __device__ __forceinline__ uint32_t off_of(int d) const {
        return d < CA ? a_off[AKC ? d : 0] : b_off[BKC ? d - CA : 0];
    }
    // The lane's chunk of the set, and whether it begins before the end of k.
    __device__ __forceinline__ bool chunk_of(int kt, int d, uint64_t &p) const {
        const bool is_a = d < CA;
        const int i = is_a ? d : d - CA;
        const int tid = thread_again();
        const int a_r = tid / IA::CPR, a_c = (tid % IA::CPR) ^ IA::swz(a_r);
        const int b_r = tid / IB::CPR, b_c = (tid % IB::CPR) ^ IB::swz(b_r);
        // first k of the chunk, counted from the tile's
        const int k = is_a ? (AKC ? a_c * 8 : i * A_STEP + a_r) : (BKC ? b_c * 8 : i * B_STEP + b_r);
        p = (uint64_t)(uintptr_t)(base_of(kt, d) + off_of(d));
        return k < len - kt * 64;
    }

    // Copies chunk set d of K tile kt into its buffer.
    template <bool CHECKED>
    __device__ __forceinline__ void issue(int kt, int d) const {
        const uint32_t m0 = lds_at + stage(kt) + (uint32_t)((d < CA ? 0 : IA::BYTES) + (d < CA ? d : d - CA) * NT * 16);
        kt = __builtin_amdgcn_readfirstlane(kt);
        if constexpr (CHECKED) {
            uint64_t p;
            const bool in = chunk_of(kt, d, p) && p + 16 <= (d < CA ? a_stop : b_stop);
            const uint64_t src = in ? p : (uint64_t)(uintptr_t)tdg_zero16;
            copy_to_lds(src, m0);
        } else {
            copy_to_lds(base_of(kt, d), off_of(d), m0);
        }
    }

    // The first tiles into the buffers, all of which are free.  (Not unrolled:
    // a workgroup that runs once waits for its instructions too.)
    __device__ __forceinline__ void start() const {
#pragma unroll 1
        for (int p = 0; p < min(STAGES, nt); p++) {
            if (cut() && p == nt - 1) {
#pragma unroll
                for (int d = 0; d < ND; d++) issue<true>(p, d);
            } else {
#pragma unroll
                for (int d = 0; d < ND; d++) issue<false>(p, d);
            }
        }
    }

    // Waits until at most the n youngest tiles are still in flight.
    __device__ static __forceinline__ void wait_tiles(int n) {
        if (n >= AHEAD) wait_vmcnt<AHEAD * ND>();
        else if (AHEAD > 2 && n == 2) wait_vmcnt<2 * ND <= 63 ? 2 * ND : 0>();
        else if (AHEAD > 1 && n == 1) wait_vmcnt<ND <= 63 ? ND : 0>();
        else wait_vmcnt<0>();
    }

    // What the last K tile lacks when it has landed.  Chunks that were kept off
    // the DMA: each lane writes what there is of its own.  Rows along k whose
    // end splits a chunk: its elements from that end on are cleared, one thread
    // per row.
    __device__ __forceinline__ void mend_last(unsigned char *smem, int t) const {
        if (t != nt - 1) return;
        if (edge()) {
#pragma unroll
            for (int d = 0; d < ND; d++) {
                uint64_t p;
                const uint64_t stop = d < CA ? a_stop : b_stop;
                if (!chunk_of(t, d, p) || p + 16 <= stop) continue;
                u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 7; e++)
                    if (p + 2 * e < stop) v[e / 2] |= (uint32_t)*(const TDG_GLOBAL uint16_t *)(p + 2 * e) << (16 * (e & 1));
                lds_write16(smem + stage(t) + (d < CA ? 0 : IA::BYTES) + ((d < CA ? d : d - CA) * NT + threadIdx.x) * 16, v);
            }
            __syncthreads();
        }
        const int split = AKC || BKC ? len & 7 : 0;
        if (split == 0) return;
        const int c = (len & 63) >> 3;
        auto clear = [&](unsigned char *p) __attribute__((always_inline)) {
            const u32x4 v = lds_read16(p);
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int left = split - 2 * j;  // elements of word j that stay
                w[j] = v[j] & (left >= 2 ? ~0u : left == 1 ? 0xffffu : 0u);
            }
            lds_write16(p, w);
        };
        unsigned char *st = smem + stage(t);
        if (AKC)
            for (int r = threadIdx.x; r < BM; r += NT) clear(st + r * 128 + ((c ^ IA::swz(r)) << 4));
        if (BKC)
            for (int r = threadIdx.x; r < BN; r += NT) clear(st + IA::BYTES + r * 128 + ((c ^ IB::swz(r)) << 4));
        __syncthreads();
    }

    // acc += the product of a tile whose copies have been started.  `stores`:
    // STORES store instructions of this wave came after start(): they may be
    // under way still.  Loads and stores leave the vmcnt counter in the order of
    // issue, so the waits for the tiles of start() let the stores run on.
    // Every copy has landed at the end.
    __device__ __forceinline__ void finish(unsigned char *smem, f32x16 (&acc)[MI][NI], bool stores) const {
        if (nt <= 0) return;
        const int tid = thread_again(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave % WM, wn = wave / WM;
        // Fragment reads: KC one offset per step, RC one per 32-wide block
        // (the swizzle of a k row repeats every four rows).
        uint32_t fa_off[AKC ? 4 : MI], fb_off[BKC ? 4 : NI];
#pragma unroll
        for (int i = 0; i < (AKC ? 4 : MI); i++)
            fa_off[i] = AKC ? IA::frag(lane, wm * WTM, i, 0) : IA::frag(lane, wm * WTM + i * 32, 0, 0);
#pragma unroll
        for (int i = 0; i < (BKC ? 4 : NI); i++)
            fb_off[i] = IA::BYTES + (BKC ? IB::frag(lane, wn * WTN, i, 0) : IB::frag(lane, wn * WTN + i * 32, 0, 0));
        auto read_a = [&](const unsigned char *st, int s, int mi) __attribute__((always_inline)) -> u32x4 {
            if constexpr (AKC) return lds_read16(st + fa_off[s] + mi * 32 * 128);
            else return Mfma<DT_F16>::read_b(st + fa_off[mi] + (s * 16) * IA::ROWB,
                                             st + fa_off[mi] + (s * 16 + 4) * IA::ROWB);
        };
        auto read_b = [&](const unsigned char *st, int s, int ni) __attribute__((always_inline)) -> u32x4 {
            if constexpr (BKC) return lds_read16(st + fb_off[s] + ni * 32 * 128);
            else return Mfma<DT_F16>::read_b(st + fb_off[ni] + (s * 16) * IB::ROWB,
                                             st + fb_off[ni] + (s * 16 + 4) * IB::ROWB);
        };
        u32x4 fa[4][MI], fb[4][NI];

        // One k step's MFMAs, with the fragment reads of step rs (of buffer
        // rst) and copies [lo, hi) of tile kt spread between them.
        auto step = [&](int s, const unsigned char *rst, int rs, int kt, int lo, int hi,
                        auto checked) __attribute__((always_inline)) {
            constexpr int NM = MI * NI, NR = MI + NI;
#pragma unroll
            for (int m = 0; m < NM; m++) {
                acc[m / NI][m % NI] = Mfma<DT_F16>::mac_sub(fa[s][m / NI], fb[s][m % NI], acc[m / NI][m % NI], 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int u = (m * NR + NM - 1) / NM; u < ((m + 1) * NR + NM - 1) / NM; u++) {
                    if (u < MI) fa[rs][u] = read_a(rst, rs, u);
                    else fb[rs][u - MI] = read_b(rst, rs, u - MI);
                }
                const int nd = hi - lo;
#pragma unroll
                for (int d = (m * nd + NM - 1) / NM; d < ((m + 1) * nd + NM - 1) / NM; d++)
                    issue<decltype(checked)::value>(kt, lo + d);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (stores) wait_vmcnt<STORES <= 63 ? STORES : 63>();  // the tiles may be the older ones: all of them then
        else wait_tiles(min(AHEAD, nt - 1));
        __syncthreads();
        mend_last(smem, 0);
#pragma unroll
        for (int s = 0; s < FD; s++) {
#pragma unroll
            for (int mi = 0; mi < MI; mi++) fa[s][mi] = read_a(smem, s, mi);
#pragma unroll
            for (int ni = 0; ni < NI; ni++) fb[s][ni] = read_b(smem, s, ni);
        }
        // Tiles t0 .. t1 - 1.  `copies`: tile t + STAGES is copied meanwhile,
        // into tile t's buffer; it exists (and only it can be the cut one).
        auto tiles = [&](int t0, int t1, auto copies, auto checked) __attribute__((always_inline)) {
            for (int t = t0; t < t1; t++) {
                const unsigned char *cur = smem + stage(t), *next = cur;
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    const int r = s + FD;
                    if (r == 4) {
                        // tile t+1 has landed, and every wave has read tile t
                        if constexpr (decltype(copies)::value) {
                            if (!(stores && t < AHEAD)) wait_vmcnt<(AHEAD - 1) * ND>();
                            __syncthreads();
                        } else if (t + 1 < nt) {
                            if (!(stores && t < AHEAD)) wait_tiles(nt - 2 - t);
                            __syncthreads();
                            mend_last(smem, t + 1);
                        }
                        next = smem + stage(t + 1);
                    }
                    const int part = decltype(copies)::value && r >= 4 && r < 6 ? r - 4 : -1;
                    step(s, r < 4 ? cur : next, r & 3, t + STAGES, part < 0 ? 0 : part * ND / 2,
                         part < 0 ? 0 : (part + 1) * ND / 2, checked);
                }
            }
        };
        const bool cut = this->cut();
        const int full = max(0, nt - STAGES);  // tiles with a later one to copy
        tiles(0, cut ? max(0, full - 1) : full, std::true_type{}, std::false_type{});
        if (cut) tiles(max(0, full - 1), full, std::true_type{}, std::true_type{});
        tiles(full, nt, std::false_type{}, std::false_type{});
    }
};

template <int MI, int NI>
__device__ static __forceinline__ void clear_acc(f32x16 (&acc)[MI][NI]) {
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int ni = 0; ni < NI; ni++) acc[mi][ni] = f32x16{};
}

// The race screen of TDG_DEBUG_POISON_LDS: LDS full of NaN before the first
// tile is asked for.
template <int BYTES, int NT>
__device__ static __forceinline__ void poison_lds(int flags, unsigned char *smem) {
    if (flags & TDG_DEBUG_POISON_LDS) {
        for (int o = threadIdx.x * 16; o < BYTES; o += NT * 16) lds_write16(smem + o, u32x4{~0u, ~0u, ~0u, ~0u});
        __syncthreads();
    }
}

// Whether C tiles remain for workgroup b, and where: A's and C's rows (TN:
// A's columns) x0 .. x_end - 1, the columns from y0 on, k_lo .. k_hi - 1.
template <int LAY, int BM, int BN, bool CUT = false>
struct GroupedWork {
    GroupedTile t;
    __device__ __forceinline__ bool find(const GroupedArgs &a, int b) {
        t = find_tile<LAY, BM, CUT>(a, b);
        return t.ok;
    }
    __device__ __forceinline__ int x_end(const GroupedArgs &a) const { return LAY == LAY_TN ? a.M : t.hi; }
    __device__ __forceinline__ int y0() const { return t.tn * BN + (CUT && t.half > 0 ? BN / 2 : 0); }
    __device__ __forceinline__ const unsigned char *A(const GroupedArgs &a) const {
        return a.A + (LAY == LAY_TN ? 0 : (int64_t)t.x0 * a.lda);
    }
    __device__ __forceinline__ const unsigned char *B(const GroupedArgs &a) const {
        return a.B + (LAY == LAY_TN ? 0 : (int64_t)t.g * a.stride_b);
    }
    __device__ __forceinline__ uint64_t b_stop(const GroupedArgs &a) const {
        if (LAY == LAY_TN || !a.b_each) return a.b_stop;
        const int rows = LAY == LAY_NN ? a.K : a.N, cols = LAY == LAY_NN ? a.N : a.K;
        return page_stop((uint64_t)(uintptr_t)B(a) + (uint64_t)((int64_t)(rows - 1) * a.ldb), cols);
    }
    __device__ __forceinline__ int k_lo() const { return LAY == LAY_TN ? t.lo : 0; }
    __device__ __forceinline__ int k_hi(const GroupedArgs &a) const { return LAY == LAY_TN ? t.hi : a.K; }
    template <class E, int WM>
    __device__ __forceinline__ bool store(const GroupedArgs &a, const f32x16 (&acc)[E::MI][E::NI]) const {
        const int wave = __builtin_amdgcn_readfirstlane(thread_again() >> 6);
        return store_tile<E::MI, E::NI>(a.C + (LAY == LAY_TN ? (int64_t)t.g * a.stride_c : 0), a.ldc,
                                        t.x0 + (wave % WM) * E::WTM, x_end(a), y0() + (wave / WM) * E::WTN, a.N, acc);
    }
};

template <int LAY, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM *WN * 64, 1) tdg_grouped_any(GroupedArgs a) {
    typedef GroupedAny<LAY, BM, BN, WM, WN> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    GroupedWork<LAY, BM, BN> w;
    if (!w.find(a, blockIdx.x)) return;
    poison_lds<E::SMEM, E::NT>(a.flags, smem);
    f32x16 acc[E::MI][E::NI];
    clear_acc(acc);
    E::run(w.A(a), a.lda, RowsFrom{w.t.x0, a.lda}, w.B(a), a.ldb, w.t.x0, w.x_end(a), w.y0(), a.N, w.k_lo(), w.k_hi(a),
           a.a_stop, w.b_stop(a), smem, acc);
    w.template store<E, WM>(a, acc);
}

template <int LAY, int BM, int BN, int WM, int WN, int STAGES>
__global__ void __launch_bounds__(WM *WN * 64, 1) tdg_grouped_ring(GroupedArgs a) {
    typedef GroupedRing<LAY, BM, BN, WM, WN, STAGES> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    GroupedWork<LAY, BM, BN> w;
    if (!w.find(a, blockIdx.x)) return;
    poison_lds<E::SMEM, E::NT>(a.flags, smem);
    f32x16 acc[E::MI][E::NI];
    clear_acc(acc);
    E::run(w.A(a), a.lda, RowsFrom{w.t.x0, a.lda}, w.B(a), a.ldb, w.t.x0, w.x_end(a), w.y0(), a.N, w.k_lo(), w.k_hi(a),
           a.a_stop, w.b_stop(a), smem, acc);
    w.template store<E, WM>(a, acc);
}

// 256 x 256 tiles, one workgroup per CU: the last round's are cut where that
// fills the CUs (xcd_tile_cut).
template <int LAY>
__global__ void __launch_bounds__(512, 1) tdg_grouped_cut(GroupedArgs a) {
    typedef GroupedRing<LAY, 256, 256, 2, 4, 2> E;
    typedef GroupedRing<LAY, 256, 128, 4, 2, 3> H;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[H::SMEM > E::SMEM ? H::SMEM : E::SMEM];
    GroupedWork<LAY, 256, 256, true> w;
    if (!w.find(a, blockIdx.x)) return;
    if (w.y0() >= a.N) return;
    poison_lds<sizeof(smem), E::NT>(a.flags, smem);
    if (w.t.half < 0) {
        f32x16 acc[E::MI][E::NI];
        clear_acc(acc);
        E::run(w.A(a), a.lda, RowsFrom{w.t.x0, a.lda}, w.B(a), a.ldb, w.t.x0, w.x_end(a), w.y0(), a.N, w.k_lo(),
               w.k_hi(a), a.a_stop, w.b_stop(a), smem, acc);
        w.template store<E, 2>(a, acc);
    } else {
        f32x16 acc[H::MI][H::NI];
        clear_acc(acc);
        H::run(w.A(a), a.lda, RowsFrom{w.t.x0, a.lda}, w.B(a), a.ldb, w.t.x0, w.x_end(a), w.y0(),
               min(a.N, w.y0() + 128), w.k_lo(), w.k_hi(a), a.a_stop, w.b_stop(a), smem, acc);
        w.template store<H, 4>(a, acc);
    }
}

// Asks for a word of every 128-byte line of a rows x cols matrix of 2-byte
// elements, the lines dealt to all threads of the grid; the words land in 256
// bytes of LDS that nobody reads.
__device__ static __forceinline__ void touch(const unsigned char *P, int64_t ld, int lo, int hi, int cols,
                                             unsigned char *lds) {
    const int lines = (cols * 2 + 127) / 128;
    const uint32_t m0 = (uint32_t)(uintptr_t)(TDG_LDS unsigned char *)lds;
    const int64_t all = (int64_t)(hi - lo) * lines, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
        const int row = (int)(i / lines), line = (int)(i - (int64_t)row * lines);
        // a word that holds a byte of the row: it lies in that byte's page
        const uint64_t src = (uint64_t)(uintptr_t)(P + (int64_t)(lo + row) * ld + line * 128) & ~(uint64_t)3;
        asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "{m0}"(m0) : "memory");
    }
}

// Weight gradients of many tiles: the sums are short (a group's rows), and
// writing C takes most of the time.  A workgroup takes tiles b, b + gridDim.x,
// ... (gridDim.x is a multiple of 8, so it stays with its XCD's run).  The
// next tile's first copies go out before this one's stores: they land, and the
// first K tiles are computed, while the stores drain.
// `warm`: A and B are read once before all else, by all CUs at HBM's full
// rate, which leaves them in the memory-side cache.  With HBM busy writing C,
// a read that misses that cache takes long, and every tile waits for some.
// (8192 rows, 32 groups, 2048 x 4000: 330 us without, 271 with, A and B in no
// cache; 269 and 277 where they are in it.  One tile per workgroup: 338.)
template <int BM, int BN, int WM, int WN, int STAGES>
__global__ void __launch_bounds__(WM *WN * 64, 1) tdg_grouped_tn_loop(GroupedArgs a) {
    typedef GroupedRing<LAY_TN, BM, BN, WM, WN, STAGES> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM + 256];
    if (a.warm) {
        const int lo = group_offset(a, 0), hi = group_offset(a, a.groups);
        touch(a.A, a.lda, lo, hi, a.M, smem + E::SMEM);
        touch(a.B, a.ldb, lo, hi, a.N, smem + E::SMEM);
    }
    GroupedWork<LAY_TN, BM, BN> w;
    int b = blockIdx.x;
    if (w.find(a, b)) {
        poison_lds<E::SMEM, E::NT>(a.flags, smem);
        E r;
        auto start = [&]() __attribute__((always_inline)) {
            r.aim(w.A(a), a.lda, RowsFrom{w.t.x0, a.lda}, w.B(a), a.ldb, w.t.x0, w.x_end(a), w.y0(), a.N, w.k_lo(),
                  w.k_hi(a), a.a_stop, w.b_stop(a), smem);
            r.start();
        };
        start();
        bool stores = false;
        for (bool more = true; more;) {
            f32x16 acc[E::MI][E::NI];
            clear_acc(acc);
            r.finish(smem, acc, stores);
            const GroupedWork<LAY_TN, BM, BN> done = w;
            b += gridDim.x;
            more = b < a.tiles_most && w.find(a, b);
            if (more) {
                __syncthreads();  // every wave has read this tile's last fragments
                start();
            }
            stores = done.template store<E, WM>(a, acc);
        }
    }
    wait_vmcnt<0>();  // the words of touch() land before the LDS is given away
}

}  // namespace tdg
