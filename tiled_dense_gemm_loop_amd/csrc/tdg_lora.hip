// tdg_lora.hip -- a shared projection with low-rank adapters of many requests
// beside it: C[t] = A[t] . B + scale[a] * (A[t] . down[a]) . up[a], where
// a = adapter[t], and the second term is left out where a is not in
// [0, adapters).
//
// low[t] = A[t] . down[a] is a thin product that K is cut for so that it fills
// the chip (k_lora_parts_*): a workgroup takes a tile of rows and, one after
// the other, the distinct adapters among them.  Rows are sorted by adapter
// first, so that there are few.
//   * Many rows: k_lora_sort sorts each 4096 rows; k_lora_parts_* makes low;
//     k_lora_split sums its parts and cuts each row into two FP16 rows, high
//     and rest: 21 bits or more of every element.  k_lora_main_* then makes the
//     shared product's tiles over the sorted rows, and on each wave's 32-row
//     blocks low . up on the matrix cores, one pass per distinct adapter of the
//     block, added to the accumulators of that adapter's rows alone: C is
//     written once, and no row sees another's adapter.  A row whose elements
//     differ too much in size for two FP16 rows takes its sums from an FP32
//     product instead.
//   * Few rows or few tiles: the shared product is bound by reading B, or by
//     the latency of its K loop, and has too few tiles to do it at full rate.
//     Its parts over K are made in the same launch as low's, and a second
//     (k_lora_join) sums them and adds low . up in FP32.  Up to 256 rows are
//     sorted in each workgroup, more by k_lora_sort.
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
    float *part;  // parts x M x N: the shared product over slices of K (cut in K)
    float *low;   // low_parts x M x rank; many rows: k_lora_split leaves their sum in the first
    _Float16 *cut;  // M rows of low's high part and rest, rank16 each (many rows)
    int32_t *ex;    // M: their rows' power of two, or kWide
    int rank16;     // the rank, rounded up to 16
    int2 *seat;     // M: row and adapter, sorted by adapter (more than kFewRows)
    int64_t lda, ldb, ldc, ld_down, stride_down, ld_up, stride_up;  // bytes
    uint64_t a_stop, b_stop, down_stop;  // chunks end at this address or below (chunk_stop)
    int down_each;  // each adapter's down has a stop of its own (stops_each)
    int up_apart;   // up's rows' last chunks are loaded element by element
    int M, N, K, adapters, rank;
    int row_tiles, col_tiles;           // of the shared product
    int parts, k_per_part;              // K tiles of each slice
    int low_parts, low_k_per_part;
    int low_cols, low_lanes;            // blocks of the rank; workgroups that share a row tile's adapters
    int low_wgs;                        // workgroups on low, the first ones
    int flags;
};

// Row x of a product over sorted rows.
struct RowsSeated {
    const int2 *seat;
    int64_t ld;
    __device__ __forceinline__ int64_t off(int x) const { return (int64_t)seat[x].x * ld; }
};

// At most this many rows are sorted in each workgroup, and their product is
// always cut in K: the key of sort_few holds them in 8 bits.
// (us as few / as many, 8 adapters of rank 64, K x N = 4096 x 4096: 128 rows
// 28 / 39, 192 rows 34 / 36, 256 rows 38 / 39; 9 of rank 24, 1000 x 5095: 128
// rows 22 / 27, 192 rows 25 / 25, 256 rows 29 / 27.)
constexpr int kFewRows = 256;

// Most slices of K that a product is cut into: they are read again.
constexpr int MAX_PARTS = 8;

// Which adapter a row has, -1 for none.
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int row) {
    const int a = row < p.M ? p.adapter[row] : -1;
    return (unsigned)a < (unsigned)p.adapters ? a : -1;
}

// Each SORT_ROWS rows sorted by adapter (by its remainder, where there are
// more adapters than counters: rows that share a counter may mix), those with
// none last.  Equal keys come out in any order: where a row is worked on does
// not change its values.
constexpr int SORT_ROWS = 4096, SORT_THREADS = 1024;

// Adds 1 to count[key] for every active lane; returns what was there before.
// One request's rows follow each other, so a wave's keys are often all the
// same, and one addition for all of them spares 64 in turn.
__device__ __forceinline__ int take(int *count, int key, int lane) {
    const unsigned long long on = __ballot(1);
    const int first = __builtin_amdgcn_readfirstlane(key);
    if (__ballot(key == first) == on) {
        int at = 0;
        const int leader = __ffsll(on) - 1;
        if (lane == leader) at = atomicAdd(&count[first], __popcll(on));
        return __builtin_amdgcn_readlane(at, leader) + __popcll(on & ((1ull << lane) - 1));
    }
    return atomicAdd(&count[key], 1);
}

__global__ void __launch_bounds__(SORT_THREADS) k_lora_sort(LoraArgs p) {
    __shared__ int count[SORT_THREADS], wave_sum[SORT_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int base = blockIdx.x * SORT_ROWS;
    count[tid] = 0;
    __syncthreads();
    int id[SORT_ROWS / SORT_THREADS], key[SORT_ROWS / SORT_THREADS];
#pragma unroll
    for (int i = 0; i < SORT_ROWS / SORT_THREADS; i++) id[i] = adapter_of(p, base + i * SORT_THREADS + tid);
#pragma unroll
    for (int i = 0; i < SORT_ROWS / SORT_THREADS; i++)
        key[i] = base + i * SORT_THREADS + tid >= p.M ? -1
                 : id[i] < 0                          ? SORT_THREADS - 1
                                                      : id[i] % (SORT_THREADS - 1);
#pragma unroll
    for (int i = 0; i < SORT_ROWS / SORT_THREADS; i++)
        if (key[i] >= 0) take(count, key[i], lane);
    __syncthreads();
    const int mine = count[tid];
    int incl = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(incl, d);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int start = incl - mine;
    for (int w = 0; w < wave; w++) start += wave_sum[w];
    count[tid] = start;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_ROWS / SORT_THREADS; i++)
        if (key[i] >= 0)
            p.seat[base + take(count, key[i], lane)] = make_int2(base + i * SORT_THREADS + tid, id[i]);
}

// Few rows, more than one tile of them: every workgroup sorts them all for
// itself, by counting the smaller keys; list[i] is the i-th row.
__device__ __forceinline__ void sort_few(const LoraArgs &p, int32_t *key, int32_t *list) {
    for (int row = threadIdx.x; row < kFewRows; row += blockDim.x) {
        const int a = adapter_of(p, row);
        key[row] = row >= p.M ? INT32_MAX : (a < 0 ? 1 << 22 : a & ((1 << 22) - 1)) << 8 | row;
    }
    __syncthreads();
    for (int row = threadIdx.x; row < p.M; row += blockDim.x) {
        const int mine = key[row];
        int before = 0;
#pragma unroll 4
        for (int i = 0; i < kFewRows; i += 4) {
            const i32x4 k = *(const i32x4 *)(key + i);
            before += (k[0] < mine) + (k[1] < mine) + (k[2] < mine) + (k[3] < mine);
        }
        list[before] = row;
    }
    __syncthreads();
}

// Tiles of the shared product over a slice of K (where it is cut), and of low.
// A tile of low belongs to 64 rows of the sorted order; its workgroups take
// the distinct adapters among them in turn, each a whole product of which the
// adapter's own rows are kept.
constexpr int PART_TILE = 64;

template <class E>
__device__ __forceinline__ void lora_parts(const LoraArgs &p, unsigned char *smem) {
    constexpr int BM = PART_TILE, BN = PART_TILE, WM = 2;
    __shared__ __attribute__((aligned(16))) int32_t key[kFewRows], list[kFewRows];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    poison_lds<E::SMEM, E::NT>(p.flags, smem);
    f32x16 acc[E::MI][E::NI];
    int b = (int)blockIdx.x - p.low_wgs;
    if (b >= 0) {
        // XCD b % 8 takes a run of tiles, rows first: B's tile is read once
        // into its L2 for all row tiles.
        const int per = ((int)gridDim.x - p.low_wgs) >> 3;
        b = (b & 7) * per + (b >> 3);
        if (b >= p.row_tiles * p.col_tiles * p.parts) return;
        const int tm = b % p.row_tiles, rest = b / p.row_tiles;
        const int tn = rest % p.col_tiles, part = rest / p.col_tiles;
        const int k_lo = part * p.k_per_part * 64, k_hi = min(p.K, k_lo + p.k_per_part * 64);
        clear_acc(acc);
        E::run(p.A + (int64_t)(tm * BM) * p.lda, p.lda, RowsFrom{tm * BM, p.lda}, p.B, p.ldb, tm * BM, p.M, tn * BN,
               p.N, k_lo, k_hi, p.a_stop, p.b_stop, smem, acc);
        store_tile<E::MI, E::NI>((unsigned char *)(p.part + (int64_t)part * p.M * p.N), (int64_t)p.N * 4,
                                 tm * BM + wm * E::WTM, p.M, tn * BN + wn * E::WTN, p.N, acc);
        return;
    }
    b = blockIdx.x;
    const int turn = b % p.low_lanes;
    b /= p.low_lanes;
    const int tc = b % p.low_cols;
    b /= p.low_cols;
    const int part = b % p.low_parts, row0 = b / p.low_parts * BM;
    if (row0 >= p.M) return;
    const int k_lo = part * p.low_k_per_part * 64, k_hi = min(p.K, k_lo + p.low_k_per_part * 64);
    float *low = p.low + (int64_t)part * p.M * p.rank;
    if (!p.seat && p.M > BM) sort_few(p, key, list);
    const int rows = min(BM, p.M - row0);
    int row = -1, id = -1;
    if (lane < rows) {
        if (p.seat) {
            const int2 seat = p.seat[row0 + lane];
            row = seat.x, id = seat.y;
        } else {
            row = p.M > BM ? list[row0 + lane] : lane;
            id = adapter_of(p, row);
        }
    }
    unsigned long long left = __ballot(id >= 0);
    for (int n = 0; left; n++) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffsll(left) - 1));
        const unsigned long long mine = __ballot(id == a);
        left &= ~mine;
        if (n % p.low_lanes != turn) continue;
        // every wave is done with the LDS of the product before; the rows of
        // this tile are in its first words
        if (threadIdx.x < BM) key[threadIdx.x] = max(row, 0);
        __syncthreads();
        clear_acc(acc);
        const unsigned char *down = p.down + (int64_t)a * p.stride_down;
        const uint64_t down_stop =
            p.down_each ? page_stop((uint64_t)(uintptr_t)down + (uint64_t)((int64_t)(p.K - 1) * p.ld_down), p.rank)
                        : p.down_stop;
        E::run(p.A, p.lda, RowsBy{key, p.lda}, down, p.ld_down, 0, rows, tc * BN, p.rank, k_lo, k_hi, p.a_stop, down_stop,
               smem, acc);
#pragma unroll
        for (int mi = 0; mi < E::MI; mi++)
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int r = wm * E::WTM + mi * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
                const int at = __shfl(row, r);
                if (!((mine >> r) & 1)) continue;
#pragma unroll
                for (int ni = 0; ni < E::NI; ni++) {
                    const int c = tc * BN + wn * E::WTN + ni * 32 + (lane & 31);
                    if (c < p.rank) low[(int64_t)at * p.rank + c] = acc[mi][ni][v];
                }
            }
    }
}

__global__ void __launch_bounds__(256, 1) k_lora_parts_ring(LoraArgs p) {
    typedef GroupedRing<LAY_NN, PART_TILE, PART_TILE, 2, 2, 4> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    lora_parts<E>(p, smem);
}
__global__ void __launch_bounds__(256, 1) k_lora_parts_any(LoraArgs p) {
    typedef GroupedAny<LAY_NN, PART_TILE, PART_TILE, 2, 2> E;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[E::SMEM];
    lora_parts<E>(p, smem);
}

// Between the launches for many rows: a wave per row sums low's parts, finds
// the row's largest finite magnitude and writes the row as two FP16 rows,
// x 2^-ex = high + rest 2^-12 with |x 2^-ex| < 2^14.  Their products are summed
// apart, so that rest has a grid of its own: an element down to about 2^-30 of
// the row's largest keeps 21 bits or more.  A row with one that does not (or
// with one that is not finite) is marked kWide, and its sums come from FP32
// products of the row as it is, which is left where the first part was.
constexpr int SPLIT_THREADS = 256;
constexpr float REST_SIZE = 4096.0f;
constexpr int32_t kWide = INT32_MAX;
__global__ void __launch_bounds__(SPLIT_THREADS) k_lora_split(LoraArgs p) {
    const int row = blockIdx.x * (SPLIT_THREADS / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (row >= p.M || adapter_of(p, row) < 0) return;
    constexpr int PER = TDG_LORA_MAX_RANK / 64;
    float x[PER];
#pragma unroll
    for (int q = 0; q < PER; q++) {
        float v[MAX_PARTS];
#pragma unroll
        for (int i = 0; i < MAX_PARTS; i++)
            v[i] = i < p.low_parts && q * 64 + lane < p.rank
                       ? p.low[((int64_t)i * p.M + row) * p.rank + q * 64 + lane]
                       : 0.0f;
        x[q] = v[0];
#pragma unroll
        for (int i = 1; i < MAX_PARTS; i++) x[q] += v[i];
    }
    float most = 0.0f;
#pragma unroll
    for (int q = 0; q < PER; q++) {
        const float m = fabsf(x[q]);
        most = m <= 3.402823466e38f ? fmaxf(most, m) : most;
    }
    for (int d = 32; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
    const int ex = most > 0.0f ? ilogbf(most) - 13 : 0;
    _Float16 *hi = p.cut + (int64_t)row * 2 * p.rank16, *rest = hi + p.rank16;
    bool kept = true;
#pragma unroll
    for (int q = 0; q < PER; q++) {
        const int c = q * 64 + lane;
        if (c >= p.rank16) break;
        const float v = ldexpf(x[q], -ex);
        const _Float16 h = (_Float16)v;
        const float left = (v - (float)h) * REST_SIZE;
        const _Float16 r = (_Float16)left;
        hi[c] = h;
        rest[c] = r;
        // |v - high - rest 2^-12| <= 2^-21 |v|, and v not rounded to 0 (never
        // so for what is not finite)
        kept &= fabsf(left - (float)r) <= fabsf(v) * (REST_SIZE * 0x1p-21f) && (v != 0.0f || x[q] == 0.0f);
        if (c < p.rank && p.low_parts > 1) p.low[(int64_t)row * p.rank + c] = x[q];
    }
    if (__ballot(!kept)) {
        if (lane == 0) p.ex[row] = kWide;
    } else if (lane == 0) {
        p.ex[row] = ex;
    }
}

// What a tile's end needs of each of its rows, kept in LDS from the start.
template <int BM>
struct TileRows {
    __attribute__((aligned(16))) int32_t row[BM], id[BM], ex[BM];
    __device__ __forceinline__ void fill(const LoraArgs &p, int x0) {
        for (int i = threadIdx.x; i < BM; i += blockDim.x) {
            const int2 seat = p.seat[min(x0 + i, p.M - 1)];
            row[i] = seat.x;
            id[i] = x0 + i < p.M ? seat.y : -1;
            ex[i] = seat.y >= 0 ? p.ex[seat.x] : 0;
        }
    }
};

// acc += scale * low . up for a BM-row tile, 64 of the rank at a time.  Both
// parts of low's rows are staged in LDS for the whole tile, as the products'
// operands are; the columns of up[a] that a wave needs are staged in a part of
// LDS of its own, one distinct adapter of its 32-row block after the other.
// The wave's rows begin at r0, its columns at col0.  Chunks of up are read whole,
// as the DMA reads those of B, unless one of them would leave up's last page.
// Rows marked kWide are left to add_exact, and elements whose column of up holds
// an infinity or NaN (the parts' products with it are not low's).  Returns which
// of the wave's 32-row blocks have such (the bits of `odd`).
template <int MI, int NI, int BM, int WAVES>
__device__ __forceinline__ uint32_t add_adapters(const LoraArgs &p, const TileRows<BM> &rows, int r0, int col0,
                                             unsigned char *smem, f32x16 (&acc)[MI][NI]) {
    typedef Image<true, BM> IL;        // the tile's rows by 64 of the rank
    typedef Image<false, NI * 32> IU;  // 64 of the rank by the wave's columns
    const int tid = thread_again(), lane = tid & 63;
    unsigned char *up_at = smem + 2 * IL::BYTES + (tid >> 6) * IU::BYTES;
    uint32_t odd = 0;    // bits mi, mi + 16: the wave's block mi has such rows, such elements
    static_assert(MI <= 16, "a bit per block");
    float probe = 0.0f;  // NaN: what the lane has staged of up is not all finite
    auto look_at = [&](const u32x4 &v) __attribute__((always_inline)) {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t word = v[i];
            probe = __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, word), h2{0, 0}, probe, false);
        }
    };
    for (int c0 = 0; c0 < p.rank; c0 += 64) {
        if (c0) __syncthreads();  // every wave is done with the block before
        // Chunks of up[a]'s rows c0 + q / CPR: U of them per lane at a time.
        constexpr int U = MI * NI <= 4 ? 8 : 4;
        const int need = min(64, p.rank16 - c0) * IU::CPR;  // the rank's rows, in steps of the MFMA's 16
        // (The chunk of a lane is the same in every eighth row: swz repeats.)
        static_assert(64 % IU::CPR == 0 && (64 / IU::CPR) % 4 == 0, "the swizzle must repeat");
        const int up_r = lane / IU::CPR, up_c = ((lane % IU::CPR) ^ IU::swz(up_r)) * 8;
        const bool up_on = col0 + up_c < p.N, up_whole = !p.up_apart || col0 + up_c + 8 <= p.N;
        auto load_up = [&](int a, int q0, u32x4 (&u)[U]) __attribute__((always_inline)) {
            const int r0 = c0 + q0 / IU::CPR + up_r;
            const unsigned char *src = p.up + (int64_t)a * p.stride_up + (int64_t)r0 * p.ld_up + (int64_t)(col0 + up_c) * 2;
            const int64_t step = 64 / IU::CPR * p.ld_up;
#pragma unroll
            for (int i = 0; i < U; i++) {
                const bool ok = r0 + i * (64 / IU::CPR) < p.rank;
                u[i] = load16_global(ok && up_on && up_whole ? src + i * step : (const unsigned char *)tdg_zero16);
            }
        };
        auto store_up = [&](int a, int q0, const u32x4 (&u)[U]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < U; i++) {
                lds_write16(up_at + (q0 + i * 64 + lane) * 16, u[i]);
                look_at(u[i]);
            }
            if (up_on && !up_whole) {  // (zeros so far)
#pragma unroll 1
                for (int q = q0; q < q0 + U * 64; q += 64) {
                    const int r = c0 + q / IU::CPR + up_r;
                    const unsigned char *src = p.up + (int64_t)a * p.stride_up + (int64_t)r * p.ld_up;
                    const u32x4 v = load_chunk(src, r < p.rank, col0 + up_c, p.N);
                    lds_write16(up_at + (q + lane) * 16, v);
                    look_at(v);
                }
            }
        };
        // Small tiles have the registers to load the first adapter's up beside
        // low, and each later one's while the matrix cores work on the one
        // before.
        constexpr bool early = MI * NI <= 4;
        static_assert(!early || IU::CHUNKS <= U * 64, "one batch holds a block of up");
        u32x4 u[U];
        int loaded = -1;
        if (early) {
            const int id = rows.id[r0 + (lane & 31)];
            const uint32_t some = (uint32_t)__ballot(id >= 0);
            if (some) {
                loaded = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffs(some) - 1));
                load_up(loaded, 0, u);
            }
        }
        constexpr int PER = 2 * IL::CHUNKS / (WAVES * 64);
        u32x4 v[PER];
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int q = i * WAVES * 64 + thread_again(), part = q / IL::CHUNKS, r = q / IL::CPR % BM;
            const int c = c0 + ((q % IL::CPR) ^ IL::swz(r)) * 8;
            // rows without an adapter read what is there: their sums are not used
            const _Float16 *src = p.cut + ((int64_t)rows.row[r] * 2 + part) * p.rank16 + c;
            v[i] = load16_global(c < p.rank16 ? (const unsigned char *)src : (const unsigned char *)tdg_zero16);
        }
#pragma unroll
        for (int i = 0; i < PER; i++) lds_write16(smem + (i * WAVES * 64 + tid) * 16, v[i]);
        __syncthreads();
        int staged = -1;
#pragma unroll
        for (int mi = 0; mi < MI; mi++) {
            const int at = r0 + mi * 32;
            // (offsets made anew for each block leave the registers to the sums)
            const int lane = thread_again() & 63;
            const int id = rows.id[at + (lane & 31)];
            uint32_t left = (uint32_t)__ballot(id >= 0);  // both halves of the wave hold the same rows
            if (!left) continue;
            const uint32_t wide = (uint32_t)__ballot(id >= 0 && rows.ex[at + (lane & 31)] == kWide);
            if (wide) odd |= 1u << mi;
            int a = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffs(left) - 1));
            if (early && MI > 1 && staged != a && loaded != a) load_up(a, 0, u);  // (one block: loaded above)
            for (;;) {
                const uint32_t mine = (uint32_t)__ballot(id == a);
                left &= ~mine;
                if (staged != a) {
                    probe = 0.0f;
                    if (early) {
                        store_up(a, 0, u);
                    } else {
                        for (int q0 = 0; q0 < need; q0 += U * 64) {
                            load_up(a, q0, u);
                            store_up(a, q0, u);
                        }
                    }
                    staged = a;
                    __builtin_amdgcn_wave_barrier();
                }
                const int next =
                    left ? __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffs(left) - 1)) : a;
                if (early && next != a) load_up(next, 0, u);
                loaded = -1;
                const float scale = p.scale ? p.scale[a] : 1.0f;
                const uint32_t fit = mine & ~wide;
                f32x16 sum[NI], fine[NI];  // of high, and of rest
#pragma unroll
                for (int ni = 0; ni < NI; ni++) sum[ni] = fine[ni] = f32x16{};
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    if (c0 + s * 16 >= p.rank) break;
                    const u32x4 hi = IL::read(smem, lane, at, s), rest = IL::read(smem + IL::BYTES, lane, at, s);
#pragma unroll
                    for (int ni = 0; ni < NI; ni++) {
                        const u32x4 b = IU::read(up_at, lane, ni * 32, s);
                        sum[ni] = Mfma<DT_F16>::mac_sub(hi, b, sum[ni], 0);
                        fine[ni] = Mfma<DT_F16>::mac_sub(rest, b, fine[ni], 0);
                    }
                }
                __builtin_amdgcn_wave_barrier();
                // an accumulator's rows 4 q .. 4 q + 3 follow each other; `checked`
                // where up's block has an infinity or NaN somewhere
                auto add = [&](auto checked) __attribute__((always_inline)) {
                    bool out = false;
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const int r = q * 8 + (lane >> 5) * 4;
                        const i32x4 e = *(const i32x4 *)&rows.ex[at + r];
#pragma unroll
                        for (int w = 0; w < 4; w++) {
                            const bool on = (fit >> (r + w)) & 1;
#pragma unroll
                            for (int ni = 0; ni < NI; ni++) {
                                const float c = acc[mi][ni][q * 4 + w];
                                const float x = fmaf(fine[ni][q * 4 + w], 1.0f / REST_SIZE, sum[ni][q * 4 + w]);
                                const float more = c + scale * ldexpf(x, e[w]);
                                const bool fits = !decltype(checked)::value || fabsf(x) <= 3.402823466e38f;
                                acc[mi][ni][q * 4 + w] = on && fits ? more : c;
                                out |= on && !fits && col0 + ni * 32 + (lane & 31) < p.N;
                            }
                        }
                    }
                    if (decltype(checked)::value && __ballot(out)) odd |= 0x10000u << mi;
                };
                if (__ballot(!(probe == 0.0f))) add(std::true_type{});
                else add(std::false_type{});
                if (!left) break;
                a = next;
            }
        }
    }
    return odd;
}

// C += scale * low . up where add_adapters has left it out, once the rest of C
// is stored: v_mfma_f32_32x32x2_f32 on low as it is, one distinct adapter of
// each 32-row block after the other, its up straight from memory.  Each lane
// adds to elements that it has stored itself.  Few come here, so it is kept
// small rather than fast, and outside the registers and the instructions of all
// others (4096 rows, K = N = 4096, rank 64: 156 us with no row marked kWide, 169
// with one in 500, 265 with all).  An element's value depends on its row, its
// adapter and its column of up alone, and so does whether it comes from here:
// it is the same whatever block the row lies in.
template <int MI, int NI, int BM>
__device__ __forceinline__ void add_exact(const LoraArgs &p, const TileRows<BM> &rows, int r0, int col0,
                                          uint32_t odd) {
    const int lane = threadIdx.x & 63;
#pragma unroll 1
    for (int mi = 0; mi < MI; mi++) {
        if (!((odd >> mi) & 0x10001)) continue;
        const int at = r0 + mi * 32;
        const int id = rows.id[at + (lane & 31)];
        const float *low = p.low + (int64_t)rows.row[at + (lane & 31)] * p.rank;
        const uint32_t wide = (uint32_t)__ballot(rows.ex[at + (lane & 31)] == kWide);
        uint32_t left = (uint32_t)__ballot(id >= 0);
        if (!((odd >> mi) & 0x10000)) left &= wide;
#pragma unroll 1
        while (left) {
            const int a = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(__ffs(left) - 1));
            const uint32_t mine = (uint32_t)__ballot(id == a);
            left &= ~mine;
            const float scale = p.scale ? p.scale[a] : 1.0f;
#pragma unroll 1
            for (int ni = 0; ni < NI && col0 + ni * 32 < p.N; ni++) {
                const int col = col0 + ni * 32 + (lane & 31);
                const unsigned char *up = p.up + (int64_t)a * p.stride_up + (int64_t)col * 2;
                f32x16 sum = {};
                bool whole = true;  // the lane's half of the column is finite
#pragma unroll 1
                for (int c0 = 0; c0 < p.rank; c0 += 8) {
                    // the lane's four of the step's eight k: the same for both operands
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int c = c0 + (lane >> 5) * 4 + i;
                        const float x = c < p.rank ? low[c] : 0.0f;
                        const float u = c < p.rank && col < p.N ? (float)*(const _Float16 *)(up + (int64_t)c * p.ld_up) : 0.0f;
                        whole &= fabsf(u) <= 65504.0f;
                        sum = __builtin_amdgcn_mfma_f32_32x32x2f32(x, u, sum, 0, 0, 0);
                    }
                }
                const uint64_t halves = __ballot(whole);
                const uint32_t columns = (uint32_t)halves & (uint32_t)(halves >> 32);
                const uint32_t take = (columns >> (lane & 31)) & 1 ? mine & wide : mine;
#pragma unroll
                for (int v = 0; v < 16; v++) {
                    const int r = (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
                    if (!((take >> r) & 1) || col >= p.N) continue;
                    float *dst = (float *)((unsigned char *)p.C + (int64_t)rows.row[at + r] * p.ldc) + col;
                    *dst += scale * sum[v];
                }
            }
        }
    }
}

// The shared product's tiles for many rows, with the adapters added to the
// accumulators.  Tile row x is row seat[x] of A and C.
template <class E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void lora_main(const LoraArgs &p, unsigned char *smem) {
    static_assert(E::SMEM >= 2 * Image<true, BM>::BYTES + WM * WN * Image<false, E::NI * 32>::BYTES,
                  "LDS for low and up");
    __shared__ TileRows<BM> rows;
    const int id = xcd_tile(blockIdx.x, p.row_tiles * p.col_tiles);
    if (id < 0) return;
    int tm, tn;
    order_tile(id, p.row_tiles, p.col_tiles, tm, tn);
    poison_lds<E::SMEM, E::NT>(p.flags, smem);
    rows.fill(p, tm * BM);  // read behind the barriers of run()
    f32x16 acc[E::MI][E::NI];
    clear_acc(acc);
    E::run(p.A, p.lda, RowsSeated{p.seat, p.lda}, p.B, p.ldb, tm * BM, p.M, tn * BN, p.N, 0, p.K, p.a_stop, p.b_stop, smem, acc);
    __syncthreads();  // every wave is done with the tiles in LDS
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r0 = (wave % WM) * E::WTM, x0 = tm * BM + r0, col0 = tn * BN + (wave / WM) * E::WTN;
    const uint32_t odd = add_adapters<E::MI, E::NI, BM, WM * WN>(p, rows, r0, col0, smem, acc);
    // whole 128-byte lines past the caches, as in store_tile
    auto store = [&](auto masked, auto streaming) __attribute__((always_inline)) {
#pragma unroll
        for (int mi = 0; mi < E::MI; mi++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int r = mi * 32 + q * 8 + (lane >> 5) * 4;
                const i32x4 at = *(const i32x4 *)&rows.row[r0 + r];
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    float *dst = (float *)((unsigned char *)p.C + (int64_t)at[w] * p.ldc) + col0 + (lane & 31);
                    const bool row_on = !decltype(masked)::value || x0 + r + w < p.M;
#pragma unroll
                    for (int ni = 0; ni < E::NI; ni++) {
                        if (decltype(masked)::value && !(row_on && col0 + ni * 32 + (lane & 31) < p.N)) continue;
                        if constexpr (decltype(streaming)::value)
                            __builtin_nontemporal_store(acc[mi][ni][q * 4 + w], dst + ni * 32);
                        else
                            dst[ni * 32] = acc[mi][ni][q * 4 + w];
                    }
                }
            }
    };
    const bool inside = x0 + E::WTM <= p.M && col0 + E::WTN <= p.N;
    const bool lines = (((uintptr_t)p.C | (uint64_t)p.ldc) & 127) == 0;
    if (inside && lines) store(std::false_type{}, std::true_type{});
    else if (inside) store(std::false_type{}, std::false_type{});
    else store(std::true_type{}, std::false_type{});
    if (odd) add_exact<E::MI, E::NI>(p, rows, r0, col0, odd);
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

// The last launch where the product is cut in K: C[t][n] = its parts, in
// order, plus scale * sum_c low[t][c] * up[c][n].  A workgroup has one row, a
// thread V <= N of its columns; where V does not divide N the last thread's
// begin earlier, and it and the one before make the same values for those that
// both have.  Bound by latency: up's loads go out eight at a time, and the
// parts' before them.
constexpr int JOIN_THREADS = 256;
static_assert(JOIN_THREADS >= TDG_LORA_MAX_RANK, "a thread per element of low's row");

template <int V>
__global__ void __launch_bounds__(JOIN_THREADS) k_lora_join(LoraArgs p) {
    typedef float fv __attribute__((ext_vector_type(V)));
    typedef _Float16 hv __attribute__((ext_vector_type(V)));
    typedef fv fv_ua __attribute__((aligned(4)));
    typedef hv hv_ua __attribute__((aligned(2)));
    __shared__ float low[TDG_LORA_MAX_RANK];
    const int t = blockIdx.x, tid = threadIdx.x;
    int64_t n = ((int64_t)blockIdx.y * JOIN_THREADS + tid) * V;
    const bool on = n < p.N;
    n = min(n, (int64_t)p.N - V);
    fv v[MAX_PARTS];
#pragma unroll
    for (int i = 0; i < MAX_PARTS; i++)
        v[i] = on && i < p.parts ? *(const fv_ua *)(p.part + ((int64_t)i * p.M + t) * p.N + n) : fv{};
    fv sum = v[0];
#pragma unroll
    for (int i = 1; i < MAX_PARTS; i++) sum += v[i];
    const int id = __builtin_amdgcn_readfirstlane(adapter_of(p, t));
    if (id >= 0 && tid < p.rank) {
        float l[MAX_PARTS];
#pragma unroll
        for (int i = 0; i < MAX_PARTS; i++)
            l[i] = i < p.low_parts ? p.low[((int64_t)i * p.M + t) * p.rank + tid] : 0.0f;
        float s = l[0];
#pragma unroll
        for (int i = 1; i < MAX_PARTS; i++) s += l[i];
        low[tid] = s;
    }
    __syncthreads();
    if (!on) return;
    if (id >= 0) {
        const unsigned char *up = p.up + (int64_t)id * p.stride_up + n * 2;
        fv side = {};
        for (int c0 = 0; c0 < p.rank; c0 += 8) {
            hv u[8];
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (c0 + e < p.rank) u[e] = *(const hv_ua *)(up + (int64_t)(c0 + e) * p.ld_up);
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (c0 + e < p.rank) {
                    const float l = low[c0 + e];
#pragma unroll
                    for (int q = 0; q < V; q++) side[q] = fmaf(l, (float)u[e][q], side[q]);
                }
        }
        const float scale = p.scale ? p.scale[id] : 1.0f;
#pragma unroll
        for (int q = 0; q < V; q++) sum[q] = fmaf(scale, side[q], sum[q]);
    }
    *(fv_ua *)((unsigned char *)p.C + (int64_t)t * p.ldc + n * 4) = sum;
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
    bool cut;             // parts of the shared product over K and a join
    bool sorted;          // the rows are sorted by a launch of their own
    int64_t parts, k_per_part, low_parts, low_k_per_part;
    uint64_t low_at, cut_at, ex_at, seat_at, bytes;  // workspace: parts, low, its FP16 rows, their powers, the seats
};

Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t rank) {
    Plan p = {};
    const int64_t kt = ceil_quot(K, 64);
    const int64_t row_tiles = ceil_quot(M, PART_TILE), tiles = row_tiles * ceil_quot(N, 64);
    p.sorted = M > kFewRows;
    // More rows are cut too where their tiles leave the chip half empty, with a
    // short K a little longer (us cut / not cut: 277 rows, 3023 x 410 18 / 46;
    // 1024 rows, 4096 x 1024 33 / 41; 3946 rows, 3832 x 256 42 / 51; 320 tiles:
    // 300 rows, 4096 x 4096 46 / 39, 1024 x 4096 23 / 25; 384: 333 rows, 1000 x
    // 4095 28 / 31; 560: 2179 rows, 704 x 987 44 / 38).
    p.cut = !p.sorted || tiles <= (kt <= 16 ? 384 : 256);
    auto cut = [&](int64_t tiles, int64_t want, int64_t *parts, int64_t *per) {
        int64_t n = ceil_quot(want, tiles > 0 ? tiles : 1);
        n = n > MAX_PARTS ? MAX_PARTS : n;       // the parts are read again
        n = n * 4 > kt ? (kt + 3) / 4 : n;       // a slice is four K tiles or more
        n = n < 1 ? 1 : n;
        *per = ceil_quot(kt, n);
        *parts = *per > 0 ? ceil_quot(kt, *per) : 1;
    };
    if (p.cut) cut(tiles, 512, &p.parts, &p.k_per_part);
    // low has few tiles, and a workgroup of it starts slowly: slices of K as
    // for 512 workgroups, but longer ones where a few tiles hold many adapters.
    cut(row_tiles * ceil_quot(rank, 64), !p.sorted && row_tiles > 1 ? 4 * row_tiles : 512, &p.low_parts,
        &p.low_k_per_part);
    auto up16 = [](uint64_t n) { return (n + 15) / 16 * 16; };
    p.low_at = p.cut ? up16((uint64_t)p.parts * M * N * 4) : 0;
    p.cut_at = p.low_at + up16((uint64_t)p.low_parts * M * rank * 4);
    p.ex_at = p.cut_at + (p.cut ? 0 : (uint64_t)M * 2 * up16(rank) * 2);
    p.seat_at = p.ex_at + (p.cut ? 0 : up16((uint64_t)M * 4));
    p.bytes = p.seat_at + (p.sorted ? up16((uint64_t)M * 8) : 0);
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
    p.cut = (_Float16 *)((unsigned char *)workspace + plan.cut_at);
    p.ex = (int32_t *)((unsigned char *)workspace + plan.ex_at);
    p.seat = plan.sorted ? (int2 *)((unsigned char *)workspace + plan.seat_at) : nullptr;
    p.rank16 = (int)((rank + 15) / 16 * 16);
    p.lda = lda * 2, p.ldb = ldb * 2, p.ldc = ldc * 4;
    p.ld_down = ld_down * 2, p.stride_down = stride_down * 2, p.ld_up = ld_up * 2, p.stride_up = stride_up * 2;
    p.M = (int)M, p.N = (int)N, p.K = (int)K, p.adapters = (int)adapters, p.rank = (int)rank;
    p.flags = debug_flags_now();
    p.parts = (int)plan.parts, p.k_per_part = (int)plan.k_per_part;
    p.low_parts = (int)plan.low_parts, p.low_k_per_part = (int)plan.low_k_per_part;
    p.a_stop = chunk_stop(A, M, K, lda), p.b_stop = chunk_stop(B, K, N, ldb);
    p.down_stop = chunk_stop(down, K, rank, ld_down, adapters, stride_down);
    p.down_each = stops_each(K, rank, ld_down, adapters, stride_down);
    p.up_apart = stops_each(rank, N, ld_up, adapters, stride_up) ||
                 chunk_stop(up, rank, N, ld_up, adapters, stride_up) != kNoStop;
    // The DMA's lanes reach a tile's rows with 32-bit byte offsets; and rows of
    // B and down whose last chunk must not be copied have to be long enough for
    // no other row's chunk to reach as far.
    const int64_t far = (int64_t)UINT32_MAX / 2 / 256 - 256;
    const bool ring_main = lda <= far && ldb <= far && M * lda <= (int64_t)UINT32_MAX / 2 &&
                           (ldb >= 8 || p.b_stop == kNoStop);
    const bool ring = ring_main && ld_down <= far && (ld_down >= 8 || (!p.down_each && p.down_stop == kNoStop));

    const int64_t low_tiles = ceil_quot(M, PART_TILE);
    p.low_cols = (int)ceil_quot(rank, 64);
    // Workgroups that share a row tile's distinct adapters, of which it has at
    // most as many as rows (one without work costs about 3 us of a slot).
    const int64_t tall = M < PART_TILE ? M : PART_TILE;
    const int64_t lanes = 512 / (low_tiles * plan.low_parts * p.low_cols);
    p.low_lanes = (int)(lanes < 1 ? 1 : lanes > tall ? tall : lanes);
    // Every launch's grid is looked at before the first one goes out.
    const int64_t low_wgs = ceil_quot(low_tiles * plan.low_parts * p.low_cols * p.low_lanes, 8) * 8;
    const void *main_fn = nullptr, *join_fn = nullptr;
    int bm = PART_TILE, bn = PART_TILE, main_threads = 256, join_v = 1;
    if (plan.cut) {
        // (4 columns a thread: 4 x 4096 x 4096 with adapters of rank 64 20.8 us,
        // 128 rows 29.1; 2: 19.9 and 28.1.)
        join_v = N > 1 ? 2 : 1;
        join_fn = N > 1 ? (const void *)&k_lora_join<2> : (const void *)&k_lora_join<1>;
    } else {
        // The largest tile that gives most CUs a workgroup (M x 4096 x 4096 with 8
        // adapters of rank 64, us, 256 / 128 / 128 x 64 wide tiles: M = 4096 148 /
        // 186 / 237, M = 1024 95 / 59 / 72, M = 512 96 / 48 / 44).
        auto tiles = [&](int64_t m, int64_t n) { return ceil_quot(M, m) * ceil_quot(N, n); };
        bm = bn = 128;
        if (!ring_main) {
            main_fn = (const void *)&k_lora_main_any<128, 128, 2, 2>;
        } else if (tiles(256, 256) >= 128) {
            main_fn = (const void *)&k_lora_main_ring<256, 256, 2, 4, 2>;
            bm = bn = 256, main_threads = 512;
        } else if (tiles(128, 128) >= 192) {
            main_fn = (const void *)&k_lora_main_ring<128, 128, 2, 2, 4>;
        } else {
            main_fn = (const void *)&k_lora_main_ring<128, 64, 4, 1, 4>;
            bn = 64;
        }
    }
    const int64_t row_tiles = ceil_quot(M, bm), col_tiles = ceil_quot(N, bn);
    const int64_t join_y = ceil_quot(N, (int64_t)JOIN_THREADS * join_v);
    // HIP counts a launch's threads in 32 bits (row_tiles * col_tiles fits 64).
    auto grid_ok = [](int64_t wgs, int64_t threads) { return wgs <= (int64_t)UINT32_MAX / threads; };
    const int64_t tiles = ceil_quot(row_tiles * col_tiles * (plan.cut ? plan.parts : 1), 8) * 8;
    const int64_t parts_wgs = low_wgs + (plan.cut ? tiles : 0), split_wgs = ceil_quot(M, SPLIT_THREADS / 64);
    if (!grid_ok(parts_wgs, 256) || !grid_ok(tiles, main_threads) || (!plan.cut && !grid_ok(split_wgs, SPLIT_THREADS)) ||
        (plan.cut && (join_y > 65535 || !grid_ok(M * join_y, JOIN_THREADS))))
        return TDG_ERR_UNSUPPORTED;
    p.low_wgs = (int)low_wgs, p.row_tiles = (int)row_tiles, p.col_tiles = (int)col_tiles;
    rc = device_check();
    if (rc != TDG_OK) return rc;
    const void *parts_fn = ring ? (const void *)&k_lora_parts_ring : (const void *)&k_lora_parts_any;
    if (plan.sorted)
        rc = launch((const void *)&k_lora_sort, dim3((unsigned)ceil_quot(M, SORT_ROWS)), SORT_THREADS, &p, stream);
    if (rc == TDG_OK) rc = launch(parts_fn, dim3((unsigned)parts_wgs), 256, &p, stream);
    if (plan.cut)
        return rc != TDG_OK ? rc
                            : launch(join_fn, dim3((unsigned)M, (unsigned)join_y), JOIN_THREADS, &p, stream);
    if (rc == TDG_OK) rc = launch((const void *)&k_lora_split, dim3((unsigned)split_wgs), SPLIT_THREADS, &p, stream);
    return rc != TDG_OK ? rc : launch(main_fn, dim3((unsigned)tiles), main_threads, &p, stream);
}

}  // extern "C"
