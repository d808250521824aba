// bf16_mm.hip -- products grouped by expert in bf16 (gfx950), for every token row m of
// group g with weight W_g (N, K):
//   Y[m, :] = X[m, :] W_g^T;   dX[m, :] = dY[m, :] W_g;   dW_g = sum over m of dY[m, :]^T X[m, :].
//
// One kernel serves the three: a tile of results is 256 columns (of the operand that MFMA
// takes as A: W for Y and dX, X for dW) by at most 256 rows (operand B: X, dY, dY), and the
// sum runs along the memory rows of an operand ("along", X and W of Y, dY of dX) or across
// them ("across": W of dX, both of dW).
//
// Persistent workgroups (one a CU, 4 waves in 2 x 2 of 128 x 128 results) walk over tiles.  The
// sum advances 64 values a slot through a 2-slot LDS ring of 32 KB of each operand, filled by
// buffer-load-to-LDS in whole 128-byte lines.  A slot is two MFMA steps of 32 (16 x 16
// results an instruction; 32 x 32 by 16 has half the LDS reads' addresses but leaves a lower clock:
// 1277 / 1276 / 1451 us for Y / dX / dW below, against 1199 / 1221 / 1438); a step's operands are
// read from LDS during the step before it.  An "along" operand is 256 rows of 128
// bytes in LDS, read 16 bytes a lane; an "across" one 64 rows of 512 bytes, read with the
// transposing LDS read, which gives a lane four consecutive values of its own column.  With one
// wave a SIMD nothing issues while a load or an LDS read waits for its pipe, so both are spread
// between the MFMAs.
//
// The slots of successive tiles form one stream: the loads run ahead of the products across the
// end of a tile, so the next tile's operands arrive while this one's results are stored.
//
// Every workgroup finds its own tiles from the group offsets (a scan in LDS), so no launch comes
// before.  Where there are fewer tiles than CUs, the sum is split: the parts go to the workspace
// in fp32 and a second launch adds them in order.
//
// 16640 x 8192 x 5120 over 16 ragged groups (1.4 TFLOP): Y 1196 us, dX 1230, dW in fp32 1395; one group
// of 16384 rows 993, 1003, 1044 (1.39, 1.37, 1.32 PFLOP/s; nothing but these MFMAs on random values
// runs at 1.94).  Bound by the MFMAs at the clock their power leaves and by the loads' path from L2 (a copy
// without loads 821 / 749 / 846 us); dW also by its stores, whose time adds to the products' (2.7 GB:
// 480 us with next to nothing to sum).
#include "device_common.hpp"
#include "internal.hpp"
#include "mm_tile.hpp"

#include "../../include/mxq.h"

namespace mxq {

namespace {

constexpr int kThreads = kTileThreads;
constexpr int kCols = 256;                               // columns of a tile
constexpr int kSlotK = 64;
constexpr uint32_t kOperandBytes = 32 * 1024;            // of one operand in one slot
constexpr uint32_t kSlotBytes = 2 * kOperandBytes;
constexpr uint32_t kLdsBytes = 2 * kSlotBytes;
constexpr int kMaxEntries = 64;                          // tiles of one workgroup: one a lane
// Column tiles of a block of the tile order.  16 uniform groups of 1040 rows, Y / dX / dW: 4 1357 /
// 1324 / 1413 us, 8 1367 / 1371 / 1369.
template <int P>
constexpr int kColBlock = P == MXQ_PRODUCT_DW ? 8 : 4;
constexpr int kXcds = 8;
constexpr int kMaxGroups = 4095;
constexpr int kMaxSplit = 16;
constexpr int kListBytes = (3 * (kMaxGroups + 1) + kThreads) * 4 + kMaxEntries * 64;
static_assert(kListBytes <= (int)kLdsBytes, "the list's arrays fit the ring");
// What a tile of 129 to 256 rows, of 65 to 128 and of up to 64 costs next to the others in a full round,
// where the columns' operand is most of it: a round of 256-, 128- and 64-row tiles after others at
// K = 5120 was measured as 1, 0.72 and 0.6 in the sum of a call (0.82, 0.8 and 0.73 alone); lists dealt by
// 16 / 10 / 9 took Y / dX of 16 groups of 1040 rows from 1357 / 1324 us to 1309 / 1293.
constexpr int kCostWhole = 16, kCostHalf = 10, kCostQuarter = 9;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i* LdsV4i;
typedef __attribute__((address_space(3))) v4s* LdsV4s;

struct MmArgs {
    const uint16_t *a, *b;                               // W or X; X or dY
    const int32_t* offs;
    void* out;
    int M, N, K, G;
    int rows;                                            // rows of a tile, at most: 128 or 256
    int split;                                           // parts of the sum
};

// The three products: which operands run across memory rows; what a tile's columns, its rows
// and the sum's length are.
template <int P>
struct Shape {
    static constexpr bool kDw = P == MXQ_PRODUCT_DW;
    static constexpr bool kAcrossA = P != MXQ_PRODUCT_Y, kAcrossB = kDw;
    static __host__ __device__ __forceinline__ int cols(int N, int K) { return P == MXQ_PRODUCT_Y ? N : K; }
    static __device__ __forceinline__ int depth(int N, int K) { return P == MXQ_PRODUCT_Y ? K : N; }      // (not dW's)
    static __device__ __forceinline__ uint32_t lda(int N, int K) { return 2u * (uint32_t)K; }
    static __device__ __forceinline__ uint32_t ldb(int N, int K) { return 2u * (uint32_t)(P == MXQ_PRODUCT_Y ? K : N); }
};

struct Tile {
    int g, r0, r1, c;                                    // group, rows [r0, r1) (dW: of the group's N), column tile
    int k0, k1, part;                                    // the sum's range (dW: token rows), its part
};

// A workgroup's list: tile e in lane e of every wave.
struct TileList {
    Tile mine;
    __device__ __forceinline__ Tile at(int e) const
    {
        return Tile{__builtin_amdgcn_readlane(mine.g, e),  __builtin_amdgcn_readlane(mine.r0, e),
                    __builtin_amdgcn_readlane(mine.r1, e), __builtin_amdgcn_readlane(mine.c, e),
                    __builtin_amdgcn_readlane(mine.k0, e), __builtin_amdgcn_readlane(mine.k1, e),
                    __builtin_amdgcn_readlane(mine.part, e)};
    }
};

__device__ __forceinline__ int slots_of(const Tile& t)
{
    const int n = (t.k1 - t.k0 + kSlotK - 1) / kSlotK;
    return n > 0 ? n : 1;                                // (an empty sum: one slot that loads nothing)
}

// -------------------------------------------------------------- tile list ---
// Part p of S of a sum of n values from `base`: whole slots but for the last.
__device__ __forceinline__ void part_of(Tile& t, int base, int n, int p, int S)
{
    const int slots = (n + kSlotK - 1) / kSlotK;
    const int a = (int)((int64_t)slots * p / S) * kSlotK, b = (int)((int64_t)slots * (p + 1) / S) * kSlotK;
    t.part = p;
    t.k0 = base + (a < n ? a : n);
    t.k1 = base + (b < n ? b : n);
}

// Place `i` of a grid of `rows` x `cols` tiles in blocks of B columns, a block's rows one after
// the other.
template <int B>
__device__ __forceinline__ void place_in(int i, int rows, int cols, int* r, int* c)
{
    const int cb = i / (rows * B), rem = i - cb * rows * B;
    const int width = cols - cb * B < B ? cols - cb * B : B;
    *r = rem / width;
    *c = cb * B + rem % width;
}

// What a tile of so many rows costs, in sixteenths of a whole one: its loads and barriers stay.
__device__ __forceinline__ int tile_cost(int rows)
{
    return rows > 128 ? kCostWhole : rows > 64 ? kCostHalf : rows > 0 ? kCostQuarter : 0;
}

// The items of one round for an XCD's CUs, one a lane: cost[lane] of item `lane` (0: none), load:
// CU `lane`'s work up to now, which grows.  Returns CU `lane`'s item: the costliest go to the CUs
// with the least work.
__device__ __forceinline__ int items_by_load(int cost, int& load, int cus)
{
    const int lane = lane_id();
    const uint64_t whole = __ballot(cost == kCostWhole), half = __ballot(cost == kCostHalf),
                   quarter = __ballot(cost == kCostQuarter), none = __ballot(cost == 0);
    const auto below = [&](uint64_t m) { return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u)); };
    const int n8 = __builtin_popcountll(whole), n4 = n8 + __builtin_popcountll(half), n2 = n4 + __builtin_popcountll(quarter);
    const int place = cost == kCostWhole ? below(whole) : cost == kCostHalf ? n8 + below(half) : cost == kCostQuarter ? n4 + below(quarter) : n2 + below(none);
    const int by_place = __builtin_amdgcn_ds_permute(4 * place, lane);      // the item at each place
    int rank = 0;
    for (int m = 0; m < cus; ++m) {
        const int other = readlane(load, m);
        rank += other < load || (other == load && m < lane);
    }
    const int item = __builtin_amdgcn_ds_bpermute(4 * (lane < cus ? rank : lane), by_place);
    load += __builtin_amdgcn_ds_bpermute(4 * item, cost);
    return item;
}

// Fills `list` with this workgroup's tiles and returns their number; *rows_end is the last
// group's clamped end.  sh: kListBytes of LDS.
template <int P>
__device__ int make_list(const MmArgs& a, uint8_t* sh, TileList& list, int* rows_end)
{
    int* end_sh = (int*)sh;                              // the groups' clamped ends
    int* first_sh = end_sh + kMaxGroups + 1;             // each group's first row tile
    int* work_sh = first_sh + kMaxGroups + 1;            // and the cost of those before it
    int* scan_sh = work_sh + kMaxGroups + 1;
    uint8_t* cost_sh = (uint8_t*)(scan_sh + kThreads);   // of the items of each round
    const int t = (int)threadIdx.x, R = a.rows, S = a.split;
    const int per = (a.G + kThreads - 1) / kThreads;
    const int ga = t * per < a.G ? t * per : a.G, gb = ga + per < a.G ? ga + per : a.G;
    int top = 0;
    for (int g = ga; g < gb; ++g) {
        const int e = a.offs[g];
        top = e > top ? e : top;
        end_sh[g] = top < a.M ? top : a.M;
    }
    const int upto = block_scan<true>(top, scan_sh);
    scan_sh[t] = upto;
    __syncthreads();
    const int before = t ? scan_sh[t - 1] : 0;
    const int base = before < a.M ? before : a.M;
    for (int g = ga; g < gb; ++g) end_sh[g] = end_sh[g] > base ? end_sh[g] : base;
    __syncthreads();

    const int NC = (Shape<P>::cols(a.N, a.K) + kCols - 1) / kCols;
    const int x = (int)blockIdx.x % kXcds, cu = (int)blockIdx.x / kXcds, cus = (int)gridDim.x / kXcds;
    const int j = lane_id();
    list.mine = Tile{0, 0, 0, 0, 0, 0, 0};
    *rows_end = end_sh[a.G - 1];

    if constexpr (Shape<P>::kDw) {
        // Every group has the same tiles and its own length of sum: a round of one tile a
        // CU is cut over the XCDs, so that each has its share of every group.
        const int NR = (a.N + R - 1) / R, per_group = NR * NC * S;
        const int V = a.G * per_group, grid = (int)gridDim.x;
        const int full = V / grid, over = V - full * grid;
        const int lo = (int)((int64_t)over * x / kXcds), last = (int)((int64_t)over * (x + 1) / kXcds) - lo;
        const int count = full + (cu < last);
        if (j < count) {
            const int L = j < full ? j * grid + (x + j) % kXcds * cus + cu : full * grid + lo + cu;
            Tile tl;
            tl.g = L / per_group;
            const int rem = L - tl.g * per_group;
            int r;
            place_in<kColBlock<P>>(rem / S, NR, NC, &r, &tl.c);
            tl.r0 = r * R;
            tl.r1 = tl.r0 + R < a.N ? tl.r0 + R : a.N;
            const int start = tl.g ? end_sh[tl.g - 1] : 0;
            part_of(tl, start, end_sh[tl.g] - start, rem % S, S);
            list.mine = tl;
        }
        return count < kMaxEntries ? count : kMaxEntries;
    }

    int tiles = 0, work = 0;
    for (int g = ga, start = base; g < gb; ++g) {
        const int m = end_sh[g] - start;
        tiles += (m + R - 1) / R;
        work += m / R * tile_cost(R) + tile_cost(m % R);
        start = end_sh[g];
    }
    int first = block_scan<false>(tiles, scan_sh) - tiles;
    int before_work = block_scan<false>(work, scan_sh) - work;
    for (int g = ga, start = base; g < gb; ++g) {
        const int m = end_sh[g] - start;
        first_sh[g] = first;
        work_sh[g] = before_work;
        first += (m + R - 1) / R;
        before_work += m / R * tile_cost(R) + tile_cost(m % R);
        start = end_sh[g];
    }
    if (t == kThreads - 1) {
        first_sh[a.G] = first;
        work_sh[a.G] = before_work;
    }
    __syncthreads();

    // Each XCD walks one stretch of the tiles, about an eighth of the work, its CUs side by
    // side; the tiles left after the last full round are cut in row parts of 64 or more while
    // that gives no more than one for each CU.
    const int V = first_sh[a.G] * NC * S, W = work_sh[a.G];
    const auto last_at = [&](const int* sh_, int v, int mul) {               // the last group that starts at or before v
        int p = 0, r = a.G - 1;
        while (p < r) {
            const int mid = (p + r + 1) >> 1;
            if (sh_[mid] * mul <= v) p = mid;
            else r = mid - 1;
        }
        return p;
    };
    const auto cut = [&](int i) {
        if (i == kXcds) return V;
        const int w = (int)((int64_t)W * i / kXcds), p = last_at(work_sh, w, 1);
        const int64_t n = (int64_t)(first_sh[p + 1] - first_sh[p]) * NC * S;
        return (int)(first_sh[p] * NC * S + (n > 0 ? (w - work_sh[p]) * n / (work_sh[p + 1] - work_sh[p]) : 0));
    };
    const int lo = cut(x), n = cut(x + 1) - lo;
    const int full = n / cus, over = n - full * cus;
    const int parts = 4 * over <= cus && R == 256 ? 4 : 2 * over <= cus ? 2 : 1;
    // Item i of round e: its tile, whole or (in the last round) a part of it.
    const auto tile_of = [&](int e, int i) {
        const int L = lo + e * cus + (e < full ? i : i / parts), V2 = L / S;
        const int p = last_at(first_sh, V2, NC);
        int rt;
        Tile tl;
        place_in<kColBlock<P>>(V2 - first_sh[p] * NC, first_sh[p + 1] - first_sh[p], NC, &rt, &tl.c);
        const int height = e < full ? R : R / parts, part = e < full ? 0 : i % parts;
        tl.g = p;
        tl.r0 = (p ? end_sh[p - 1] : 0) + rt * R + part * height;
        tl.r1 = tl.r0 + height < end_sh[p] ? tl.r0 + height : end_sh[p];
        if (tl.r1 < tl.r0) tl.r1 = tl.r0;                // a part past the group's rows
        part_of(tl, 0, Shape<P>::depth(a.N, a.K), L % S, S);
        return tl;
    };
    const int rounds = full + (over > 0);
    const auto items = [&](int e) { return e < full ? cus : over * parts; };
    int mine = cu;                                       // this CU's item of round `lane`
    if (rounds > 1 && cus <= 64) {
        for (int e = t >> 6; e < rounds && e < kMaxEntries; e += kThreads / 64) {
            const Tile tl = j < items(e) ? tile_of(e, j) : Tile{0, 0, 0, 0, 0, 0, 0};
            cost_sh[e * 64 + j] = (uint8_t)tile_cost(tl.r1 - tl.r0);
        }
        __syncthreads();
        int load = 0;
        for (int e = 0; e < rounds && e < kMaxEntries; ++e) {
            const int cost = cost_sh[e * 64 + j], one = readlane(cost, 0);
            int item = j;
            if (__ballot(j < cus && cost != one)) item = items_by_load(cost, load, cus);
            else load += cost;
            item = readlane(item, cu);
            if (j == e) mine = item;
        }
    }
    const int count = full + (rounds > full && readlane(mine, full < 63 ? full : 63) < items(full));
    if (j < count) list.mine = tile_of(j, mine);
    return count < kMaxEntries ? count : kMaxEntries;
}

// ------------------------------------------------------------------ loads ---
// The stream of slots to load.  A wave loads a quarter of each operand's slot, 8 loads of 1 KB
// of each.
//
// "Along": LDS rows of 128 bytes hold their eight 16-byte chunks at c ^ ((row >> 1) & 7): the
// 16 lanes that a 128-bit LDS read serves at a time then meet 16 different bank groups.
// "Across": LDS rows of 512 bytes hold their sixteen 32-byte parts at p ^ across_swizzle(row):
// the four rows of a transposing read, and those eight rows on, then meet different banks.  The
// swizzles are applied to the source offsets (the LDS side is linear in the lane).
__device__ __forceinline__ uint32_t across_swizzle(uint32_t row) { return 2u * (row & 3u) + (row >> 3 & 1u); }

template <bool ACROSS>
struct Operand {
    v4i r;                                               // resource that starts at the next slot
    int rows;                                            // ACROSS: the sum's values from the next slot on
    uint32_t off[8];                                     // lane offsets of the wave's loads
    uint32_t tail;                                       // bit 31 of bytes 0 and 2: this lane's chunk of even, odd loads is past a row's end

    __device__ __forceinline__ void set_lanes(uint32_t ld, int depth, int wave, int lane)
    {
        if constexpr (ACROSS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t row = (uint32_t)(16 * wave + 2 * i + (lane >> 5));
                const uint32_t part = (((uint32_t)lane >> 1) & 15u) ^ across_swizzle(row);
                off[i] = row * ld + 32u * part + 16u * ((uint32_t)lane & 1u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t row = (uint32_t)(64 * wave + 8 * i + (lane >> 3));
                const uint32_t chunk = ((uint32_t)lane & 7u) ^ ((row >> 1) & 7u);
                off[i] = row * ld + 16u * chunk;
            }
            const uint32_t even = ((uint32_t)lane & 7u) ^ ((uint32_t)lane >> 4), chunks = (uint32_t)(depth % kSlotK) / 8u;
            tail = ((even >= chunks) << 0) | (((even ^ 4u) >= chunks) << 1);
        }
    }
    // The last slot of a sum that ends inside it: chunks past the end load zeros (their lanes'
    // offsets leave the resource).  Called again to undo it.
    __device__ __forceinline__ void toggle_tail()
    {
        if constexpr (!ACROSS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) off[i] ^= (tail << ((i & 1) ? 30 : 31)) & 0x80000000u;
        }
    }
    // A tile's first slot: `base` its first value, n its rows of ld bytes ("along") or the sum's
    // length ("across"); `skip` bytes of the first row come before it.
    __device__ __forceinline__ void set(const uint16_t* base, int n, uint32_t ld, uint32_t skip)
    {
        rows = n;
        const int used = ACROSS && n > kSlotK ? kSlotK : n;
        r = resource(base, used > 0 ? (uint32_t)used * ld - skip : 0u);
    }
    // (Signed, so that the bound is a scalar maximum.)
    __device__ __forceinline__ void step(uint32_t ld, uint32_t skip)
    {
        const uint32_t bytes = ACROSS ? kSlotK * ld : 2u * kSlotK;
        const uint64_t base = (((uint64_t)(uint32_t)r.y << 32) | (uint32_t)r.x) + bytes;
        int left;
        if constexpr (ACROSS) {
            rows -= kSlotK;
            left = rows > kSlotK ? (int)(kSlotK * ld - skip) : rows > 0 ? (int)((uint32_t)rows * ld - skip) : 0;
        } else {
            left = r.z - (int)bytes > 0 ? r.z - (int)bytes : 0;
        }
        r = v4i{(int)(uint32_t)base, (int)(uint32_t)(base >> 32), left, 0x00020000};
    }
};

template <int P>
struct Loader {
    using S = Shape<P>;
    Operand<S::kAcrossA> a;
    Operand<S::kAcrossB> b;
    int entry, left;                                     // the tile's place in the list; its slots from the next one on
    uint32_t skip_a, skip_b;                             // bytes of a memory row before the tile ("across")
    int ends, masked;                                    // the tile's sum ends inside its last slot; the tail is masked now
    uint32_t lds_data;                                   // LDS address of the wave's part of ring slot 0

    __device__ __forceinline__ void set_lanes(const MmArgs& m, const uint8_t* lds, int wave, int lane)
    {
        a.set_lanes(S::lda(m.N, m.K), S::depth(m.N, m.K), wave, lane);
        b.set_lanes(S::ldb(m.N, m.K), S::depth(m.N, m.K), wave, lane);
        lds_data = (uint32_t)uniform((int)((uint32_t)(uintptr_t)(LdsPtr)lds + 8192u * (uint32_t)wave));
        masked = ends = 0;
    }

    // The scalar state that a tile starts from, in scalar registers (after the divergent stores
    // of the last one the compiler would keep it in vector registers).
    __device__ __forceinline__ void make_uniform()
    {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a.r[k] = uniform(a.r[k]);
            b.r[k] = uniform(b.r[k]);
        }
        a.rows = uniform(a.rows);
        b.rows = uniform(b.rows);
        entry = uniform(entry);
        left = uniform(left);
        skip_a = (uint32_t)uniform((int)skip_a);
        skip_b = (uint32_t)uniform((int)skip_b);
        ends = uniform(ends);
        masked = uniform(masked);
    }

    // The first slot of tile `entry` of the list; past the list's end, one that loads nothing.
    __device__ __forceinline__ void set_tile(const MmArgs& m, const TileList& list, int count)
    {
        const bool some = entry < count;
        const Tile t = list.at(some ? entry : 0);
        const int c0 = t.c * kCols, cols = S::cols(m.N, m.K), n = some ? t.k1 - t.k0 : 0;
        const int width = !some ? 0 : cols - c0 < kCols ? cols - c0 : kCols;
        left = some ? slots_of(t) : 1;
        if constexpr (S::kDw) {
            skip_a = 2u * (uint32_t)c0;
            skip_b = 2u * (uint32_t)t.r0;
            a.set(m.a + (int64_t)t.k0 * m.K + c0, n, S::lda(m.N, m.K), skip_a);
            b.set(m.b + (int64_t)t.k0 * m.N + t.r0, n, S::ldb(m.N, m.K), skip_b);
        } else {
            const int64_t depth = S::depth(m.N, m.K);
            if constexpr (S::kAcrossA) {
                skip_a = 2u * (uint32_t)c0;
                a.set(m.a + ((int64_t)t.g * m.N + t.k0) * m.K + c0, n, S::lda(m.N, m.K), skip_a);
            } else {
                skip_a = 2u * (uint32_t)t.k0;
                a.set(m.a + ((int64_t)t.g * m.N + c0) * depth + t.k0, width, S::lda(m.N, m.K), skip_a);
            }
            skip_b = 2u * (uint32_t)t.k0;
            b.set(m.b + (int64_t)t.r0 * depth + t.k0, some ? t.r1 - t.r0 : 0, S::ldb(m.N, m.K), skip_b);
            ends = t.k1 % kSlotK != 0;
        }
        mask();
    }
    __device__ __forceinline__ void mask()
    {
        if constexpr (!S::kDw) {
            const int want = ends && left == 1;
            if (want != masked) {
                a.toggle_tail();
                b.toggle_tail();
                masked = want;
            }
        }
    }
    // On to the next slot of the stream.
    __device__ __forceinline__ void advance(const MmArgs& m, const TileList& list, int count)
    {
        if (left == 1) {
            ++entry;
            set_tile(m, list, count);
        } else {
            --left;
            a.step(S::lda(m.N, m.K), skip_a);
            b.step(S::ldb(m.N, m.K), skip_b);
            mask();
        }
    }
    // Load I of the slot into ring slot s: A, then B.
    template <int I>
    __device__ __forceinline__ void issue(uint32_t s)
    {
        const uint32_t to = lds_data + s * kSlotBytes;
        if constexpr (I < 8) load_to_lds(a.r, to + 1024u * I, a.off[I]);
        else load_to_lds(b.r, to + kOperandBytes + 1024u * (I - 8), b.off[I - 8]);
    }
    template <int I, int END>
    __device__ __forceinline__ void issue_some(uint32_t s)
    {
        if constexpr (I < END) {
            issue<I>(s);
            issue_some<I + 1, END>(s);
        }
    }
};

// --------------------------------------------------------------- products ---
// v_mfma_f32_16x16x32_bf16 and not 32x32x16: of the same rate, it moves half the accumulators a
// flop, and the clock follows the power (loops of nothing else on random values: 1.94 against 1.71
// PFLOP/s).  In a 32-value step lane (r, q) = (lane % 16, lane / 16) holds the values 8q .. 8q + 7
// of row (or column) r of each 16-wide part.  A wave has 8 parts of A and TB of B.
template <int T>
struct Fragments {
    v4i v[T];
};

// A lane's LDS addresses of an operand in the ring slot that is read: "along", by the step, for
// part 0 (part i is 16 rows on); "across", by the part, for step 0 and the first of its two
// reads (step n is 32 rows on, the second read four).
template <bool ACROSS>
struct Places {
    static constexpr int kN = ACROSS ? 8 : 2;
    uint32_t at[kN];
    // base: the operand's place in the slot; part: the wave's first 16-wide part.
    __device__ __forceinline__ void set(uint32_t base, uint32_t part)
    {
        const uint32_t lane = (uint32_t)lane_id(), q = lane >> 4;
#pragma unroll
        for (uint32_t n = 0; n < kN; ++n) {
            if constexpr (ACROSS) {                      // row 8q + s, four columns of a 32-byte part
                const uint32_t s = (lane >> 2) & 3u, row = 8u * q + s;
                at[n] = base + row * 512u + (((part + n) ^ across_swizzle(row)) << 5) + 8u * (lane & 3u);
            } else {                                     // row r, chunk 4n + q
                at[n] = base + (16u * part + (lane & 15u)) * 128u + (((4u * n + q) ^ ((lane >> 1) & 7u)) << 4);
            }
        }
    }
    // (The ring is the kernel's only LDS and so starts at 0: a slot's address is a bit.)
    __device__ __forceinline__ void other_slot()
    {
#pragma unroll
        for (int n = 0; n < kN; ++n) at[n] ^= kSlotBytes;
    }
};

// Piece Q of a step's operand (0 .. T - 1, twice that "across").
template <bool ACROSS, int ST, int Q, int T>
__device__ __forceinline__ void read_piece(Fragments<T>& f, const Places<ACROSS>& l)
{
    if constexpr (ACROSS) {
        constexpr int i = Q / 2, half = Q % 2;
        const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4s)(uintptr_t)(l.at[i] + 16384u * ST + 2048u * half));
        const uint2 w = __builtin_bit_cast(uint2, v);
        f.v[i][2 * half] = (int)w.x;
        f.v[i][2 * half + 1] = (int)w.y;
    } else {
        f.v[Q] = *(LdsV4i)(uintptr_t)(l.at[ST] + 2048u * Q);
    }
}
template <int P>
struct Lane {
    uint32_t row, q;
    uint32_t wn, wm;                                     // the wave's place in the 2 x 2
    Places<Shape<P>::kAcrossA> a;
    Places<Shape<P>::kAcrossB> b;
};
template <int TB>
struct Operands {
    Fragments<8> a;
    Fragments<TB> b;
};
template <int P, int TB>
constexpr int kPieces = 8 * (Shape<P>::kAcrossA ? 2 : 1) + TB * (Shape<P>::kAcrossB ? 2 : 1);
// Pieces Q .. END - 1 of step ST's operands.
template <int P, int TB, int ST, int Q, int END>
__device__ __forceinline__ void read_step(Operands<TB>& f, const Lane<P>& l)
{
    if constexpr (Q < END) {
        constexpr int na = 8 * (Shape<P>::kAcrossA ? 2 : 1);
        if constexpr (Q < na) read_piece<Shape<P>::kAcrossA, ST, Q>(f.a, l.a);
        else read_piece<Shape<P>::kAcrossB, ST, Q - na>(f.b, l.b);
        read_step<P, TB, ST, Q + 1, END>(f, l);
    }
}

// MFMAs I .. END - 1 of a step, each followed by its share of the other work of that stretch:
// work(k, n) does part k of n.  ZERO: the sums start here.
template <int TB, bool ZERO, int I, int END, int K = 0, class Work>
__device__ __forceinline__ void mfmas(v4f (&acc)[8][TB], const Operands<TB>& f, const Work& work)
{
    if constexpr (I < END) {
        constexpr int i = I / TB, j = I % TB;
        v4f c = acc[i][j];
        if constexpr (ZERO) c = v4f{};
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, f.a.v[i]), __builtin_bit_cast(v8bf, f.b.v[j]),
                                                            c, 0, 0, 0);
        work(Int<K>{}, Int<K + END - I>{});
        __builtin_amdgcn_sched_barrier(0);
        mfmas<TB, ZERO, I + 1, END, K + 1>(acc, f, work);
    }
}
// The bounds of part k of n of a .. b.
#define MXQ_PART(a, b) (a) + K.value * ((b) - (a)) / N.value, (a) + (K.value + 1) * ((b) - (a)) / N.value

// The order of a slot's two steps of 8 TB MFMAs, in eighths; what is read and loaded under each
// stretch (16 loads a slot), and the barriers between them ("read": all waves' LDS reads are
// done; "there": all waves' loads have landed):
//   step 0   0 .. 5   LDS: step 1
//                     (the slot is read)
//            5 .. 8   slot + 2: loads 0 .. 4
//   step 1   0 .. 2   slot + 2: 5 .. 7
//                     (slot + 1 is there)
//            2 .. 8   slot + 2: 8 .. 15; LDS: step 0 of slot + 1
// A load has twenty-one (the first) to ten eighths (the last) of a step to arrive, a step being 1024 cycles of
// MFMAs.
constexpr int kLoads0 = 5, kLoads1 = 8;                  // loads issued by the end of each stretch

template <int P, int TB, bool FIRST>
__device__ __forceinline__ void step0(v4f (&acc)[8][TB], Operands<TB> (&f)[2], Loader<P>& ld, Lane<P>& l, uint32_t s)
{
    constexpr int n = 8 * TB, Q = kPieces<P, TB>;
    __builtin_amdgcn_sched_barrier(0);
    mfmas<TB, FIRST, 0, 5 * TB>(acc, f[0], [&](auto K, auto N) { read_step<P, TB, 1, MXQ_PART(0, Q)>(f[1], l); });
    l.a.other_slot();
    l.b.other_slot();
    slot_barrier<63>();
    mfmas<TB, FIRST, 5 * TB, n>(acc, f[0], [&](auto K, auto N) { ld.template issue_some<MXQ_PART(0, kLoads0)>(s); });
}
// On exit f[0] holds the next slot's first step, unless this is the tile's LAST.
template <int P, int TB, bool LAST>
__device__ __forceinline__ void step1(v4f (&acc)[8][TB], Operands<TB> (&f)[2], Loader<P>& ld, Lane<P>& l, uint32_t s)
{
    constexpr int n = 8 * TB, Q = kPieces<P, TB>;
    mfmas<TB, false, 0, 2 * TB>(acc, f[1], [&](auto K, auto N) { ld.template issue_some<MXQ_PART(kLoads0, kLoads1)>(s); });
    slot_barrier<kLoads1>();                             // (newer: the slot after it)
    mfmas<TB, false, 2 * TB, n>(acc, f[1], [&](auto K, auto N) {
        if constexpr (!LAST) read_step<P, TB, 0, MXQ_PART(0, Q)>(f[0], l);
        ld.template issue_some<MXQ_PART(kLoads1, 16)>(s);
    });
}
#undef MXQ_PART

// The sums are needed here: without this the compiler moves MFMAs past the loads that are meant
// to run under them, into the next basic block.
template <int TB>
__device__ __forceinline__ void pin(v4f (&acc)[8][TB])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) asm volatile("" : "+a"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
}

// Stores: lane (r, q) holds, of row r of each 16 x 16 part, columns 4q .. 4q + 3.  fp32: 16 bytes
// a lane, 64 of a row.  bf16: two parts side by side change lanes, so that those of even q have
// eight columns of the first and those of odd q of the second: 16 bytes a lane, 64 of a row.
// Through a buffer resource that ends with the tile's last row; a lane past the last column
// leaves it too, so that no branch stands between the stores.
template <int P, int TB, bool F32OUT, bool ADD>
__device__ __forceinline__ void store_tile(v4f (&acc)[8][TB], const MmArgs& a, const Tile& t, const Lane<P>& l)
{
    constexpr int kSize = F32OUT ? 4 : 2, kParts = F32OUT ? 1 : 2;
    const int cols = Shape<P>::cols(a.N, a.K), c0 = t.c * kCols;
    const int64_t rows_before = (int64_t)t.part * (Shape<P>::kDw ? (int64_t)a.G * a.N : a.M) + (Shape<P>::kDw ? (int64_t)t.g * a.N : 0);
    const int rows = ADD && t.k0 == t.k1 ? 0 : t.r1 - t.r0;                 // (nothing to add: nothing is touched)
    const int ld = cols * kSize;
    const auto out = __builtin_amdgcn_make_buffer_rsrc((uint8_t*)a.out + ((rows_before + t.r0) * cols + c0) * kSize, 0,
                                                       rows > 0 ? rows * ld - c0 * kSize : 0, 0x00020000);
    int r = (int)l.row, q = (int)l.q;
    asm volatile("" : "+v"(r), "+v"(q));                 // (keeps the addresses from being made before the sums)
    const int n = (int)(128u * l.wn) + (F32OUT ? 4 * q : 16 * (q & 1) + 8 * (q >> 1));
    int at = ((int)(16u * TB * l.wm) + r) * ld + n * kSize;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const auto place = [&](int i) { return c0 + n + 16 * i < cols ? at + 16 * i * kSize : (int)0x80000000; };
        v4f old[8];
        if constexpr (ADD) {                             // (a row of parts asked for together)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) old[i] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(out, place(i), 0, 0));
        }
#pragma unroll
        for (int i = 0; i < 8; i += kParts) {
            // one part at a time leaves the accumulators' registers
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < kParts; ++k) asm volatile("" : "+a"(acc[i + k][j]));
            const v4f v = acc[i][j];
            u32x4 p;
            if constexpr (F32OUT) {
                p = __builtin_bit_cast(u32x4, v);
            } else {
                const v4f w = acc[i + 1][j];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const auto x = __builtin_amdgcn_permlane16_swap(f32_pair_to_bf16(v[2 * k], v[2 * k + 1]),
                                                                    f32_pair_to_bf16(w[2 * k], w[2 * k + 1]), false, false);
                    p[k] = x[0];
                    p[k + 2] = x[1];
                }
            }
            if constexpr (ADD) p = __builtin_bit_cast(u32x4, old[i] + v);
            __builtin_amdgcn_raw_buffer_store_b128(p, out, place(i), 0, 0);
        }
        at += 16 * ld;
    }
}

// One tile: its slots are the next to come out of the stream, the first of them in ring slot s;
// the slot after it has been asked for.
template <int P, int TB, bool F32OUT, bool ADD>
__device__ __forceinline__ void tile_product(Loader<P>& ld, const MmArgs& a, const TileList& list, int count, const Tile& t,
                                             Lane<P>& l, uint32_t base, uint32_t& s)
{
    v4f acc[8][TB];
    Operands<TB> f[2];
    l.b.set(base + s * kSlotBytes + kOperandBytes, TB * l.wm);
    const int nslots = uniform(slots_of(t));
    s = (uint32_t)uniform((int)s);
    ld.make_uniform();
    read_step<P, TB, 0, 0, kPieces<P, TB>>(f[0], l);
    step0<P, TB, true>(acc, f, ld, l, s);
    for (int i = 1; i < nslots; ++i) {
        step1<P, TB, false>(acc, f, ld, l, s);
        pin<TB>(acc);
        ld.advance(a, list, count);
        s ^= 1u;
        step0<P, TB, false>(acc, f, ld, l, s);
        pin<TB>(acc);
    }
    step1<P, TB, true>(acc, f, ld, l, s);
    pin<TB>(acc);
    ld.advance(a, list, count);
    s ^= 1u;
    store_tile<P, TB, F32OUT, ADD>(acc, a, t, l);
}

template <int P, bool F32OUT, bool ADD>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void bf16_mm_kernel(const MmArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLdsBytes];
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    TileList list;
    int rows_end;
    int count;
    {
        count = uniform(make_list<P>(a, lds, list, &rows_end));
        rows_end = uniform(rows_end);
    }
    __syncthreads();                                     // the scan's arrays are free
    if (count > 0) {
        const Tile last = list.at(count - 1);
        if (last.r0 == last.r1) --count;
    }

    if (count > 0) {
        Lane<P> l;
        l.row = (uint32_t)(lane & 15);
        l.q = (uint32_t)(lane >> 4);
        l.wn = (uint32_t)(wave >> 1);
        l.wm = (uint32_t)(wave & 1);
        const uint32_t base = (uint32_t)(uintptr_t)(LdsPtr)lds;
        l.a.set(base, 8 * l.wn);
        Loader<P> ld;
        ld.set_lanes(a, lds, wave, lane);
        ld.entry = 0;
        ld.set_tile(a, list, count);
        ld.template issue_some<0, 16>(0);
        ld.advance(a, list, count);
        ld.template issue_some<0, 16>(1);
        ld.advance(a, list, count);
        slot_barrier<16>();
        uint32_t s = 0;
        for (int e = 0; e < count; ++e) {
            const Tile t = list.at(e);
            // a group's last tile runs at the smallest of three heights that holds its rows
            const int rows = t.r1 - t.r0;
            if (rows > 128) tile_product<P, 8, F32OUT, ADD>(ld, a, list, count, t, l, base, s);
            else if (rows > 64) tile_product<P, 4, F32OUT, ADD>(ld, a, list, count, t, l, base, s);
            else tile_product<P, 2, F32OUT, ADD>(ld, a, list, count, t, l, base, s);
        }
        slot_barrier<0>();                               // the loads past the end land before the LDS goes away
    }

    if constexpr (!Shape<P>::kDw) {                      // rows past the last end: zeros, in every part
        const int64_t per_row = (int64_t)Shape<P>::cols(a.N, a.K) * (F32OUT ? 4 : 2) / 16;
        const int64_t total = (int64_t)(a.M - rows_end) * per_row;
        for (int p = 0; p < a.split; ++p) {
            uint4* y = (uint4*)a.out + ((int64_t)p * a.M + rows_end) * per_row;
            for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads)
                y[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

// out = the sum of `parts` arrays of n4 float4, in order (and of what out holds).
template <bool F32OUT>
__global__ __launch_bounds__(kThreads)
void join_parts_kernel(const float4* __restrict__ part, int parts, int64_t n4, void* out, int accumulate)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n4; i += (int64_t)gridDim.x * kThreads) {
        float4 v = part[i];
        for (int p = 1; p < parts; ++p) {
            const float4 w = part[p * n4 + i];
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
        }
        if constexpr (F32OUT) {
            float4* to = (float4*)out + i;
            if (accumulate) {
                const float4 w = *to;
                v.x += w.x;
                v.y += w.y;
                v.z += w.z;
                v.w += w.w;
            }
            *to = v;
        } else {
            ((uint2*)out)[i] = make_uint2(f32_pair_to_bf16(v.x, v.y), f32_pair_to_bf16(v.z, v.w));
        }
    }
}

// How a product is cut: rows of a tile, parts of its sum, tiles at most (parts counted).
struct Plan {
    int rows, split;
    int64_t items;
};
constexpr int kCus = 256;
Plan plan_of(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    const bool dw = product == MXQ_PRODUCT_DW;
    const int64_t cols = ((product == MXQ_PRODUCT_Y ? N : K) + kCols - 1) / kCols;
    const auto tiles = [&](int rows) {
        return (dw ? G * ((N + rows - 1) / rows) : (M + rows - 1) / rows + (G < M ? G : M) - 1) * cols;
    };
    Plan p;
    p.rows = tiles(256) >= kCus ? 256 : 128;
    const int64_t n = tiles(p.rows);
    // Slots of an average sum; a part has four or more.  A short sum is not worth the second
    // launch (8192 rows x 512 x 512, 8 slots: 28 us in two parts, 16 in one).
    const int64_t slots = ((dw ? M / G : product == MXQ_PRODUCT_Y ? K : N) + kSlotK - 1) / kSlotK;
    int64_t split = n > 0 ? kCus / n : 1;
    if (split > slots / 4) split = slots / 4;
    if (slots < 16) split = 1;
    if (split > kMaxSplit) split = kMaxSplit;
    p.split = split < 1 ? 1 : (int)split;
    p.items = n * p.split;
    return p;
}
// Few rows go to launch_bf16_mm_few (Y / dX, few against tiles, us): 16 experts of 8192 x 5120, 8 rows
// 84 / 103 against 100 / 142, 256 rows 255 / 305 against 290 / 312, 512 rows 309 / 359 against 295 /
// 309; one expert, 256 rows 40 / 63 against 51 / 57.  More rows too while the whole product is
// small: one expert of 512 x 512, 4096 rows 12 / 12 against 24 / 24, 8192 rows 24 / 24 against 28 /
// 28, 16384 rows 43 / 43 against 18 / 18; 8 of 256 x 128, 16384 rows 19 / 14 against 12 / 13; 2 of
// 1736 x 1408, 1024 rows 16 / 21 against 29 / 25; 8 of 2048 x 768, 1024 rows 18 / 15 against 24 /
// 23, 2048 rows 28 / 25 against 19 / 27.  dW of few results and sums that are not long: 4000 rows, 8
// experts of 512 x 512, 15 against 27; 10 of 208 x 152, 9 against 22, 16000 rows 31 against 22; one of
// 240 x 600, 1000 rows 8 against 13, 4000 rows 23 against 19; 16 of 1024 x 1024, 1000 rows, 56 against 20.
bool few_rows(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    if (product == MXQ_PRODUCT_DW)
        return M > 0 && M <= 8192 && M <= 2048 * G && G * ((N + 63) / 64) * ((K + 63) / 64) <= 512 && M * N * K <= (int64_t)1 << 30;
    return M > 0 &&
           (M <= 256 || (M <= 1024 && M * N * K <= (int64_t)1 << 31) || (M <= 16384 && M * N * K <= (int64_t)1 << 30));
}
int64_t results_of(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    return product == MXQ_PRODUCT_Y ? M * N : product == MXQ_PRODUCT_DX ? M * K : G * N * K;
}

}  // namespace

bool bf16_mm_sizes_ok(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    constexpr int64_t kMaxSide = (int64_t)1 << 20;
    if (M < 0 || M > ((int64_t)1 << 31) - 1024 || G < 1 || G > kMaxGroups) return false;
    if (N < 8 || N > kMaxSide || N % 8 != 0 || K < 8 || K > kMaxSide || K % 8 != 0) return false;
    if (G * N * K > (int64_t)1 << 40) return false;
    const int64_t rows = product == MXQ_PRODUCT_DW ? G * ((N + 63) / 64) : M / 64 + G;
    const int64_t cols = ((product == MXQ_PRODUCT_Y ? N : K) + 255) / 256;
    return rows < ((int64_t)1 << 30) / cols;
}

// Parts of a product's sums.
static int split_of(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    if (M == 0) return 1;
    if (few_rows(product, M, N, K, G)) return bf16_mm_few_split(product, (int)M, (int)N, (int)K, (int)G);
    return plan_of(product, M, N, K, G).split;
}

size_t bf16_mm_workspace_bytes(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    const int split = split_of(product, M, N, K, G);
    return split > 1 ? (size_t)split * (size_t)results_of(product, M, N, K, G) * 4u : 0;
}

static hipError_t join_parts(const void* parts, int split, int64_t results, void* out, bool f32_out, bool accumulate,
                             hipStream_t stream)
{
    const int64_t n4 = results / 4, blocks = (n4 + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
    if (f32_out)
        hipLaunchKernelGGL(join_parts_kernel<true>, grid, dim3(kThreads), 0, stream, (const float4*)parts, split, n4, out,
                           (int)accumulate);
    else
        hipLaunchKernelGGL(join_parts_kernel<false>, grid, dim3(kThreads), 0, stream, (const float4*)parts, split, n4, out, 0);
    return hipGetLastError();
}

hipError_t launch_bf16_mm(int product, const void* rows, const void* other, const int32_t* offs, int M, int N, int K, int G,
                          void* out, bool f32_out, bool accumulate, void* workspace, hipStream_t stream)
{
    const int split = split_of(product, M, N, K, G);
    const bool joined = split > 1;
    if (few_rows(product, M, N, K, G)) {
        const hipError_t e = launch_bf16_mm_few(product, rows, other, offs, M, N, K, G, split, joined ? workspace : out,
                                                f32_out || joined, accumulate, stream);
        if (e != hipSuccess || !joined) return e;
        return join_parts(workspace, split, results_of(product, M, N, K, G), out, f32_out, false, stream);   // (not dW)
    }
    int device = 0, cus = 0;
    hipError_t e = hipGetDevice(&device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (e != hipSuccess) return e;
    const Plan p = plan_of(product, M, N, K, G);
    // One workgroup a CU, fewer when there are not that many tiles (their row parts counted), a
    // multiple of it when a workgroup's list would not hold its tiles: an XCD's stretch of the
    // work has at most kCostWhole / kCostQuarter times an eighth of the tiles and two, a
    // workgroup of grid / 8 its part of them and one.
    const int64_t parts = p.items * (p.rows / 64), most =
        (product == MXQ_PRODUCT_DW ? p.items : p.items * kCostWhole / kCostQuarter) + 2 * kXcds + 1;
    int64_t grid = parts < cus ? (parts > 0 ? parts : 1) : cus;
    grid *= (most + grid * (kMaxEntries - 1) - 1) / (grid * (kMaxEntries - 1));
    grid = (grid + kXcds - 1) / kXcds * kXcds;
    const bool wide = f32_out || joined;
    const MmArgs a = {(const uint16_t*)other, (const uint16_t*)rows, offs, joined ? workspace : out, M, N, K, G, p.rows,
                      split};
#define MXQ_LAUNCH(P, F32, ADD) \
    hipLaunchKernelGGL((bf16_mm_kernel<P, F32, ADD>), dim3((unsigned)grid), dim3(kThreads), 0, stream, a)
    if (product == MXQ_PRODUCT_DW && accumulate && !joined) MXQ_LAUNCH(MXQ_PRODUCT_DW, true, true);
    else if (product == MXQ_PRODUCT_DW && wide) MXQ_LAUNCH(MXQ_PRODUCT_DW, true, false);
    else if (product == MXQ_PRODUCT_DW) MXQ_LAUNCH(MXQ_PRODUCT_DW, false, false);
    else if (product == MXQ_PRODUCT_DX && wide) MXQ_LAUNCH(MXQ_PRODUCT_DX, true, false);
    else if (product == MXQ_PRODUCT_DX) MXQ_LAUNCH(MXQ_PRODUCT_DX, false, false);
    else if (wide) MXQ_LAUNCH(MXQ_PRODUCT_Y, true, false);
    else MXQ_LAUNCH(MXQ_PRODUCT_Y, false, false);
#undef MXQ_LAUNCH
    if (!joined) return hipGetLastError();
    return join_parts(workspace, split, results_of(product, M, N, K, G), out, f32_out, accumulate, stream);
}

}  // namespace mxq
