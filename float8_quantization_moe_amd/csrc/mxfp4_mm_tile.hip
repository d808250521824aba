// mxfp4_mm_tile.hip -- the product of MXFP8 or MXFP4 token rows with MXFP4 expert
// weights for groups of many rows (mxfp4_mm.hip states the operation and takes the
// calls with few rows).
//
// Persistent workgroups (one a CU, 4 waves in 2 x 2) walk over output tiles of 256
// columns x 256 rows (128 where that leaves CUs idle).  K advances 256 values a slot
// through a 2-slot LDS ring of 32 KB of W codes and 32 KB of X codes (of E4M3 tokens, with
// twice the bytes and MFMAs of twice the time, half a slot's), filled by
// buffer-load-to-LDS in whole 128-byte lines.  Scales come 32 bytes a row for four slots.
// A slot is four MFMA steps of 64 k; a step's operands are read from LDS during the step
// before it.  With one wave a SIMD nothing issues while a load or an LDS read waits for
// its pipe, so both are spread between the MFMAs, one or two after each (`mfmas`).
// Measured, E4M3 / E2M1: one group of 16384 x 8192 x 5120 480 / 328 us (2.9 / 4.2 PFLOP/s), 16640
// rows in 16 ragged groups 553 / 393.  What bounds it is the clock under this power (on
// zeros 370 / 244 us) and the load path; eight waves of 128 x 64, two a SIMD, took 485 / 333.
//
// The slots of successive tiles form one stream: the loads run ahead of the
// products across the end of a tile, so the next tile's operands arrive while this
// one's results are stored (straight from the accumulators: the LDS belongs to the
// next tile by then).  One workgroup a CU leaves nothing else to hide them.
//
// Tile list: row tiles never straddle a group.  Group by group, inside a group in
// blocks of kColBlock column tiles with the block's row tiles consecutive, so that
// neighbours in the list share W and X tiles; each of the 8 XCDs (workgroup index
// mod 8) walks one contiguous stretch, its CUs side by side, the last round's tiles in
// smaller parts where that fills CUs.  Every workgroup finds
// its own tiles from the group offsets (a scan in LDS), so no launch comes before.
//
// MFMA operand A is W (output columns), B is X (token rows).  In a 64-k step, lane
// (r, h) = (lane % 32, lane / 32) holds of row r: E2M1, the 16 bytes of scale block
// h; E4M3, the 16-byte chunks h and h + 2.  Its scale byte is that of block h.
#include "device_common.hpp"
#include "internal.hpp"
#include "mm_tile.hpp"

namespace mxq {

namespace {

constexpr int kThreads = kTileThreads;
constexpr int kCols = 256;                               // columns of a tile
constexpr int kSlotK = 256;
constexpr uint32_t kOperandBytes = 32 * 1024;            // codes of one operand in one slot
constexpr uint32_t kSlotBytes = 2 * kOperandBytes;
constexpr uint32_t kScaleOperand = 256 * 32;             // scales of one operand for four slots
constexpr uint32_t kScaleBase = 2 * kSlotBytes;
constexpr uint32_t kLdsBytes = kScaleBase + 2 * 2 * kScaleOperand;
constexpr int kMaxEntries = 64;                          // tiles of one workgroup: one a lane
static_assert(kLdsBytes <= 160 * 1024, "LDS of a CU");
// Tiles of 128 rows while there is less than one of 256 rows for each CU: 777 ragged
// rows x 1736 x 1408 over 16 groups (126 tiles of 256 rows) 14.4 / 12.2 us (E4M3 /
// E2M1) against 17.7 / 14.5; the other way round above that: one group of 16384 rows
// 632 / 486 against 538 / 379.
constexpr int kManyTiles = 1;
// Column tiles of a block of the tile order.  One group of 16384 x 8192 x 5120, E4M3 / E2M1:
// 1 530 / 359 us, 2 482 / 317, 3 471 / 316, 4 468 / 316; 16 ragged groups 559 / 389, 553 /
// 389, 557 / 392, 557 / 394.
constexpr int kColBlock = 2;
// CUs by which the order moves on each round.  The short last tiles of equal groups come at
// one place of every round, and would come to the same CUs; with a shift of 6, 16640 x 8192
// x 5120 over 16 ragged groups, E4M3, 622 -> 590 us, 20000 x 4096 x 4096 over 24 320 -> 300
// (E2M1 434 -> 434, 232 -> 225; shifts of 1, 2, 3, 10 within the noise of it).
constexpr int kShift = 6;
constexpr int kXcds = 8;
constexpr int kMaxGroups = 4095;
static_assert((2 * (kMaxGroups + 2) + kThreads) * 4 <= (int)kScaleBase, "the scan's arrays fit the ring");

struct Tile {
    int g, r0, r1, c;                                    // group, rows [r0, r1), column tile c
};

// A workgroup's list: tile e in lane e of every wave.
struct TileList {
    Tile mine;
    __device__ __forceinline__ Tile at(int e) const
    {
        return Tile{__builtin_amdgcn_readlane(mine.g, e), __builtin_amdgcn_readlane(mine.r0, e),
                    __builtin_amdgcn_readlane(mine.r1, e), __builtin_amdgcn_readlane(mine.c, e)};
    }
};

struct MmArgs {
    const uint8_t *xq, *xs, *wq, *ws;
    const int32_t* offs;
    void* y;
    uint32_t ldx, ldxs;
    int M, N, K, G;
    int rows;                                            // token rows of a tile, at most: 128 or 256
};

// -------------------------------------------------------------- tile list ---
// Fills `list` with this workgroup's tiles and returns their number; *rows_end is
// the last group's clamped end.  end_sh: the groups' clamped ends; first_sh: each
// group's first row tile.
__device__ int make_list(const MmArgs& a, int* end_sh, int* first_sh, int* scan_sh, TileList& list, int* rows_end)
{
    const int t = (int)threadIdx.x, R = a.rows;
    const int per = (a.G + kThreads - 1) / kThreads;
    const int ga = t * per < a.G ? t * per : a.G, gb = ga + per < a.G ? ga + per : a.G;
    int top = 0;
    for (int g = ga; g < gb; ++g) {
        const int e = a.offs[g];
        top = e > top ? e : top;
        end_sh[g] = top < a.M ? top : a.M;
    }
    const int upto = block_scan<true>(top, scan_sh);
    if (t < kThreads) scan_sh[t] = upto;
    __syncthreads();
    const int before = t ? scan_sh[t - 1] : 0;
    const int base = before < a.M ? before : a.M;
    for (int g = ga; g < gb; ++g) end_sh[g] = end_sh[g] > base ? end_sh[g] : base;
    int tiles = 0;
    for (int g = ga, start = base; g < gb; ++g) {
        tiles += (end_sh[g] - start + R - 1) / R;
        start = end_sh[g];
    }
    __syncthreads();
    int first = block_scan<false>(tiles, scan_sh) - tiles;
    for (int g = ga, start = base; g < gb; ++g) {
        first_sh[g] = first;
        first += (end_sh[g] - start + R - 1) / R;
        start = end_sh[g];
    }
    if (t == kThreads - 1) first_sh[a.G] = first;
    __syncthreads();

    const int NC = (a.N + kCols - 1) / kCols;
    const int V = first_sh[a.G] * NC;
    const int x = (int)blockIdx.x % kXcds, cu = (int)blockIdx.x / kXcds, cus = (int)gridDim.x / kXcds;
    const int lo = (int)((int64_t)V * x / kXcds), n = (int)((int64_t)V * (x + 1) / kXcds) - lo;
    // The tiles left after the last full round are cut in row parts of 64 or more while
    // that gives no more than one for each CU (2048 x 8192 x 5120 over 4 groups, 12 tiles
    // for 8 CUs: 90 / 66 us E4M3 / E2M1 against 114 / 76; 8192 x 4096 x 2048 over 32: 92 /
    // 68 against 102 / 74).
    const int full = n / cus, over = n - full * cus;
    const int parts = 4 * over <= cus && R == 256 ? 4 : 2 * over <= cus ? 2 : 1;
    const int count = full + (cu < over * parts);
    const int j = lane_id();
    list.mine = Tile{0, 0, 0, 0};
    if (j < count) {
        const int L = lo + j * cus + (j < full ? (cu + kShift * j) % cus : cu / parts);
        int p = 0, r = a.G - 1;                          // the last group whose tiles start at or before L
        while (p < r) {
            const int mid = (p + r + 1) >> 1;
            if (first_sh[mid] * NC <= L) p = mid;
            else r = mid - 1;
        }
        const int rt = first_sh[p + 1] - first_sh[p];
        const int local = L - first_sh[p] * NC;
        const int cb = local / (rt * kColBlock);
        const int rem = local - cb * rt * kColBlock;
        const int width = NC - cb * kColBlock < kColBlock ? NC - cb * kColBlock : kColBlock;
        const int height = j < full ? R : R / parts, part = j < full ? 0 : cu % parts;
        Tile tl;
        tl.g = p;
        tl.r0 = (p ? end_sh[p - 1] : 0) + rem / width * R + part * height;
        tl.r1 = tl.r0 + height < end_sh[p] ? tl.r0 + height : end_sh[p];
        if (tl.r1 < tl.r0) tl.r1 = tl.r0;                // a part past the group's rows
        tl.c = cb * kColBlock + rem % width;
        list.mine = tl;
    }
    *rows_end = end_sh[a.G - 1];
    return count < kMaxEntries ? count : kMaxEntries;
}

// ------------------------------------------------------------------ loads ---
// The stream of slots to load.  E2M1 tokens: a slot's X codes (128 bytes a row)
// travel with its W codes and scales.  E4M3 tokens: 256 bytes a row, in two halves
// that each have one place in LDS; they run a slot behind the W codes, half by half.
//
// LDS rows of 128 bytes hold their eight 16-byte chunks at c ^ ((row >> 1) & 7): the
// 16 lanes that a 128-bit LDS read serves at a time then meet 16 different bank
// groups.  The swizzle is applied to the source offsets (the LDS side is linear in
// the lane).
template <bool X8>
struct Loader {
    v4i w, ws, xs;                                       // resources that start at the next slot
    v4i x, xb;                                           // X8: at its first half's and the running slot's second half
    int entry, left;                                     // the tile's place in the list; its slots from the next one on
    int phase;                                           // the next slot's place in its chunk of scales
    uint32_t chunk;                                      // the place in LDS of the next chunk
    int xentry, xleft;                                   // X8: the same of the X codes
    uint32_t off_w[8], off_x[8], off_ws[2], off_xs[2];   // lane offsets of the wave's loads, 8 rows each (scales: 32)
    uint32_t lds_data, lds_scale;                        // LDS addresses of the wave's part of ring slot 0
    uint32_t upper;                                      // bit 31: this lane's chunk of load 0 is in the second half of a row's slot

    __device__ __forceinline__ void set_lanes(const MmArgs& a, const uint8_t* lds, int wave, int lane)
    {
        const uint32_t half = (uint32_t)a.K / 2u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t row = (uint32_t)(64 * wave + 8 * i + (lane >> 3));
            const uint32_t chunk = ((uint32_t)lane & 7u) ^ ((row >> 1) & 7u);
            off_w[i] = row * half + 16u * chunk;
            off_x[i] = row * a.ldx + 16u * chunk;
        }
        upper = ((uint32_t)lane >> 2) << 31;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t row = (uint32_t)(64 * wave + 32 * i + (lane >> 1));
            const uint32_t part = 16u * (((uint32_t)lane ^ (row >> 3)) & 1u);
            off_ws[i] = row * ((uint32_t)a.K / 32u) + part;
            off_xs[i] = row * a.ldxs + part;
        }
        const uint32_t base = (uint32_t)uniform((int)(uint32_t)(uintptr_t)(LdsPtr)lds);
        lds_data = base + 8192u * (uint32_t)wave;
        lds_scale = base + kScaleBase + 2048u * (uint32_t)wave;
    }

    // Tile e of the list; past its end, one that loads nothing.
    struct Place {
        int64_t wrow;
        int r0;
        uint32_t nw, nx;
    };
    static __device__ __forceinline__ Place place_of(const MmArgs& a, const TileList& list, int e, int count)
    {
        const bool some = e < count;
        const Tile t = list.at(some ? e : 0);
        const int n0 = t.c * kCols;
        Place p;
        p.r0 = t.r0;
        p.nx = some ? (uint32_t)(t.r1 - t.r0) : 0u;
        p.nw = some ? (uint32_t)(a.N - n0 < kCols ? a.N - n0 : kCols) : 0u;
        p.wrow = (int64_t)t.g * a.N + n0;
        return p;
    }
    // The first slot of tile `entry`: W codes and both scales, and of E2M1 tokens the X codes.
    __device__ __forceinline__ void set_tile(const MmArgs& a, const TileList& list, int count, int nslots)
    {
        const uint32_t half = (uint32_t)a.K / 2u, kb = (uint32_t)a.K / 32u;
        const Place p = place_of(a, list, entry, count);
        left = nslots;
        phase = 0;
        w = resource(a.wq + p.wrow * half, p.nw * half);
        ws = resource(a.ws + p.wrow * kb, p.nw * kb);
        xs = resource(a.xs + (int64_t)p.r0 * a.ldxs, p.nx ? (p.nx - 1u) * a.ldxs + kb : 0u);
        if constexpr (!X8) x = resource(a.xq + (int64_t)p.r0 * a.ldx, p.nx ? (p.nx - 1u) * a.ldx + half : 0u);
    }
    __device__ __forceinline__ void set_x_tile(const MmArgs& a, const TileList& list, int count, int nslots)
    {
        const Place p = place_of(a, list, xentry, count);
        xleft = nslots;
        x = resource(a.xq + (int64_t)p.r0 * a.ldx, p.nx ? (p.nx - 1u) * a.ldx + (uint32_t)a.K : 0u);
    }

    // (Signed, so that the bound is a scalar maximum: an unsigned saturating subtraction
    // is vector code, and the resources have to stay in scalar registers.)
    static __device__ __forceinline__ v4i stepped(const v4i& r, int bytes, bool nothing = false)
    {
        const uint64_t base = (((uint64_t)(uint32_t)r.y << 32) | (uint32_t)r.x) + (uint32_t)bytes;
        const int left = r.z - bytes > 0 ? r.z - bytes : 0;
        return v4i{(int)(uint32_t)base, (int)(uint32_t)(base >> 32), nothing ? 0 : left, 0x00020000};
    }
    // On to the next slot of the stream.  Where K ends half way through a tile's last
    // slot, that slot's X codes past K are to be zeros: E4M3, its second half loads
    // nothing; E2M1, for its loads their lanes' offsets leave the resource (bit 31).
    __device__ __forceinline__ void advance(const MmArgs& a, const TileList& list, int count, int nslots)
    {
        if constexpr (X8) {
            xb = stepped(x, 128, xleft == 1 && a.K % kSlotK != 0);
            if (xleft == 1) {
                ++xentry;
                set_x_tile(a, list, count, nslots);
            } else {
                --xleft;
                x = stepped(x, 256);
            }
        }
        const bool was_last = left == 1;
        if (was_last) {
            ++entry;
            set_tile(a, list, count, nslots);
        } else {
            --left;
            phase = (phase + 1) & 3;
            w = stepped(w, 128);
            ws = stepped(ws, 8);
            xs = stepped(xs, 8);
            if constexpr (!X8) x = stepped(x, 128);
        }
        if constexpr (!X8) {
            if (a.K % kSlotK != 0 && was_last != (left == 1)) toggle_half();
        }
    }
    __device__ __forceinline__ void toggle_half()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) off_x[i] ^= (i & 1) ? upper ^ 0x80000000u : upper;
    }

    // Scales travel in chunks of 32 bytes a row, four slots' worth: a row is a line of its
    // own, which costs the memory pipe as much as 128 bytes of codes.  (One group of 16384 x
    // 8192 x 5120, E2M1: 16 bytes a slot, half of them unused, 374 us; 16 for two slots 351;
    // with the later steps' gains, 16 for two 341, 32 for four 333.)  The two 16-byte parts
    // of a row trade places in every other 8 rows, so that 16 rows' words meet 16 different
    // pairs of banks.
    __device__ __forceinline__ void issue_scales()
    {
        const uint32_t to = lds_scale + chunk * 2u * kScaleOperand;
        load_to_lds<3>(ws, to, off_ws[0]);
        load_to_lds<3>(ws, to + 1024u, off_ws[1]);
        load_to_lds<3>(xs, to + kScaleOperand, off_xs[0]);
        load_to_lds<3>(xs, to + kScaleOperand + 1024u, off_xs[1]);
        chunk ^= 1u;
    }
    // Load I of the slot's codes into ring slot b: W, then (E2M1) X.
    template <int I>
    __device__ __forceinline__ void issue(uint32_t b)
    {
        constexpr int i = I % 8;
        if constexpr (I < 8) load_to_lds(w, lds_data + b * kSlotBytes + 1024u * i, off_w[i]);
        else load_to_lds(x, lds_data + b * kSlotBytes + kOperandBytes + 1024u * i, off_x[i]);
    }
    template <int I, int END>
    __device__ __forceinline__ void issue_some(uint32_t b)
    {
        if constexpr (I < END) {
            issue<I>(b);
            issue_some<I + 1, END>(b);
        }
    }
    // X8: loads I .. END - 1 (of 8) of X half H.
    template <int H, int I, int END>
    __device__ __forceinline__ void issue_x()
    {
        if constexpr (I < END) {
            load_to_lds(H ? xb : x, lds_data + H * kSlotBytes + kOperandBytes + 1024u * I, off_x[I]);
            issue_x<H, I + 1, END>();
        }
    }
};

// --------------------------------------------------------------- products ---
template <bool X8, int TM>
struct Operands {
    v4i w[4];
    v4i x[TM][X8 ? 2 : 1];
};
template <int TM>
struct Scales {
    uint2 w[4], x[TM];                                   // two words of four blocks each: a slot
};

struct Lane {
    uint32_t row, h, swz;                                // lane % 32, lane / 32, and its rows' swizzle
    uint32_t wn, wm;                                     // the wave's place in the 2 x 2
};

// Pieces P .. END - 1 of a step's operands: 4 of W, then those of X.
template <bool X8, int TM>
constexpr int kPieces = 4 + TM * (X8 ? 2 : 1);
template <bool X8, int TM, int T, int P, int END>
__device__ __forceinline__ void read_step(Operands<X8, TM>& f, const uint8_t* lds, uint32_t b, const Lane& l)
{
    if constexpr (P < END) {
        if constexpr (P < 4) {
            const uint8_t* W = lds + b * kSlotBytes + (128u * l.wn + l.row) * 128u + (((2u * T + l.h) ^ l.swz) << 4);
            f.w[P] = *(const v4i*)(W + 4096 * P);
        } else {
            constexpr int p = (P - 4) / TM, i = (P - 4) % TM;
            const uint8_t* X = lds + (X8 ? (uint32_t)(T / 2) : b) * kSlotBytes + kOperandBytes + (32u * TM * l.wm + l.row) * 128u +
                               ((((X8 ? 4u * (T % 2) + 2u * p : 2u * T) + l.h) ^ l.swz) << 4);
            f.x[i][p] = *(const v4i*)(X + 4096 * i);
        }
        read_step<X8, TM, T, P + 1, END>(f, lds, b, l);
    }
}

// A slot's scale words: place `at` in LDS is its chunk's and 8 bytes a slot.
__device__ __forceinline__ uint32_t next_scales(uint32_t at, bool new_tile)
{
    constexpr uint32_t kChunk = 2u * kScaleOperand;
    return new_tile || (at & 24u) == 24u ? (at & kChunk) ^ kChunk : at + 8u;
}
template <int TM, int P, int END>
__device__ __forceinline__ void read_scales(Scales<TM>& s, const uint8_t* lds, uint32_t at, const Lane& l)
{
    if constexpr (P < END) {
        const uint8_t* p = lds + kScaleBase + (at ^ (2u * (l.row & 8u)));
        if constexpr (P < 4) s.w[P] = *(const uint2*)(p + (128u * l.wn + 32u * P + l.row) * 32u);
        else s.x[P - 4] = *(const uint2*)(p + kScaleOperand + (32u * TM * l.wm + 32u * (P - 4) + l.row) * 32u);
        read_scales<TM, P + 1, END>(s, lds, at, l);
    }
}
// Shifted so that bytes 0 and 2 of a word are the lane's blocks.
template <int TM>
__device__ __forceinline__ void shift_scales(Scales<TM>& s, const Lane& l)
{
    const uint32_t n = 8u * l.h;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.w[i].x >>= n, s.w[i].y >>= n;
#pragma unroll
    for (int i = 0; i < TM; ++i) s.x[i].x >>= n, s.x[i].y >>= n;
}

__device__ __forceinline__ v8i low4(const v4i& v) { return v8i{v.x, v.y, v.z, v.w, 0, 0, 0, 0}; }

// MFMA I of the 4 x TM of step T; ZERO: the sums start here.
template <bool X8, int TM, int T, bool ZERO, int I>
__device__ __forceinline__ void mfma(v16f (&acc)[4][TM], const Operands<X8, TM>& f, const Scales<TM>& s)
{
    constexpr int i = I / TM, j = I % TM;
    const int sw = (int)(T < 2 ? s.w[i].x : s.w[i].y), sx = (int)(T < 2 ? s.x[j].x : s.x[j].y);
    v16f c = acc[i][j];
    if constexpr (ZERO) c = v16f{};
    v8i x;
    if constexpr (X8) x = v8i{f.x[j][0].x, f.x[j][0].y, f.x[j][0].z, f.x[j][0].w, f.x[j][1].x, f.x[j][1].y, f.x[j][1].z, f.x[j][1].w};
    else x = low4(f.x[j][0]);
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low4(f.w[i]), x, c, 4, X8 ? 0 : 4, 2 * (T & 1), sw,
                                                                2 * (T & 1), sx);
}

// MFMAs I .. END - 1 of step T, each followed by its share of the other work of that
// stretch: work(k, n) does part k of n.
template <bool X8, int TM, int T, bool ZERO, int I, int END, int K = 0, class Work>
__device__ __forceinline__ void mfmas(v16f (&acc)[4][TM], const Operands<X8, TM>& f, const Scales<TM>& s, const Work& work)
{
    if constexpr (I < END) {
        mfma<X8, TM, T, ZERO, I>(acc, f, s);
        work(Int<K>{}, Int<K + END - I>{});
        __builtin_amdgcn_sched_barrier(0);
        mfmas<X8, TM, T, ZERO, I + 1, END, K + 1>(acc, f, s, work);
    }
}
// The bounds of part k of n of a .. b.
#define MXQ_PART(a, b) (a) + K.value * ((b) - (a)) / N.value, (a) + (K.value + 1) * ((b) - (a)) / N.value

// The order of a slot: its four steps in halves, what is loaded under each, and the
// barriers between them ("read": all waves' LDS reads are done; "there": all waves' loads
// have landed).
//
//                 E2M1 (16 loads a slot)             E4M3 (8 of W, 8 of each X half)
//   step 0        slot + 1: 8 .. 13                  W of slot + 1: 4 .. 7
//                                                    X half 0 is read
//     2nd half                                       X half 0 of slot + 1: 0 .. 3
//   step 1        slot + 1: 14, 15                                         4 .. 7
//                                                    X half 1 is there
//     2nd half
//   step 2
//                 the slot is read                   the slot is read
//     2nd half    slot + 2: 0, 1                     X half 1 of slot + 1: 0 .. 3
//   step 3        slot + 2: 2 .. 4                                         4 .. 7
//                 slot + 1 is there                  W, X half 0 of slot + 1 are there
//     2nd half    slot + 2: 5 .. 7                   W of slot + 2: 0 .. 3
//
// A place in LDS is loaded anew from half a step after its last operands were asked for,
// and waited for half a step before its first are used: a load has two steps or more to
// arrive.  16640 x 8192 x 5120 over 16 ragged groups, E4M3 / E2M1: 602 / 423 us with one
// barrier for both between steps 2 and 3 and a step's LDS reads ahead of its MFMAs, 586 /
// 421 with this order, 581 / 405 with the reads between the MFMAs too.
constexpr int kLoads2 = 2, kLoads3 = 5, kLoads3b = 8, kLoads0 = 14;   // E2M1: loads issued by the end of each stretch

template <bool X8, int TM, bool FIRST>
__device__ __forceinline__ void steps01(v16f (&acc)[4][TM], Operands<X8, TM> (&f)[2], Scales<TM>& s, Loader<X8>& ld,
                                        const uint8_t* lds, const Lane& l, uint32_t b)
{
    constexpr int h = 2 * TM, n = 4 * TM, P = kPieces<X8, TM>;
    if (ld.phase == 0) ld.issue_scales();
    shift_scales<TM>(s, l);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (X8) {
        mfmas<X8, TM, 0, FIRST, 0, h>(acc, f[0], s, [&](auto K, auto N) {
            read_step<X8, TM, 1, MXQ_PART(0, P)>(f[1], lds, b, l);
            ld.template issue_some<MXQ_PART(4, 8)>(b ^ 1u);
        });
        slot_barrier<63>();
        mfmas<X8, TM, 0, FIRST, h, n>(acc, f[0], s, [&](auto K, auto N) { ld.template issue_x<0, MXQ_PART(0, 4)>(); });
        mfmas<X8, TM, 1, false, 0, h>(acc, f[1], s, [&](auto K, auto N) { ld.template issue_x<0, MXQ_PART(4, 8)>(); });
        slot_barrier<16>();                              // (newer: W and X half 0 of the next slot)
        mfmas<X8, TM, 1, false, h, n>(acc, f[1], s, [&](auto K, auto N) { read_step<X8, TM, 2, MXQ_PART(0, P)>(f[0], lds, b, l); });
    } else {
        mfmas<X8, TM, 0, FIRST, 0, n>(acc, f[0], s, [&](auto K, auto N) {
            read_step<X8, TM, 1, MXQ_PART(0, P)>(f[1], lds, b, l);
            ld.template issue_some<MXQ_PART(kLoads3b, kLoads0)>(b ^ 1u);
        });
        mfmas<X8, TM, 1, false, 0, h>(acc, f[1], s, [&](auto K, auto N) {
            ld.template issue_some<MXQ_PART(kLoads0, 16)>(b ^ 1u);
            read_step<X8, TM, 2, MXQ_PART(0, P / 2)>(f[0], lds, b, l);
        });
        mfmas<X8, TM, 1, false, h, n>(acc, f[1], s, [&](auto K, auto N) { read_step<X8, TM, 2, MXQ_PART(P / 2, P)>(f[0], lds, b, l); });
    }
}

// On exit f[0] and s hold the next slot's first step and scales, unless this is the
// tile's LAST.
template <bool X8, int TM, bool LAST>
__device__ __forceinline__ void steps23(v16f (&acc)[4][TM], Operands<X8, TM> (&f)[2], Scales<TM>& s, Loader<X8>& ld,
                                        const uint8_t* lds, const Lane& l, uint32_t b, uint32_t scales)
{
    constexpr int h = 2 * TM, n = 4 * TM, P = kPieces<X8, TM>;
    mfmas<X8, TM, 2, false, 0, h>(acc, f[0], s, [&](auto K, auto N) { read_step<X8, TM, 3, MXQ_PART(0, P)>(f[1], lds, b, l); });
    slot_barrier<63>();
    mfmas<X8, TM, 2, false, h, n>(acc, f[0], s, [&](auto K, auto N) {
        if constexpr (X8) ld.template issue_x<1, MXQ_PART(0, 4)>();
        else ld.template issue_some<MXQ_PART(0, kLoads2)>(b);
    });
    mfmas<X8, TM, 3, false, 0, h>(acc, f[1], s, [&](auto K, auto N) {
        if constexpr (X8) ld.template issue_x<1, MXQ_PART(4, 8)>();
        else ld.template issue_some<MXQ_PART(kLoads2, kLoads3)>(b);
    });
    slot_barrier<X8 ? 8 : kLoads3>();                         // (newer: X half 1 of the next slot; the slot after it)
    const Scales<TM> now = s;
    mfmas<X8, TM, 3, false, h, n>(acc, f[1], now, [&](auto K, auto N) {
        if constexpr (!LAST) {
            read_step<X8, TM, 0, MXQ_PART(0, P)>(f[0], lds, b ^ 1u, l);
            read_scales<TM, MXQ_PART(0, 4 + TM)>(s, lds, scales, l);
        }
        ld.template issue_some<MXQ_PART(X8 ? 0 : kLoads3, X8 ? 4 : kLoads3b)>(b);
    });
}
#undef MXQ_PART

// The sums are needed here: without this the compiler moves MFMAs past the loads
// that are meant to run under them, into the next basic block.
template <int TM>
__device__ __forceinline__ void pin(v16f (&acc)[4][TM])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) asm volatile("" : "+a"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
}

// Stores: lane (r, h) holds, of row r of each 32 x 32 part, columns 8 q + 4 h .. + 3
// for q = 0 .. 3.  bf16: the halves of the wave exchange every other 4 columns, so
// that a lane has 8 consecutive ones (16 bytes).  One group of 16384 x 8192 x 5120,
// E2M1 (bf16 out): 32-byte stretches 357 us, 64-byte ones 338, whole lines 337.
template <int TM, bool F32OUT>
__device__ __forceinline__ void store_tile(const v16f (&acc)[4][TM], const MmArgs& a, const Tile& t, const Lane& l)
{
    constexpr int kSize = F32OUT ? 4 : 2, kParts = F32OUT ? 1 : 2;
    const int n_lane = (int)(64u * (l.row >> 3 & 1u) + 32u * (l.row >> 4) + 16u * l.h) / kSize;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int m = t.r0 + (int)(32u * TM * l.wm + 32u * j + (l.row & 7u));
#pragma unroll
        for (int i = 0; i < 4; i += kParts) {
            __builtin_amdgcn_sched_barrier(0);           // (one block at a time in VGPRs)
            v4i p[4];
            if constexpr (F32OUT) {
                const v16f& v = acc[i][j];
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int k = 0; k < 4; ++k) p[s][k] = __float_as_int(v[4 * s + k]);
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const v16f& v = acc[i + s / 2][j];
                    const int q = 8 * (s % 2);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const auto w = __builtin_amdgcn_permlane32_swap(f32_pair_to_bf16(v[q + 2 * k], v[q + 2 * k + 1]),
                                                                        f32_pair_to_bf16(v[q + 2 * k + 4], v[q + 2 * k + 5]), false, false);
                        p[s][k] = (int)w[0];
                        p[s][k + 2] = (int)w[1];
                    }
                }
            }
            join_lines(p);
            const int n = t.c * kCols + (int)(128u * l.wn) + 32 * i + n_lane;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int row = m + 16 * (s % 2) + 8 * (s / 2);
                if (row < t.r1 && n < a.N) *(v4i*)((uint8_t*)a.y + ((int64_t)row * a.N + n) * kSize) = p[s];
            }
        }
    }
}

// One tile: its slots are the next to come out of the stream, the first of them in
// ring slot b; the loads are part way into the slot after it.
template <bool X8, int TM, bool F32OUT>
__device__ __forceinline__ void tile_product(Loader<X8>& ld, const MmArgs& a, const uint8_t* lds, const TileList& list, int count,
                                             const Tile& t, const Lane& l, int nslots, uint32_t& b, uint32_t& scales)
{
    v16f acc[4][TM];
    Operands<X8, TM> f[2];
    Scales<TM> s;
    read_scales<TM, 0, 4 + TM>(s, lds, scales, l);
    read_step<X8, TM, 0, 0, kPieces<X8, TM>>(f[0], lds, b, l);
    steps01<X8, TM, true>(acc, f, s, ld, lds, l, b);
    pin<TM>(acc);
    ld.advance(a, list, count, nslots);
    for (int i = 1; i < nslots; ++i) {
        scales = next_scales(scales, false);
        steps23<X8, TM, false>(acc, f, s, ld, lds, l, b, scales);
        pin<TM>(acc);
        b ^= 1u;
        steps01<X8, TM, false>(acc, f, s, ld, lds, l, b);
        pin<TM>(acc);
        ld.advance(a, list, count, nslots);
    }
    if (a.K % kSlotK != 0) {                             // (no scales past K)
#pragma unroll
        for (int i = 0; i < 4; ++i) s.w[i].y = 0;
#pragma unroll
        for (int j = 0; j < TM; ++j) s.x[j].y = 0;
    }
    steps23<X8, TM, true>(acc, f, s, ld, lds, l, b, scales);
    pin<TM>(acc);
    b ^= 1u;
    scales = next_scales(scales, true);
    store_tile<TM, F32OUT>(acc, a, t, l);
}

template <bool X8, bool F32OUT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mxfp4_mm_tile_kernel(const MmArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLdsBytes];
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    TileList list;
    int rows_end;
    int count;
    {
        int* end_sh = (int*)lds;
        int* first_sh = end_sh + kMaxGroups + 1;
        int* scan_sh = first_sh + kMaxGroups + 1;
        count = uniform(make_list(a, end_sh, first_sh, scan_sh, list, &rows_end));
        rows_end = uniform(rows_end);
    }
    __syncthreads();                                     // the scan's arrays are free
    if (count > 0) {
        const Tile last = list.at(count - 1);
        if (last.r0 == last.r1) --count;
    }

    if (count > 0) {
        const Lane l = {(uint32_t)(lane & 31), (uint32_t)(lane >> 5), (uint32_t)((lane >> 1) & 7),
                        (uint32_t)(wave >> 1), (uint32_t)(wave & 1)};
        const int nslots = (a.K + kSlotK - 1) / kSlotK;
        Loader<X8> ld;
        ld.set_lanes(a, lds, wave, lane);
        ld.entry = ld.xentry = 0;
        ld.chunk = 0;
        ld.set_tile(a, list, count, nslots);
        if constexpr (X8) ld.set_x_tile(a, list, count, nslots);
        else if (a.K < kSlotK) ld.toggle_half();
        ld.issue_scales();
        ld.template issue_some<0, X8 ? 8 : 16>(0);
        if constexpr (X8) ld.template issue_x<0, 0, 8>();
        ld.advance(a, list, count, nslots);
        if constexpr (X8) ld.template issue_x<1, 0, 8>();
        ld.template issue_some<0, X8 ? 4 : kLoads3b>(1);
        slot_barrier<0>();
        uint32_t b = 0, scales = 0;
        for (int e = 0; e < count; ++e) {
            const Tile t = list.at(e);
            // a group's last tile runs at the smallest of three heights that holds its rows
            const int rows = t.r1 - t.r0;
            if (rows > 128) tile_product<X8, 4, F32OUT>(ld, a, lds, list, count, t, l, nslots, b, scales);
            else if (rows > 64) tile_product<X8, 2, F32OUT>(ld, a, lds, list, count, t, l, nslots, b, scales);
            else tile_product<X8, 1, F32OUT>(ld, a, lds, list, count, t, l, nslots, b, scales);
        }
        slot_barrier<0>();                               // the loads past the end land before the LDS goes away
    }

    // rows past the last end: zeros
    const int64_t per_row = (int64_t)a.N * (F32OUT ? 4 : 2) / 16;
    uint4* y = (uint4*)a.y + (int64_t)rows_end * per_row;
    const int64_t total = (int64_t)(a.M - rows_end) * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads)
        y[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

hipError_t launch_mxfp4_mm_tile(const void* xq, const void* xs, bool x8, int64_t ldx, int64_t ldxs, const void* wq,
                                const void* wsc, const int32_t* offs, int M, int N, int K, int G, void* y, bool f32_out,
                                hipStream_t stream)
{
    int device = 0, cus = 0;
    hipError_t e = hipGetDevice(&device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (e != hipSuccess) return e;
    const int64_t cols = (N + kCols - 1) / kCols;
    const auto tiles = [&](int rows) { return (((int64_t)M + rows - 1) / rows + G) * cols; };   // at most
    const int rows = tiles(256) >= kManyTiles * cus ? 256 : 128;
    // One workgroup a CU, fewer when there are not that many tiles, a multiple of it (which
    // then run one after the other) when a workgroup's list would not hold its tiles: it
    // has at most (most + 8) / grid + 1.
    const int64_t most = tiles(rows), parts = most * (rows / 64);
    int64_t grid = parts < cus ? parts : cus;
    grid *= (most + kXcds + grid * (kMaxEntries - 1) - 1) / (grid * (kMaxEntries - 1));
    grid = (grid + kXcds - 1) / kXcds * kXcds;
    const MmArgs a = {(const uint8_t*)xq, (const uint8_t*)xs, (const uint8_t*)wq, (const uint8_t*)wsc, offs, y,
                      (uint32_t)ldx, (uint32_t)ldxs, M, N, K, G, rows};
#define MXQ_LAUNCH(X8, F) \
    hipLaunchKernelGGL((mxfp4_mm_tile_kernel<X8, F>), dim3((unsigned)grid), dim3(kThreads), 0, stream, a)
    if (x8 && f32_out) MXQ_LAUNCH(true, true);
    else if (x8) MXQ_LAUNCH(true, false);
    else if (f32_out) MXQ_LAUNCH(false, true);
    else MXQ_LAUNCH(false, false);
#undef MXQ_LAUNCH
    return hipGetLastError();
}

}  // namespace mxq
