// mxfp4_mm_tile.hip -- the product of MXFP8 or MXFP4 token rows with MXFP4 expert
// weights for groups of many rows (mxfp4_mm.hip states the operation and takes the
// calls with few rows).
//
// Persistent workgroups (one a CU, 4 waves in 2 x 2) walk over output tiles of 256
// columns x R rows: R = 256 for E2M1 tokens, 128 for E4M3 tokens, whose codes take
// twice the space and whose MFMA takes twice the time, so that the K loop has one
// shape for both.  K advances 256 values a slot through a 2-slot LDS ring of 32 KB
// of W and 32 KB of X codes and 16 bytes of scales a row, filled by
// buffer-load-to-LDS in whole 128-byte lines.  A slot is four MFMA steps of 64 k; a
// step's operands are read from LDS during the step before it.  The one barrier that
// a slot needs comes before its last step, when all its operands are in registers:
// the loads of the slot after next go into its place from there on, spread between
// the MFMAs of three steps.
//
// The slots of successive tiles form one stream: the loads run ahead of the
// products across the end of a tile, so the next tile's operands arrive while this
// one's results are stored (straight from the accumulators: the LDS belongs to the
// next tile by then).  One workgroup a CU leaves nothing else to hide them.
//
// Tile list: row tiles never straddle a group.  Group by group, inside a group in
// blocks of kColBlock column tiles with the block's row tiles consecutive, so that
// neighbours in the list share W and X tiles; each of the 8 XCDs (workgroup index
// mod 8) walks one contiguous stretch, its CUs side by side.  Every workgroup finds
// its own tiles from the group offsets (a scan in LDS), so no launch comes before.
//
// MFMA operand A is W (output columns), B is X (token rows).  In a 64-k step, lane
// (r, h) = (lane % 32, lane / 32) holds of row r: E2M1, the 16 bytes of scale block
// h; E4M3, the 16-byte chunks h and h + 2.  Its scale byte is that of block h.
#include "device_common.hpp"
#include "internal.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 256;                               // columns of a tile
constexpr int kSlotK = 256;
constexpr uint32_t kOperandBytes = 32 * 1024;            // codes of one operand in one slot
constexpr uint32_t kSlotBytes = 2 * kOperandBytes;
constexpr uint32_t kScaleOperand = 256 * 16;             // scales of one operand in one slot
constexpr uint32_t kScaleBase = 2 * kSlotBytes;
constexpr uint32_t kEntryBase = kScaleBase + 2 * 2 * kScaleOperand;
constexpr int kMaxEntries = 1024;                        // tiles of one workgroup
constexpr uint32_t kLdsBytes = kEntryBase + kMaxEntries * 16;
static_assert(kLdsBytes <= 160 * 1024, "LDS of a CU");
constexpr int kColBlock = 4;                             // column tiles of a block of the tile order
constexpr int kXcds = 8;
constexpr int kMaxGroups = 4095;
static_assert((2 * (kMaxGroups + 2) + kThreads) * 4 <= (int)kScaleBase, "the scan's arrays fit the ring");

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t* LdsPtr;

struct Tile {
    int g, r0, r1, c;                                    // group, rows [r0, r1), column tile c
};

struct MmArgs {
    const uint8_t *xq, *xs, *wq, *ws;
    const int32_t* offs;
    void* y;
    uint32_t ldx, ldxs;
    int M, N, K, G;
};

template <bool X8>
constexpr int tile_rows() { return X8 ? 128 : 256; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Buffer resource: base, stride 0, size in bytes (loads past it return zeros).
__device__ __forceinline__ v4i resource(const void* base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    v4i r = {uniform((int)(uint32_t)b), uniform((int)(uint32_t)(b >> 32)), uniform((int)bytes), 0x00020000};
    return r;
}

// Buffer load straight into LDS: lane l's 16 bytes land at lds + 16 l.  Counted by
// vmcnt, which slot_barrier waits on; in asm so that the compiler adds no wait of
// its own before later LDS reads.
__device__ __forceinline__ void load_to_lds(const v4i& srd, uint32_t lds, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(srd)
                 : "memory");
}

// Every load of this wave has landed and its LDS reads are done; then meet the
// other waves.
__device__ __forceinline__ void slot_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// -------------------------------------------------------------- tile list ---
// Inclusive scan over the workgroup's threads (maximum or sum) through sh.
template <bool MAX>
__device__ int block_scan(int v, int* sh)
{
    const int t = (int)threadIdx.x;
    v = MAX ? wave_incl_max(v) : wave_incl_sum(v);
    if ((t & 63) == 63) sh[t >> 6] = v;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < (t >> 6); ++w) before = MAX ? (sh[w] > before ? sh[w] : before) : before + sh[w];
    __syncthreads();
    return MAX ? (v > before ? v : before) : v + before;
}

// Fills `list` with this workgroup's tiles and returns their number; *rows_end is
// the last group's clamped end.  end_sh: the groups' clamped ends; first_sh: each
// group's first row tile.
template <int R>
__device__ int make_list(const MmArgs& a, int* end_sh, int* first_sh, int* scan_sh, Tile* list, int* rows_end)
{
    const int t = (int)threadIdx.x;
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
    const int q = (V + kXcds - 1) / kXcds;
    const int x = (int)blockIdx.x % kXcds, stride = (int)gridDim.x / kXcds;
    const int lo = x * q + (int)blockIdx.x / kXcds, hi = (x + 1) * q < V ? (x + 1) * q : V;
    const int count = lo < hi ? (hi - lo + stride - 1) / stride : 0;
    for (int j = t; j < count && j < kMaxEntries; j += kThreads) {
        const int L = lo + j * stride;
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
        Tile tl;
        tl.g = p;
        tl.r0 = (p ? end_sh[p - 1] : 0) + rem / width * R;
        tl.r1 = tl.r0 + R < end_sh[p] ? tl.r0 + R : end_sh[p];
        tl.c = cb * kColBlock + rem % width;
        list[j] = tl;
    }
    *rows_end = end_sh[a.G - 1];
    return count < kMaxEntries ? count : kMaxEntries;
}

// ------------------------------------------------------------------ loads ---
// The stream of slots to load: the current tile's resources and its next slot.
// LDS rows of 128 bytes hold their eight 16-byte chunks at c ^ ((row >> 1) & 7),
// rows of 256 bytes (E4M3) their sixteen at c ^ (row & 15): the 16 lanes that a
// 128-bit LDS read serves at a time then meet 16 different bank groups.  The
// swizzle is applied to the source offsets (the LDS side is linear in the lane).
template <bool X8>
struct Loader {
    v4i w, x, ws, xs;                                    // resources that start at the next slot
    uint32_t off_w[8], off_x[8], off_ws, off_xs;         // lane offsets of the wave's loads
    uint32_t lds_data, lds_ws, lds_xs;                   // LDS addresses of the wave's part of ring slot 0
    uint32_t upper;                                      // bit 31: this lane's chunk of load 0 is in the second half of a row's slot
    int entry, left;                                     // the tile's place in the list; its slots from the next one on
    static constexpr int kXStep = X8 ? 256 : 128;        // bytes of an X row in a slot

    __device__ __forceinline__ void set_lanes(const MmArgs& a, const uint8_t* lds, int wave, int lane)
    {
        const uint32_t half = (uint32_t)a.K / 2u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t row = (uint32_t)(64 * wave + 8 * i + (lane >> 3));        // 8 rows of 128 bytes a load
            const uint32_t chunk = ((uint32_t)lane & 7u) ^ ((row >> 1) & 7u);
            off_w[i] = row * half + 16u * chunk;
            if constexpr (X8) {
                const uint32_t xrow = (uint32_t)(32 * wave + 4 * i + (lane >> 4));   // 4 rows of 256 bytes a load
                off_x[i] = xrow * a.ldx + 16u * (((uint32_t)lane & 15u) ^ (xrow & 15u));
            } else {
                off_x[i] = row * a.ldx + 16u * chunk;
            }
        }
        const int xw = X8 ? wave & 1 : wave;             // 128 rows: two waves bring the same scales
        upper = ((uint32_t)lane >> (X8 ? 3 : 2)) << 31;
        off_ws = (uint32_t)(64 * wave + lane) * ((uint32_t)a.K / 32u);
        off_xs = (uint32_t)(64 * xw + lane) * a.ldxs;
        const uint32_t base = (uint32_t)uniform((int)(uint32_t)(uintptr_t)(LdsPtr)lds);
        lds_data = base + 8192u * (uint32_t)wave;
        lds_ws = base + kScaleBase + 1024u * (uint32_t)wave;
        lds_xs = base + kScaleBase + kScaleOperand + 1024u * (uint32_t)xw;
    }

    // The first slot of tile `entry` of the list; past its end, loads of nothing.
    __device__ __forceinline__ void set_tile(const MmArgs& a, const Tile* list, int e, int count, int nslots)
    {
        left = nslots;
        const uint32_t half = (uint32_t)a.K / 2u, kb = (uint32_t)a.K / 32u;
        const bool some = e < count;
        const Tile t = list[some ? e : 0];
        const int g = some ? uniform(t.g) : 0, r0 = some ? uniform(t.r0) : 0;
        const uint32_t nx = some ? (uint32_t)(uniform(t.r1) - r0) : 1u;
        const int n0 = some ? uniform(t.c) * kCols : 0;
        const uint32_t nw = (uint32_t)(a.N - n0 < kCols ? a.N - n0 : kCols);
        const int64_t wrow = (int64_t)g * a.N + n0;
        w = resource(a.wq + wrow * half, some ? nw * half : 0u);
        ws = resource(a.ws + wrow * kb, some ? nw * kb : 0u);
        x = resource(a.xq + (int64_t)r0 * a.ldx, some ? (nx - 1u) * a.ldx + (X8 ? (uint32_t)a.K : half) : 0u);
        xs = resource(a.xs + (int64_t)r0 * a.ldxs, some ? (nx - 1u) * a.ldxs + kb : 0u);
    }

    static __device__ __forceinline__ void step(v4i& r, uint32_t bytes)
    {
        const uint64_t base = (((uint64_t)(uint32_t)r.y << 32) | (uint32_t)r.x) + bytes;
        const uint32_t left = (uint32_t)r.z;
        r.x = uniform((int)(uint32_t)base);              // (resources stay in scalar registers)
        r.y = uniform((int)(uint32_t)(base >> 32));
        r.z = uniform((int)(left < bytes ? 0u : left - bytes));
    }
    // On to the next slot of the stream.  Where K ends half way through a tile's last
    // slot, that slot's X codes past K are to be zeros: for its loads their lanes'
    // offsets leave the resource (bit 31).
    __device__ __forceinline__ void advance(const MmArgs& a, const Tile* list, int count, int nslots)
    {
        const bool was_last = left == 1;
        if (was_last) {
            set_tile(a, list, ++entry, count, nslots);
        } else {
            --left;
            step(w, 128u);
            step(x, kXStep);
            step(ws, 8u);
            step(xs, 8u);
        }
        if (a.K % kSlotK != 0 && was_last != (left == 1)) toggle_half();
    }
    __device__ __forceinline__ void toggle_half()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) off_x[i] ^= (i & (X8 ? 2 : 1)) ? upper ^ 0x80000000u : upper;
    }

    // Load I (0 .. 17) of the slot into ring slot b.
    template <int I>
    __device__ __forceinline__ void issue(uint32_t b)
    {
        constexpr int i = (I - 2) / 2;
        if constexpr (I == 0) load_to_lds(ws, lds_ws + b * 2u * kScaleOperand, off_ws);
        else if constexpr (I == 1) load_to_lds(xs, lds_xs + b * 2u * kScaleOperand, off_xs);
        else if constexpr (I % 2 == 0) load_to_lds(w, lds_data + b * kSlotBytes + 1024u * i, off_w[i]);
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
    uint32_t row, h, swz, swx;                           // lane % 32, lane / 32, and its rows' swizzles
    uint32_t wn, wm;                                     // the wave's place in the 2 x 2
};

template <bool X8, int TM, int T>
__device__ __forceinline__ void read_step(Operands<X8, TM>& f, const uint8_t* lds, uint32_t b, const Lane& l)
{
    const uint8_t* W = lds + b * kSlotBytes + (128u * l.wn + l.row) * 128u + (((2u * T + l.h) ^ l.swz) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.w[i] = *(const v4i*)(W + 4096 * i);
    if constexpr (X8) {
        const uint8_t* X = lds + b * kSlotBytes + kOperandBytes + (32u * TM * l.wm + l.row) * 256u;
        const uint8_t* X0 = X + (((4u * T + l.h) ^ l.swx) << 4);
        const uint8_t* X1 = X + (((4u * T + 2u + l.h) ^ l.swx) << 4);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            f.x[i][0] = *(const v4i*)(X0 + 8192 * i);
            f.x[i][1] = *(const v4i*)(X1 + 8192 * i);
        }
    } else {
        const uint8_t* X = lds + b * kSlotBytes + kOperandBytes + (32u * TM * l.wm + l.row) * 128u +
                           (((2u * T + l.h) ^ l.swz) << 4);
#pragma unroll
        for (int i = 0; i < TM; ++i) f.x[i][0] = *(const v4i*)(X + 4096 * i);
    }
}

// The scale words of ring slot b, shifted so that bytes 0 and 2 are the lane's blocks.
template <int TM>
__device__ __forceinline__ void read_scales(Scales<TM>& s, const uint8_t* lds, uint32_t b, const Lane& l)
{
    const uint8_t* p = lds + kScaleBase + b * 2u * kScaleOperand;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.w[i] = *(const uint2*)(p + (128u * l.wn + 32u * i + l.row) * 16u);
#pragma unroll
    for (int i = 0; i < TM; ++i) s.x[i] = *(const uint2*)(p + kScaleOperand + (32u * TM * l.wm + 32u * i + l.row) * 16u);
}
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

// Step T's MFMAs, with loads A .. B - 1 of the next slot of the stream into ring
// slot b spread between them.
template <bool X8, int TM, int T, bool ZERO, int A, int B, int I = 0>
__device__ __forceinline__ void mfmas(v16f (&acc)[4][TM], const Operands<X8, TM>& f, const Scales<TM>& s, Loader<X8>& ld,
                                      uint32_t b)
{
    constexpr int n = 4 * TM;
    if constexpr (I < n) {
        mfma<X8, TM, T, ZERO, I>(acc, f, s);
        ld.template issue_some<A + I * (B - A) / n, A + (I + 1) * (B - A) / n>(b);
        if constexpr (A < B) __builtin_amdgcn_sched_barrier(0);
        mfmas<X8, TM, T, ZERO, A, B, I + 1>(acc, f, s, ld, b);
    }
}

// How a slot's loads are spread: the first kLoadsA in the last step of the slot two
// before it, up to kLoadsB in the first step of the slot before it, the rest in the
// second.  All 18 at once fill the memory pipe's queue and hold up the MFMAs behind
// them: 16640 x 8192 x 5120 over 16 groups 723 / 481 us (E4M3 / E2M1 tokens) against
// 658 / 451 in thirds (9 + 9: 662 / 450; 12 + 6: 687 / 466).
constexpr int kLoadsA = 6, kLoadsB = 12, kLoadsC = 18;

// Steps 0 and 1 of the slot in ring slot b, with the second part of the loads of
// the slot after it.  f[0] and s hold (or are being read with) its first step and
// scales; f[1] is left with step 1's successor: f[0] holds step 2.
template <bool X8, int TM, bool FIRST>
__device__ __forceinline__ void steps01(v16f (&acc)[4][TM], Operands<X8, TM> (&f)[2], Scales<TM>& s, Loader<X8>& ld,
                                        const uint8_t* lds, const Lane& l, uint32_t b)
{
    shift_scales<TM>(s, l);
    read_step<X8, TM, 1>(f[1], lds, b, l);
    __builtin_amdgcn_sched_barrier(0);
    mfmas<X8, TM, 0, FIRST, kLoadsA, kLoadsB>(acc, f[0], s, ld, b ^ 1u);
    __builtin_amdgcn_sched_barrier(0);
    read_step<X8, TM, 2>(f[0], lds, b, l);
    __builtin_amdgcn_sched_barrier(0);
    mfmas<X8, TM, 1, false, kLoadsB, kLoadsC>(acc, f[1], s, ld, b ^ 1u);
    __builtin_amdgcn_sched_barrier(0);
}

// Steps 2 and 3, with the barrier between them and the first part of the loads into
// this ring slot; on exit f[0] and s hold the next slot's, unless this is the
// tile's LAST.
template <bool X8, int TM, bool LAST>
__device__ __forceinline__ void steps23(v16f (&acc)[4][TM], Operands<X8, TM> (&f)[2], Scales<TM>& s, Loader<X8>& ld,
                                        const uint8_t* lds, const Lane& l, uint32_t b)
{
    read_step<X8, TM, 3>(f[1], lds, b, l);
    __builtin_amdgcn_sched_barrier(0);
    mfmas<X8, TM, 2, false, 0, 0>(acc, f[0], s, ld, b);
    slot_barrier();
    const Scales<TM> now = s;
    if constexpr (!LAST) {
        read_step<X8, TM, 0>(f[0], lds, b ^ 1u, l);
        read_scales<TM>(s, lds, b ^ 1u, l);
        __builtin_amdgcn_sched_barrier(0);
    }
    mfmas<X8, TM, 3, false, 0, kLoadsA>(acc, f[1], now, ld, b);
    __builtin_amdgcn_sched_barrier(0);
}

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
// that a lane stores 8 consecutive ones (16 bytes).
template <int TM, bool F32OUT>
__device__ __forceinline__ void store_tile(const v16f (&acc)[4][TM], const MmArgs& a, const Tile& t, const Lane& l)
{
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int m = t.r0 + (int)(32u * TM * l.wm + 32u * j + l.row);
        const bool row_ok = m < t.r1;
        const int64_t at = (int64_t)m * a.N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);           // (one part at a time in VGPRs)
            const int n0 = t.c * kCols + (int)(128u * l.wn) + 32 * i;
            const v16f& v = acc[i][j];
            if constexpr (F32OUT) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = n0 + 8 * q + 4 * (int)l.h;
                    if (row_ok && n < a.N)
                        *(float4*)((float*)a.y + at + n) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const uint32_t e0 = f32_pair_to_bf16(v[4 * q], v[4 * q + 1]), e1 = f32_pair_to_bf16(v[4 * q + 2], v[4 * q + 3]);
                    const uint32_t o0 = f32_pair_to_bf16(v[4 * q + 4], v[4 * q + 5]), o1 = f32_pair_to_bf16(v[4 * q + 6], v[4 * q + 7]);
                    const auto s0 = __builtin_amdgcn_permlane32_swap(e0, o0, false, false);
                    const auto s1 = __builtin_amdgcn_permlane32_swap(e1, o1, false, false);
                    const int n = n0 + 8 * q + 8 * (int)l.h;
                    if (row_ok && n < a.N)
                        *(uint4*)((uint16_t*)a.y + at + n) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
                }
            }
        }
    }
}

// One tile: its slots are the next to come out of the stream, the first of them in
// ring slot b; the loads are part way into the slot after it.
template <bool X8, int TM, bool F32OUT>
__device__ __forceinline__ void tile_product(Loader<X8>& ld, const MmArgs& a, const uint8_t* lds, const Tile* list, int count,
                                             const Tile& t, const Lane& l, int nslots, uint32_t& b)
{
    v16f acc[4][TM];
    Operands<X8, TM> f[2];
    Scales<TM> s;
    read_scales<TM>(s, lds, b, l);
    read_step<X8, TM, 0>(f[0], lds, b, l);
    steps01<X8, TM, true>(acc, f, s, ld, lds, l, b);
    pin<TM>(acc);
    ld.advance(a, list, count, nslots);
    for (int i = 1; i < nslots; ++i) {
        steps23<X8, TM, false>(acc, f, s, ld, lds, l, b);
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
    steps23<X8, TM, true>(acc, f, s, ld, lds, l, b);
    pin<TM>(acc);
    b ^= 1u;
    store_tile<TM, F32OUT>(acc, a, t, l);
}

template <bool X8, bool F32OUT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mxfp4_mm_tile_kernel(const MmArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLdsBytes];
    constexpr int R = tile_rows<X8>();
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    Tile* list = (Tile*)(lds + kEntryBase);
    int rows_end;
    int count;
    {
        int* end_sh = (int*)lds;
        int* first_sh = end_sh + kMaxGroups + 1;
        int* scan_sh = first_sh + kMaxGroups + 1;
        count = uniform(make_list<R>(a, end_sh, first_sh, scan_sh, list, &rows_end));
        rows_end = uniform(rows_end);
    }
    __syncthreads();                                     // the list is complete, the scan's arrays are free

    if (count > 0) {
        const Lane l = {(uint32_t)(lane & 31), (uint32_t)(lane >> 5), (uint32_t)((lane >> 1) & 7), (uint32_t)(lane & 15),
                        (uint32_t)(wave >> 1), (uint32_t)(wave & 1)};
        const int nslots = (a.K + kSlotK - 1) / kSlotK;
        Loader<X8> ld;
        ld.set_lanes(a, lds, wave, lane);
        ld.entry = 0;
        ld.set_tile(a, list, 0, count, nslots);
        if (a.K < kSlotK) ld.toggle_half();
        ld.template issue_some<0, kLoadsC>(0);
        ld.advance(a, list, count, nslots);
        ld.template issue_some<0, kLoadsA>(1);
        slot_barrier();
        uint32_t b = 0;
        for (int e = 0; e < count; ++e) {
            Tile t = list[e];
            t.g = uniform(t.g);
            t.r0 = uniform(t.r0);
            t.r1 = uniform(t.r1);
            t.c = uniform(t.c);
            // a group's last tile runs at the smallest of its heights that holds its rows
            const int rows = t.r1 - t.r0;
            if (rows > R / 2) tile_product<X8, R / 64, F32OUT>(ld, a, lds, list, count, t, l, nslots, b);
            else if (X8 || rows > R / 4) tile_product<X8, R / 128, F32OUT>(ld, a, lds, list, count, t, l, nslots, b);
            else tile_product<X8, 1, F32OUT>(ld, a, lds, list, count, t, l, nslots, b);
        }
        slot_barrier();                                  // the loads past the end land before the LDS goes away
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
    const MmArgs a = {(const uint8_t*)xq, (const uint8_t*)xs, (const uint8_t*)wq, (const uint8_t*)wsc, offs, y,
                      (uint32_t)ldx, (uint32_t)ldxs, M, N, K, G};
    int device = 0, cus = 0;
    hipError_t e = hipGetDevice(&device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (e != hipSuccess) return e;
    // One workgroup a CU, fewer when there are not that many tiles, more (which then run one
    // after the other) when a workgroup's list would not hold its tiles.
    const int rows = x8 ? tile_rows<true>() : tile_rows<false>();
    const int64_t most = (((int64_t)M + rows - 1) / rows + G) * ((N + kCols - 1) / kCols);
    int64_t grid = most < cus ? most : cus;
    const int64_t least = (most + kMaxEntries - kXcds - 1) / (kMaxEntries - kXcds);
    grid = grid < least ? least : grid;
    grid = (grid + kXcds - 1) / kXcds * kXcds;
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
