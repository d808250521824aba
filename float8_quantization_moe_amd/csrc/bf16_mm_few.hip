// bf16_mm_few.hip -- the products of bf16_mm.hip for few token rows and for small results.
//
// Y and dX, few rows.  The weights' bytes are the cost and each is used once or a few times, so nothing is shared
// between waves: a workgroup takes 64 columns of results by 16 TB rows of one group, its four
// waves a quarter of the sum each.  A wave has a ring of two steps of its own in LDS (64 values of
// the sum: 8 KB of weights, 2 KB a 16 rows of tokens), filled by buffer-load-to-LDS in whole
// 128-byte lines, and waits for its own loads only.  The waves' sums are added in LDS in order:
// one launch, no workspace.
//
// dW, small results.  The same with 64 x 64 results a workgroup, whose sum runs over the group's
// rows: both operands run across it.
//
// Weights whose memory rows run along the sum (Y) are read 16 bytes a lane, those that run across
// it (dX) with the transposing LDS read; MFMA operands as in bf16_mm.hip.
//
// 8 rows over 16 experts of 8192 x 5120, six of them with rows: 84 us for 503 MB, 6.0 TB/s (a ring
// shared by the four waves and its barriers 99).  Against the tile kernel: few_rows() in bf16_mm.hip.
#include "device_common.hpp"
#include "internal.hpp"
#include "mm_tile.hpp"

#include "../../include/mxq.h"

namespace mxq {

namespace {

constexpr int kThreads = kTileThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kCols = 64;                                // columns of a workgroup
constexpr int kStepK = 64;
constexpr uint32_t kABytes = 8192;                       // weights of one step

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i* LdsV4i;
typedef __attribute__((address_space(3))) v4f* LdsV4f;
typedef __attribute__((address_space(3))) v4s* LdsV4s;

struct FewArgs {
    const uint16_t *w, *rows;                            // W or X; X or dY
    const int32_t* offs;
    void* out;                                           // split > 1: the parts, fp32
    int M, N, K, G;
    int split;                                           // workgroups that share a sum (dW: 1)
    int add;                                             // dW: added to what out holds
};

// Rows of one workgroup.
struct Chunk {
    int g, r0, r1;                                       // g < 0: none
    int rows_end;                                        // the last group's clamped end
};

// Chunk `want` of the groups' rows, `height` rows at most each, in the groups' order.  By one wave.
__device__ __forceinline__ Chunk find_chunk(const FewArgs& a, int want, int height)
{
    const int lane = lane_id();
    Chunk c = {-1, 0, 0, 0};
    int seen = 0;
    for (int base = 0; base < a.G; base += 64) {
        int e = base + lane < a.G ? a.offs[base + lane] : 0;
        e = wave_incl_max_dpp(e > 0 ? e : 0);
        e = e > c.rows_end ? e : c.rows_end;
        e = e < a.M ? e : a.M;
        const int up = __shfl_up(e, 1, 64), start = lane ? up : c.rows_end;
        const int n = (e - start + height - 1) / height, upto = wave_incl_sum(n) + seen;
        const uint64_t hit = __ballot(upto > want);
        if (c.g < 0 && hit) {
            const int l = __builtin_ctzll(hit);
            c.g = base + l;
            c.r0 = readlane(start, l) + (want - readlane(upto - n, l)) * height;
            c.r1 = readlane(e, l);
            c.r1 = c.r0 + height < c.r1 ? c.r0 + height : c.r1;
        }
        c.rows_end = readlane(e, 63);
        seen = readlane(upto, 63);
    }
    return c;
}

// Rows [r0, r1) of group g.  By one wave.
__device__ __forceinline__ Chunk rows_of_group(const FewArgs& a, int g)
{
    const int lane = lane_id();
    Chunk c = {g, 0, 0, 0};
    for (int base = 0; base <= g; base += 64) {
        int e = base + lane < a.G ? a.offs[base + lane] : 0;
        e = wave_incl_max_dpp(e > 0 ? e : 0);
        e = e > c.rows_end ? e : c.rows_end;
        e = e < a.M ? e : a.M;
        if (g < base + 64) {
            c.r0 = g > base ? readlane(e, g - base - 1) : c.rows_end;
            c.r1 = readlane(e, g - base);
        }
        c.rows_end = readlane(e, 63);
    }
    return c;
}

// The wave's loads and all before them but the last N have landed.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_reads()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// P: an mxq_product.  TB: 16-row parts (dW: 4, of 64 columns of dY).
template <int P, int TB, bool F32OUT>
__global__ __launch_bounds__(kThreads)
void bf16_mm_few_kernel(const FewArgs a)
{
    constexpr bool ACROSS = P != MXQ_PRODUCT_Y, DW = P == MXQ_PRODUCT_DW;   // the operands that run across the sum
    constexpr int kLoads = 8 + 2 * TB;                   // of a step
    constexpr uint32_t kStepBytes = kABytes + 2048u * TB;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves * 2 * kStepBytes];
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    const int ntiles = (a.N + 16 * TB - 1) / (16 * TB);  // (dW's)
    const Chunk c = DW ? rows_of_group(a, (int)blockIdx.y / ntiles) : find_chunk(a, (int)blockIdx.y, 16 * TB);
    const int cols = ACROSS ? a.K : a.N, depth = DW ? c.r1 - c.r0 : ACROSS ? a.N : a.K;
    // "Across", a memory row's 128 bytes may end inside a line, and the next ones are the next
    // workgroup's: four neighbours share an XCD (workgroup index mod 8).  16 experts of 8192 x 5120, 16
    // rows: 141 -> 127 us; 7 of 3168 x 3160: 28 -> 23; 4 of 4096 x 4096: 18.6 -> 19.4.
    constexpr int kNear = 4, kRound = 8 * kNear;
    const int at = (int)blockIdx.x % kRound, round = (int)blockIdx.x - at;
    const int c0 = (ACROSS && round + kRound <= (int)gridDim.x ? round + at % 8 * kNear + at / 8 : (int)blockIdx.x) * kCols;

    // the result's rows: those of this workgroup from `first`, `rows` of them
    const int64_t first = DW ? (int64_t)c.g * a.N + (int)blockIdx.y % ntiles * 16 * TB : c.r0;
    const int n0 = DW ? (int)blockIdx.y % ntiles * 16 * TB : 0;
    const int rows = !DW ? c.r1 - c.r0 : a.N - n0 < 16 * TB ? a.N - n0 : 16 * TB;
    uint8_t* out = (uint8_t*)a.out + (DW ? 0 : (int64_t)blockIdx.z * a.M * cols * (F32OUT ? 4 : 2));
    if (DW && a.add && depth == 0) return;               // nothing to add: nothing is touched

    if (!DW && blockIdx.y == 0) {                        // rows past the last end: zeros
        constexpr int kPer = F32OUT ? 4 : 8;             // values of 16 bytes
        const int width = (cols - c0 < kCols ? cols - c0 : kCols) / kPer;
        for (int i = (int)threadIdx.x; i < (a.M - c.rows_end) * width; i += kThreads)
            ((uint4*)out)[((int64_t)(c.rows_end + i / width) * cols + c0) / kPer + i % width] = make_uint4(0, 0, 0, 0);
    }
    if (c.g < 0) return;

    // this wave's steps of the sum, and the resources at the first
    const int steps = (depth + kStepK - 1) / kStepK;
    const int pieces = DW ? kWaves : kWaves * a.split, piece = DW ? wave : kWaves * (int)blockIdx.z + wave;
    const int s0 = (int)((int64_t)steps * piece / pieces), s1 = (int)((int64_t)steps * (piece + 1) / pieces);
    const uint32_t lda = 2u * (uint32_t)a.K, ldb = 2u * (uint32_t)(DW ? a.N : depth);
    const int width = cols - c0 < kCols ? cols - c0 : kCols;
    const uint16_t* wbase = a.w + (DW ? (int64_t)c.r0 : (int64_t)c.g * a.N + (ACROSS ? 0 : c0)) * a.K + (ACROSS ? c0 : 0);
    const uint16_t* rbase = a.rows + (int64_t)c.r0 * (DW ? a.N : depth) + n0;

    // Lane offsets.  LDS rows of 128 bytes: "along" and the tokens', their 16-byte chunks at
    // c ^ ((row >> 1) & 7); "across", their 32-byte parts at p ^ (row & 3).  Load i is rows
    // 8i .. 8i + 7, so both swizzles repeat every second load.
    uint32_t along[2], tail[2], part[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t row = 8u * i + ((uint32_t)lane >> 3);
        const uint32_t chunk = ((uint32_t)lane & 7u) ^ ((row >> 1) & 7u);
        along[i] = 16u * chunk;
        tail[i] = depth % kStepK != 0 && chunk >= (uint32_t)(depth % kStepK) / 8u ? 0x80000000u : 0u;
        part[i] = 32u * ((((uint32_t)lane >> 1) & 3u) ^ (row & 3u)) + 16u * ((uint32_t)lane & 1u);
    }
    const uint32_t my = (uint32_t)uniform((int)((uint32_t)(uintptr_t)(LdsPtr)lds + (uint32_t)wave * 2u * kStepBytes));
    // A step into ring slot s & 1; past the wave's last one it loads nothing.
    const auto issue = [&](int s) {
        const uint32_t to = my + (uint32_t)((s - s0) & 1) * kStepBytes;
        const bool some = s < s1, last = s == steps - 1;
        const int k = s * kStepK;
        const int n = depth - k < kStepK ? depth - k : kStepK;
        const v4i ra = resource(ACROSS ? wbase + (int64_t)k * a.K : wbase + k,
                                !some ? 0u : ACROSS ? (uint32_t)n * lda - 2u * (uint32_t)c0 : (uint32_t)width * lda - 2u * (uint32_t)k);
        const v4i rb = resource(DW ? rbase + (int64_t)k * a.N : rbase + k,
                                !some ? 0u : DW ? (uint32_t)n * ldb - 2u * (uint32_t)n0 : (uint32_t)rows * ldb - 2u * (uint32_t)k);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t off = (8u * i + ((uint32_t)lane >> 3)) * lda;
            load_to_lds<3>(ra, to + 1024u * i, ACROSS ? off + part[i & 1] : (off + along[i & 1]) | (last ? tail[i & 1] : 0u));
        }
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i)
        {
            const uint32_t off = (8u * i + ((uint32_t)lane >> 3)) * ldb;
            load_to_lds<3>(rb, to + kABytes + 1024u * i, DW ? off + part[i & 1] : (off + along[i & 1]) | (last ? tail[i & 1] : 0u));
        }
    };

    v4f acc[4][TB];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = v4f{};
    const uint32_t r = (uint32_t)lane & 15u, q = (uint32_t)lane >> 4, sub = (r >> 2) & 3u;
    if (s0 < s1) {
        issue(s0);
        issue(s0 + 1);
    }
    for (int s = s0; s < s1; ++s) {
        const uint32_t slot = my + (uint32_t)((s - s0) & 1) * kStepBytes;
        wait_loads<kLoads>();                            // (newer: the next step)
        v4i fa[2][4], fb[2][TB];
        // Part i of an operand at `base`, half h of the step: "across", rows 32h + 8q + sub and four on,
        // columns 16i + 4 (r % 4) ..
        const auto read = [&](uint32_t base, bool across, int h, int i) {
            if (!across) return *(LdsV4i)(uintptr_t)(base + (16u * i + r) * 128u + (((4u * h + q) ^ ((r >> 1) & 7u)) << 4));
            const uint32_t at = base + (32u * h + 8u * q + sub) * 128u + (((uint32_t)i ^ sub) << 5) + 8u * (r & 3u);
            const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4s)(uintptr_t)at));
            const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV4s)(uintptr_t)(at + 512u)));
            return v4i{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {                    // 32 values of the sum
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[h][i] = read(slot, ACROSS, h, i);
#pragma unroll
            for (int j = 0; j < TB; ++j) fb[h][j] = read(slot + kABytes, DW, h, j);
        }
        wait_reads();
        issue(s + 2);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, fa[h][i]),
                                                                        __builtin_bit_cast(v8bf, fb[h][j]), acc[i][j], 0, 0, 0);
    }
    wait_loads<0>();                                     // (the loads past the end, before the ring is used again)

    // the waves' sums: wave i adds part i of all of them
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) *(LdsV4f)(uintptr_t)(my + (uint32_t)(i * TB + j) * 1024u + 16u * (uint32_t)lane) = acc[i][j];
    __syncthreads();
    const uint32_t base = (uint32_t)(uintptr_t)(LdsPtr)lds;
    const int col = c0 + 16 * wave + 4 * (int)q;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        v4f sum = {};
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            sum += *(LdsV4f)(uintptr_t)(base + (uint32_t)w * 2u * kStepBytes + (uint32_t)(wave * TB + j) * 1024u + 16u * (uint32_t)lane);
        const int row = 16 * j + (int)r;
        if (row < rows && col < cols) {
            const int64_t at = (first + row) * cols + col;
            if constexpr (F32OUT) {
                if (DW && a.add) sum = *(const v4f*)((float*)out + at) + sum;
                *(v4f*)((float*)out + at) = sum;
            }
            else *(uint2*)((uint16_t*)out + at) = make_uint2(f32_pair_to_bf16(sum[0], sum[1]), f32_pair_to_bf16(sum[2], sum[3]));
        }
    }
}

}  // namespace

// 16-row parts of a workgroup.
static int few_parts(int product, int M, int G)
{
    const int groups = G < M ? G : M;
    return product == MXQ_PRODUCT_DW ? 4 : M <= 16 ? 1 : M <= 32 * groups ? 2 : 4;
}
static int64_t few_groups(int product, int64_t M, int64_t N, int64_t K, int64_t G, dim3* grid)
{
    const int64_t height = 16 * few_parts(product, (int)M, (int)G);
    const int64_t x = ((product == MXQ_PRODUCT_Y ? N : K) + kCols - 1) / kCols;
    const int64_t y = product == MXQ_PRODUCT_DW ? G * ((N + height - 1) / height) : (M + height - 1) / height + (G < M ? G : M) - 1;
    *grid = dim3((unsigned)x, (unsigned)y);
    return x * y;
}

// Workgroups that share a sum, and then a second launch that adds the parts: where there are few and
// their waves' sums are long (142 rows x 6416 x 552, dX 33 -> 15 us; one row 13 -> 9; 142 rows x 512 x
// 4096 over 8 experts, Y, sums of 64 steps, 12 -> 15).  dW's sums are not long here: 2048 rows a group
// on average, see few_rows().
int bf16_mm_few_split(int product, int M, int N, int K, int G)
{
    if (product == MXQ_PRODUCT_DW) return 1;
    dim3 grid;
    const int64_t groups = few_groups(product, M, N, K, G, &grid);
    const int steps = ((product == MXQ_PRODUCT_DX ? N : K) + kStepK - 1) / kStepK;
    if (groups > 128 || steps < 20 * kWaves) return 1;
    int64_t split = 512 / groups;
    if (split > steps / (3 * kWaves)) split = steps / (3 * kWaves);
    return (int)(split < 16 ? split : 16);
}

hipError_t launch_bf16_mm_few(int product, const void* rows, const void* w, const int32_t* offs, int M, int N, int K, int G,
                              int split, void* out, bool f32_out, bool add, hipStream_t stream)
{
    const FewArgs a = {(const uint16_t*)w, (const uint16_t*)rows, offs, out, M, N, K, G, split, add};
    const int parts = few_parts(product, M, G);
    dim3 grid;
    few_groups(product, M, N, K, G, &grid);
    grid.z = (unsigned)split;
#define MXQ_LAUNCH(P, T)                                                                                               \
    do {                                                                                                               \
        if (f32_out) hipLaunchKernelGGL((bf16_mm_few_kernel<P, T, true>), grid, dim3(kThreads), 0, stream, a);         \
        else hipLaunchKernelGGL((bf16_mm_few_kernel<P, T, false>), grid, dim3(kThreads), 0, stream, a);                \
    } while (0)
    if (product == MXQ_PRODUCT_DW) MXQ_LAUNCH(MXQ_PRODUCT_DW, 4);
    else if (product == MXQ_PRODUCT_DX && parts == 1) MXQ_LAUNCH(MXQ_PRODUCT_DX, 1);
    else if (product == MXQ_PRODUCT_DX && parts == 2) MXQ_LAUNCH(MXQ_PRODUCT_DX, 2);
    else if (product == MXQ_PRODUCT_DX) MXQ_LAUNCH(MXQ_PRODUCT_DX, 4);
    else if (parts == 1) MXQ_LAUNCH(MXQ_PRODUCT_Y, 1);
    else if (parts == 2) MXQ_LAUNCH(MXQ_PRODUCT_Y, 2);
    else MXQ_LAUNCH(MXQ_PRODUCT_Y, 4);
#undef MXQ_LAUNCH
    return hipGetLastError();
}

}  // namespace mxq
