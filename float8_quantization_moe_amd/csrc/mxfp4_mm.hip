// mxfp4_mm.hip -- grouped product of MXFP8 or MXFP4 token rows with MXFP4 expert
// weights on the gfx950 scaled matrix cores.
//
// Y[m, :] = X[m, :] W_g^T for the token rows m of group g.  Every value is its
// code times its block's power of two: X holds E4M3 codes (as mxq_quantize_mx
// writes) or E2M1 codes (mxq_quantize_mxfp4), W_g E2M1 codes, blocks of 32 along
// K.  v_mfma_scale_f32_*_f8f6f4 takes the formats of its two operands separately
// and the E8M0 scales as operands, so nothing is decoded in software; sums are
// fp32, the result is rounded once to the output type.
#include "device_common.hpp"
#include "internal.hpp"

namespace mxq {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u_dword __attribute__((ext_vector_type(4), aligned(4)));   // 16 bytes at a multiple of 4

// From this many rows on the tile kernel takes a call.  This kernel passes over a group's
// weights once for every 16 rows, so the largest group would decide, but its rows are known
// on the device only: the rule goes by all rows, and a call whose rows are mostly one
// group's takes longer here than it need.  The tile kernel takes 10 us and more however few
// the rows, which counts where the experts are small.
// Measured (uneven groups; MXFP8 tokens, this kernel / the tile kernel, us):
//   8192 x 5120   1 group, 64 rows 25 / 25, 96 rows 37 / 25; 16 groups, 96 rows 73 / 77, 128 rows 84 / 77
//   4096 x 4096   4 groups, 72 rows 19 / 23, 100 rows 23 / 23; 8 groups, 72 rows 24 / 24
//   2048 x 2048   2 groups, 64 rows 9.6 / 14.4, 100 rows 13.9 / 14.7; 32 groups, 128 rows 16.6 / 16.3
//   1736 x 1408   16 groups, 168 rows 9.8 / 12.6, 256 rows 13.0 / 12.9
//   1024 x 2048   64 groups, 200 rows 15.0 / 16.2, 300 rows 19.8 / 18.6
//   1024 x 1024   1 group, 64 rows 8.3 / 10.8, 128 rows 13.8 / 11.2
int64_t many_rows(int64_t N, int64_t K, int64_t G)
{
    return 80 + (N * K >= (int64_t)1 << 22 ? G / 2 : 12 * G < 176 ? 12 * G : 176);
}
constexpr int kTN = 2, kTM = 1;       // 32 columns x 16 rows a workgroup: 24.4 us at 8 rows of 16 groups (16 columns
                                      // 27.7, 64 columns 31 and more; 32 rows 42)
constexpr int kStepK = 128;           // k of one 16x16 MFMA: four scale blocks
constexpr int kChunk = 4;             // steps whose loads go out together
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// ------------------------------------------------------------- few rows ---
// With a few rows a group the weights' bytes are the cost (HBM bound: 8 rows over 16
// experts of 8192 x 5120, six of which have rows, 134 MB in 24.4 us, 5.5 TB/s), and a
// weight is used once: no LDS staging.  A workgroup owns 16 TN columns of one group; its four
// waves split K (one wave alone would leave too few loads in flight) and join their
// sums in LDS in wave order.  A (16 columns of W) and B (16 token rows) go from
// global memory into the MFMA's registers: lane (r, b) = (lane % 16, lane / 16)
// holds row r; of E2M1 the 16 bytes of scale block b of a step, of E4M3 the 16-byte
// chunks b and b + 4.  The loads of the next four steps go out before the MFMAs of
// these.  Groups without rows cost nothing: workgroup y looks for the y-th group
// that has some.

// Rows [r0, r1) of the want-th group (from 0) with rows, and its index; -1 if there
// are not so many, and then r0 is the last group's end.  Ends are the running
// maximum of the offsets, cut to [0, M].  Every lane of the wave must call this.
__device__ __forceinline__ int nth_group(const int32_t* __restrict__ offs, int G, int M, int want, int& r0, int& r1)
{
    int prev = 0, seen = 0;
    for (int base = 0; base < G; base += kWave) {
        const int i = base + lane_id();
        int e = i < G ? offs[i] : 0;
        e = wave_incl_max_dpp(e > prev ? e : prev);
        e = e < M ? e : M;
        // the lane before's end: shifted within 16 lanes, and across their borders
        int start = __builtin_amdgcn_update_dpp(0, e, 0x111, 0xF, 0xF, false);
        const int l = lane_id();
        if (l == 0) start = prev;
        if (l == 16) start = readlane(e, 15);
        if (l == 32) start = readlane(e, 31);
        if (l == 48) start = readlane(e, 47);
        unsigned long long some = __ballot(i < G && e > start);
        const int n = __builtin_popcountll(some);
        if (seen + n > want) {
            for (int k = want - seen; k > 0; --k) some &= some - 1;
            const int at = __builtin_ctzll(some);
            r0 = readlane(start, at);
            r1 = readlane(e, at);
            return base + at;
        }
        seen += n;
        prev = readlane(e, kWave - 1);
    }
    r0 = prev;
    r1 = M;
    return -1;
}

template <bool X8, int TN, int TM>
struct Steps {                                            // the operands of kChunk steps
    uint4 w[kChunk][TN];
    uint4 x[kChunk][TM][X8 ? 2 : 1];
    v4u_dword ws[TN], xs[TM];                             // four blocks' scales a word, a word a step
};

struct FewArgs {
    const uint8_t *xq, *xs, *wq, *ws;
    const int32_t* offs;
    void* y;
    int64_t ldx, ldxs;
    int M, N, K, G;
};

template <bool X8, bool F32OUT, int TN, int TM>
__global__ __launch_bounds__(kThreads)
void mxfp4_mm_few_kernel(const FewArgs a)
{
    __shared__ v4f part[kWaves][TN * TM][kWave];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r = lane & 15, b = lane >> 4;
    int r0, r1;
    const int g = nth_group(a.offs, a.G, a.M, (int)blockIdx.y, r0, r1);
    const int n0 = (int)blockIdx.x * 16 * TN;
    if (g < 0) {
        if (blockIdx.y + 1 < gridDim.y) return;           // fewer groups with rows than workgroups' rows
        // the last row of workgroups: zeros past the last end
        const int cols = (a.N - n0 < 16 * TN ? a.N - n0 : 16 * TN) / 8;
        const int64_t total = (int64_t)(a.M - r0) * cols;
        for (int64_t i = threadIdx.x; i < total; i += kThreads) {
            const int64_t at = ((int64_t)r0 + i / cols) * a.N + n0 + 8 * (i % cols);
            if constexpr (F32OUT) {
                ((uint4*)((float*)a.y + at))[0] = make_uint4(0, 0, 0, 0);
                ((uint4*)((float*)a.y + at))[1] = make_uint4(0, 0, 0, 0);
            } else {
                *(uint4*)((uint16_t*)a.y + at) = make_uint4(0, 0, 0, 0);
            }
        }
        return;
    }

    const int steps = a.K / kStepK;
    const uint8_t *wp[TN], *wsp[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        const int n = n0 + 16 * i + r < a.N ? n0 + 16 * i + r : a.N - 1;       // columns past N: computed, not stored
        const int64_t row = (int64_t)g * a.N + n;
        wp[i] = a.wq + row * (a.K / 2) + 16 * b;
        wsp[i] = a.ws + row * (a.K / 32);
    }
    for (int m0 = r0; m0 < r1; m0 += 16 * TM) {
        const uint8_t *xp[TM], *xsp[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int64_t row = m0 + 16 * j + r < r1 ? m0 + 16 * j + r : r1 - 1;
            xp[j] = a.xq + row * a.ldx + 16 * b;
            xsp[j] = a.xs + row * a.ldxs;
        }
        v4f acc[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

        // Four steps from s on.
        auto load = [&](Steps<X8, TN, TM>& t, int s) {
            const int64_t k = (int64_t)s * kStepK;
#pragma unroll
            for (int u = 0; u < kChunk; ++u) {
#pragma unroll
                for (int i = 0; i < TN; ++i) t.w[u][i] = *(const uint4*)(wp[i] + k / 2 + 64 * u);
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    if constexpr (X8) {
                        t.x[u][j][0] = *(const uint4*)(xp[j] + k + 128 * u);
                        t.x[u][j][1] = *(const uint4*)(xp[j] + k + 128 * u + 64);
                    } else {
                        t.x[u][j][0] = *(const uint4*)(xp[j] + k / 2 + 64 * u);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < TN; ++i) t.ws[i] = *(const v4u_dword*)(wsp[i] + k / 32);
#pragma unroll
            for (int j = 0; j < TM; ++j) t.xs[j] = *(const v4u_dword*)(xsp[j] + k / 32);
        };
        auto multiply = [&](const uint4 (&w)[TN], const uint4 (&x)[TM][X8 ? 2 : 1], const uint32_t (&sw)[TN],
                            const uint32_t (&sx)[TM]) {
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const v8i av = {(int)w[i].x, (int)w[i].y, (int)w[i].z, (int)w[i].w, 0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    v8i bv;
                    if constexpr (X8)
                        bv = v8i{(int)x[j][0].x, (int)x[j][0].y, (int)x[j][0].z, (int)x[j][0].w,
                                 (int)x[j][1].x, (int)x[j][1].y, (int)x[j][1].z, (int)x[j][1].w};
                    else
                        bv = v8i{(int)x[j][0].x, (int)x[j][0].y, (int)x[j][0].z, (int)x[j][0].w, 0, 0, 0, 0};
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[i][j], 4, X8 ? 0 : 4, 0,
                                                                                 (int)(sw[i] >> (8 * b)), 0,
                                                                                 (int)(sx[j] >> (8 * b)));
                }
            }
        };
        // The steps of a chunk but its first `skip`, which an earlier chunk has had.
        auto multiply_chunk = [&](const Steps<X8, TN, TM>& t, int skip) {
#pragma unroll
            for (int u = 0; u < kChunk; ++u) {
                if (u < skip) continue;                   // (uniform)
                uint32_t sw[TN], sx[TM];
#pragma unroll
                for (int i = 0; i < TN; ++i) sw[i] = t.ws[i][u];
#pragma unroll
                for (int j = 0; j < TM; ++j) sx[j] = t.xs[j][u];
                multiply(t.w[u], t.x[u], sw, sx);
            }
        };

        if (steps >= kChunk) {
            // the last chunk starts early enough to end at K
            const int chunks = (steps + kChunk - 1) / kChunk;
            auto first = [&](int c) { return kChunk * c < steps - kChunk ? kChunk * c : steps - kChunk; };
            if (wave < chunks) {
                Steps<X8, TN, TM> now, next;
                int c = wave;
                load(now, first(c));
                for (; c + kWaves < chunks; c += kWaves) {
                    load(next, first(c + kWaves));
                    multiply_chunk(now, 0);
                    now = next;
                }
                multiply_chunk(now, kChunk * c - first(c));
            }
        } else {
            for (int s = wave; s < steps; s += kWaves) {
                uint4 w[TN], x[TM][X8 ? 2 : 1];
                uint32_t sw[TN], sx[TM];
                const int k = s * kStepK;
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    w[i] = *(const uint4*)(wp[i] + k / 2);
                    sw[i] = *(const uint32_t*)(wsp[i] + k / 32);
                }
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    x[j][0] = *(const uint4*)(xp[j] + (X8 ? k : k / 2));
                    if constexpr (X8) x[j][1] = *(const uint4*)(xp[j] + k + 64);
                    sx[j] = *(const uint32_t*)(xsp[j] + k / 32);
                }
                multiply(w, x, sw, sx);
            }
        }

        // join the four waves' sums: wave v finishes every fourth 16 x 16 part
        if (m0 > r0) __syncthreads();                     // (the last rows' parts have been read)
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) part[wave][i * TM + j][lane] = acc[i][j];
        __syncthreads();
#pragma unroll
        for (int p = 0; p < TN * TM; ++p) {
            if (p % kWaves != wave) continue;
            v4f v = part[0][p][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += part[w][p][lane];
            // lane (c, q) holds columns 4 q .. 4 q + 3 of token row c
            const int m = m0 + 16 * (p % TM) + r, n = n0 + 16 * (p / TM) + 4 * b;
            if (m < r1 && n < a.N) {
                if constexpr (F32OUT)
                    *(float4*)((float*)a.y + (int64_t)m * a.N + n) = make_float4(v[0], v[1], v[2], v[3]);
                else
                    *(uint2*)((uint16_t*)a.y + (int64_t)m * a.N + n) =
                        make_uint2(f32_pair_to_bf16(v[0], v[1]), f32_pair_to_bf16(v[2], v[3]));
            }
        }
    }
}

}  // namespace

bool mxfp4_mm_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t G)
{
    // (K: the 256 rows of a tile stay within a buffer resource of 2^31 bytes)
    if (M > ((int64_t)1 << 31) - 1024 || N > ((int64_t)1 << 31) - 1024 || K > ((int64_t)1 << 22)) return false;
    return grouped_mm_sizes_ok(M, N, K, G);
}

hipError_t launch_mxfp4_mm(const void* xq, const void* xs, bool x8, int64_t ldx, int64_t ldxs, const void* wq,
                           const void* wsc, const int32_t* offs, int M, int N, int K, int G, void* y, bool f32_out,
                           hipStream_t stream)
{
    if (M >= many_rows(N, K, G))
        return launch_mxfp4_mm_tile(xq, xs, x8, ldx, ldxs, wq, wsc, offs, M, N, K, G, y, f32_out, stream);
    const FewArgs a = {(const uint8_t*)xq, (const uint8_t*)xs, (const uint8_t*)wq, (const uint8_t*)wsc, offs, y,
                       ldx, ldxs, M, N, K, G};
    const int groups = M < G ? M : G;                     // groups with rows, at most; one more for the rows past them
    const dim3 grid((unsigned)((N + 16 * kTN - 1) / (16 * kTN)), (unsigned)(groups + 1));
#define MXQ_LAUNCH(X8, F) \
    hipLaunchKernelGGL((mxfp4_mm_few_kernel<X8, F, kTN, kTM>), grid, dim3(kThreads), 0, stream, a)
    if (x8 && f32_out) MXQ_LAUNCH(true, true);
    else if (x8) MXQ_LAUNCH(true, false);
    else if (f32_out) MXQ_LAUNCH(false, true);
    else MXQ_LAUNCH(false, false);
#undef MXQ_LAUNCH
    return hipGetLastError();
}

}  // namespace mxq
