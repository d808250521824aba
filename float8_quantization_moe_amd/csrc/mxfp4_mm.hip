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

constexpr int kStepK = 128;           // k of one 16x16 MFMA: four scale blocks
constexpr int64_t kManyRows = 48;      // rows a group, on average, from which the tile kernel takes the call
constexpr int kFewThreads = 256;
constexpr int kFewCols = 64;          // output columns of a workgroup (16 a wave)

// Rows [r0, r1) of group g: running maximum of the end offsets, cut to [0, M];
// g == G is the rows past the last end.  Every lane of the wave must call this.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offs, int G, int g, int M, int& r0, int& r1)
{
    int before = 0;
    for (int i = lane_id(); i < g; i += kWave) before = offs[i] > before ? offs[i] : before;
    before = (int)lanes_max<64>((uint32_t)before);
    int end = g < G ? offs[g] : M;
    end = end > before ? end : before;
    r0 = before < M ? before : M;
    r1 = end < M ? end : M;
}

// One workgroup: 64 columns of one group's rows, 16 rows at a time.  A (16
// columns of W) and B (16 token rows) go straight from global memory into the
// MFMA's registers: lane (r, b) = (lane % 16, lane / 16) holds row r; of E2M1 its
// 16 bytes of scale block b, of E4M3 the 16-byte chunks b and b + 4 of the step.
template <bool X8, bool F32OUT>
__global__ __launch_bounds__(kFewThreads)
void mxfp4_mm_few_kernel(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs, int64_t ldx, int64_t ldxs,
                         const uint8_t* __restrict__ wq, const uint8_t* __restrict__ wsc,
                         const int32_t* __restrict__ offs, int M, int N, int K, int G, void* __restrict__ y)
{
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    const int r = lane & 15, b = lane >> 4;
    const int g = (int)blockIdx.y;
    int r0, r1;
    group_rows(offs, G, g, M, r0, r1);
    const int n0 = (int)blockIdx.x * kFewCols + 16 * wave;
    if (n0 >= N) return;
    const int n = n0 + r;
    const bool n_ok = n < N;
    const int64_t wrow = (int64_t)(g < G ? g : 0) * N + (n_ok ? n : n0);
    const uint8_t* wp = wq + wrow * (K / 2) + 16 * b;
    const uint8_t* wsp = wsc + wrow * (K / 32);
    for (int m0 = r0; m0 < r1; m0 += 16) {
        const int m = m0 + r;
        const int64_t xrow = m < r1 ? m : m0;
        const uint8_t* xp = xq + xrow * ldx + 16 * b;
        const uint8_t* xsp = xs + xrow * ldxs;
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
        if (g < G) {
            for (int k = 0; k < K; k += kStepK) {
                const uint4 wv = *(const uint4*)(wp + k / 2);
                const int sa = (int)(*(const uint32_t*)(wsp + k / 32) >> (8 * b));
                const int sb = (int)(*(const uint32_t*)(xsp + k / 32) >> (8 * b));
                const v8i av = {(int)wv.x, (int)wv.y, (int)wv.z, (int)wv.w, 0, 0, 0, 0};
                v8i bv;
                if constexpr (X8) {
                    const uint4 x0 = *(const uint4*)(xp + k), x1 = *(const uint4*)(xp + k + 64);
                    bv = {(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
                } else {
                    const uint4 x0 = *(const uint4*)(xp + k / 2);
                    bv = {(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, 0, 0, 0, 0};
                }
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, X8 ? 0 : 4, 0, sa, 0, sb);
            }
        }
        // lane (c, q) holds columns 4 q .. 4 q + 3 of token row c
        const int mo = m0 + (lane & 15), no = n0 + 4 * (lane >> 4);
        if (mo < r1 && no < N) {
            if constexpr (F32OUT)
                *(float4*)((float*)y + (int64_t)mo * N + no) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            else
                *(uint2*)((uint16_t*)y + (int64_t)mo * N + no) =
                    make_uint2(f32_pair_to_bf16(acc[0], acc[1]), f32_pair_to_bf16(acc[2], acc[3]));
        }
    }
}

}  // namespace

bool mxfp4_mm_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t G)
{
    if (M > ((int64_t)1 << 31) - 1024 || N > ((int64_t)1 << 31) - 1024) return false;
    return grouped_mm_sizes_ok(M, N, K, G);
}

size_t mxfp4_mm_workspace_bytes(int64_t M, int64_t N, int32_t G) { return grouped_mm_workspace_bytes(M, N, G); }

hipError_t launch_mxfp4_mm(const void* xq, const void* xs, bool x8, int64_t ldx, int64_t ldxs, const void* wq,
                           const void* wsc, const int32_t* offs, int M, int N, int K, int G, void* y, bool f32_out,
                           void* workspace, hipStream_t stream)
{
    if (M >= kManyRows * G)
        return launch_mxfp4_mm_tile(xq, xs, x8, ldx, ldxs, wq, wsc, offs, M, N, K, G, y, f32_out, stream);
    const dim3 grid((unsigned)((N + kFewCols - 1) / kFewCols), (unsigned)(G + 1));
#define MXQ_LAUNCH(X8, F)                                                                                            \
    hipLaunchKernelGGL((mxfp4_mm_few_kernel<X8, F>), grid, dim3(kFewThreads), 0, stream, (const uint8_t*)xq,         \
                       (const uint8_t*)xs, ldx, ldxs, (const uint8_t*)wq, (const uint8_t*)wsc, offs, M, N, K, G, y)
    if (x8 && f32_out) MXQ_LAUNCH(true, true);
    else if (x8) MXQ_LAUNCH(true, false);
    else if (f32_out) MXQ_LAUNCH(false, true);
    else MXQ_LAUNCH(false, false);
#undef MXQ_LAUNCH
    return hipGetLastError();
}

}  // namespace mxq
