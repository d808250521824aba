// bf16_mm.hip -- products grouped by expert in bf16 (gfx950), for every token row m of
// group g with weight W_g (N, K):
//   Y[m, :] = X[m, :] W_g^T;   dX[m, :] = dY[m, :] W_g;   dW_g = sum over m of dY[m, :]^T X[m, :].
//
// A wave computes 32 x 32 results with v_mfma_f32_32x32x16_bf16, its operands straight from
// global memory.
#include "device_common.hpp"
#include "internal.hpp"

#include "../../include/mxq.h"

namespace mxq {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned short v8u16 __attribute__((ext_vector_type(8)));

struct MmArgs {
    const uint16_t *rows, *other;                         // X or dY; W or X
    const int32_t* offs;
    void* out;
    int M, N, K, G;
    bool accumulate;
};

// Values k0 .. k0 + 7 of an operand's row i along the sum; zeros past `rows` and `depth`.
// TRANS: the sum runs over the rows of memory.
template <bool TRANS>
__device__ __forceinline__ v8u16 operand(const uint16_t* p, int64_t ld, int i, int rows, int k0, int depth)
{
    v8u16 v = {};
    if (i < rows) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k0 + e < depth) v[e] = TRANS ? p[(int64_t)(k0 + e) * ld + i] : p[(int64_t)i * ld + k0 + e];
    }
    return v;
}

template <int PRODUCT, bool F32OUT>
__global__ __launch_bounds__(64)
void bf16_mm_kernel(const MmArgs a)
{
    constexpr bool dw = PRODUCT == MXQ_PRODUCT_DW;
    const int lane = lane_id(), r = lane & 31, h = lane >> 5;
    const int cols = PRODUCT == MXQ_PRODUCT_Y ? a.N : a.K;
    const int c0 = (int)blockIdx.x * 32;
    // group and rows of this tile
    int g = 0, lo = 0, hi = 0, tile = (int)blockIdx.y;
    if (dw) g = (int)blockIdx.z;
    int end = 0;
    for (int i = 0; i < a.G; ++i) {
        int e = a.offs[i];
        e = e > end ? (e < a.M ? e : a.M) : end;
        const int tiles = (e - end + 31) / 32;
        if (dw ? i == g : tile < tiles) {
            g = i;
            lo = end;
            hi = e;
            break;
        }
        if (!dw) tile -= tiles;
        end = e;
    }
    const bool zeros = !dw && lo == hi;                    // rows past the last end
    int row0 = 0, rows = a.N;
    const uint16_t *A, *B;
    int64_t lda, ldb;
    int depth;
    if (dw) {
        row0 = (int)blockIdx.y * 32;
        depth = hi - lo;
        B = a.rows + (int64_t)lo * a.N;
        A = a.other + (int64_t)lo * a.K;
        ldb = a.N, lda = a.K;
    } else {
        row0 = zeros ? end + tile * 32 : lo + tile * 32;
        rows = zeros ? a.M : hi;
        depth = zeros ? 0 : PRODUCT == MXQ_PRODUCT_Y ? a.K : a.N;
        B = a.rows;
        A = a.other + (int64_t)g * a.N * a.K;
        ldb = PRODUCT == MXQ_PRODUCT_Y ? a.K : a.N, lda = a.K;
    }
    if (row0 >= rows) return;
    v16f acc = {};
    for (int k = 0; k < depth; k += 16) {
        const v8u16 fa = operand<PRODUCT != MXQ_PRODUCT_Y>(A, lda, c0 + r, cols, k + 8 * h, depth);
        const v8u16 fb = operand<dw>(B, ldb, row0 + r, rows, k + 8 * h, depth);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fa), __builtin_bit_cast(v8bf, fb), acc, 0, 0, 0);
    }
    if (row0 + r >= rows) return;
    const int64_t at = ((dw ? (int64_t)g * a.N : 0) + row0 + r) * cols;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int c = c0 + 8 * (i / 4) + 4 * h + i % 4;
        if (c >= cols) continue;
        if constexpr (F32OUT) ((float*)a.out)[at + c] = a.accumulate ? ((float*)a.out)[at + c] + acc[i] : acc[i];
        else ((__bf16*)a.out)[at + c] = (__bf16)acc[i];
    }
}

}  // namespace

bool bf16_mm_sizes_ok(int product, int64_t M, int64_t N, int64_t K, int64_t G)
{
    constexpr int64_t kMaxSide = (int64_t)1 << 20;
    if (M < 0 || M > ((int64_t)1 << 31) - 1024 || G < 1 || G > 4095) return false;
    if (N < 8 || N > kMaxSide || N % 8 != 0 || K < 8 || K > kMaxSide || K % 8 != 0) return false;
    if (G * N * K > (int64_t)1 << 40) return false;
    const int64_t rows = product == MXQ_PRODUCT_DW ? G * ((N + 63) / 64) : M / 64 + G;
    const int64_t cols = ((product == MXQ_PRODUCT_Y ? N : K) + 255) / 256;
    return rows < ((int64_t)1 << 30) / cols;
}

size_t bf16_mm_workspace_bytes(int product, int64_t M, int64_t N, int64_t K, int64_t G) { return 0; }

hipError_t launch_bf16_mm(int product, const void* rows, const void* other, const int32_t* offs, int M, int N, int K, int G,
                          void* out, bool f32_out, bool accumulate, void* workspace, hipStream_t stream)
{
    const MmArgs a = {(const uint16_t*)rows, (const uint16_t*)other, offs, out, M, N, K, G, accumulate};
    const unsigned cols = (unsigned)(((product == MXQ_PRODUCT_Y ? N : K) + 31) / 32);
    const dim3 grid = product == MXQ_PRODUCT_DW ? dim3(cols, (unsigned)((N + 31) / 32), (unsigned)G)
                                                : dim3(cols, (unsigned)(M / 32 + G + 1));
#define MXQ_LAUNCH(P)                                                                                     \
    do {                                                                                                  \
        if (f32_out) hipLaunchKernelGGL((bf16_mm_kernel<P, true>), grid, dim3(64), 0, stream, a);         \
        else hipLaunchKernelGGL((bf16_mm_kernel<P, false>), grid, dim3(64), 0, stream, a);                \
    } while (0)
    if (product == MXQ_PRODUCT_Y) MXQ_LAUNCH(MXQ_PRODUCT_Y);
    else if (product == MXQ_PRODUCT_DX) MXQ_LAUNCH(MXQ_PRODUCT_DX);
    else MXQ_LAUNCH(MXQ_PRODUCT_DW);
#undef MXQ_LAUNCH
    return hipGetLastError();
}

}  // namespace mxq
