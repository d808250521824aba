// rows.hip -- token rows to their experts and back (gfx950): the gather into expert order,
// the weighted sum of each token's rows, and its gradients.
//
//   dispatch     rows[pair_row[t, j]] = x[t]
//   combine      out[t] = sum over j of w[t, j] * rows[pair_row[t, j]]
//   gradients    drows[pair_row[t, j]] = w[t, j] * dout[t]
//                dw[t, j] = sum over k of dout[t, k] * rows[pair_row[t, j], k]
//
// All walk over tokens, not rows: a token's own row (x, out, dout) is then read or written
// once, its topk rows once each, which is every byte once.  Sums are fp32, over j in order,
// and over k in an order fixed by K.  HBM bound: 8192 tokens x 8 rows x 5120, combine 126 us (6.0 TB/s),
// its gradients 264 us (5.4 TB/s); dispatch of 16640 tokens x 2 rows x 5120 93 us (5.5 TB/s), 5 + 5 us of
// it the two launches that find the rows.
#include "device_common.hpp"
#include "internal.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kBatch = 8;                                 // rows of a token in flight at once
constexpr int kMaxGrid = 1 << 22;
// What does not fit the 256 MB last-level cache is read as a stream (8192 tokens x 8 rows x 5120,
// combine 136 -> 126 us, its gradients 288 -> 270), and dispatched rows written as one (16640 tokens to
// 2 rows each 101 -> 93); less may be there, where its writer left it.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;
template <bool NT>
__device__ __forceinline__ uint4 load16(const uint4* p) { return NT ? load_nt(p) : *p; }
template <class T, bool NT>
__device__ __forceinline__ typename T::Raw load8(const void* row, int64_t i) { return NT ? T::load8_nt(row, i) : T::load8(row, i); }

// Row of pair p, -1 for none.
__device__ __forceinline__ int64_t row_of(const int32_t* pair_row, int64_t p, int64_t R)
{
    const int64_t r = pair_row[p];
    return r >= 0 && r < R ? r : -1;
}
// A wave's number in the launch, in a scalar register: what depends on it alone (a token, its
// rows and weights) is then loaded once a wave.
__device__ __forceinline__ int64_t wave_number()
{
    return (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// A wave takes 64 chunks of 16 bytes of a token.
template <bool NT>
__global__ __launch_bounds__(kThreads)
void dispatch_rows_kernel(const uint4* __restrict__ x, int64_t chunks, int64_t M, int topk, const int32_t* __restrict__ pair_row,
                          const int32_t* __restrict__ group_end, int E, uint4* __restrict__ rows, int32_t* __restrict__ src_pair)
{
    const int64_t slices = (chunks + 63) / 64, P = M * topk;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < P; i += (int64_t)gridDim.x * kThreads)
        if (i >= group_end[E - 1]) src_pair[i] = -1;      // past the last row
    for (int64_t u = wave_number(); u < M * slices; u += (int64_t)gridDim.x * kWaves) {
        const int64_t t = u / slices, c = (u - t * slices) * 64 + lane_id();
        if (c >= chunks) continue;
        const uint4 v = load16<NT>(x + t * chunks + c);
        for (int j = 0; j < topk; ++j) {
            const int64_t r = row_of(pair_row, t * topk + j, P);
            if (r < 0) continue;
            if constexpr (NT) store_nt(v, rows + r * chunks + c);
            else rows[r * chunks + c] = v;
        }
    }
}

__global__ __launch_bounds__(kThreads)
void fill_kernel(int32_t* p, int64_t n, int32_t v)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) p[i] = v;
}

__global__ __launch_bounds__(kThreads)
void pair_rows_kernel(const int32_t* __restrict__ src_pair, int64_t n, int32_t* __restrict__ pair_row)
{
    for (int64_t r = (int64_t)blockIdx.x * kThreads + threadIdx.x; r < n; r += (int64_t)gridDim.x * kThreads) {
        const int64_t p = src_pair[r];
        if (p >= 0 && p < n) pair_row[p] = (int32_t)r;
    }
}

// A wave takes 64 chunks of 8 values of a token.
template <class T, bool NT>
__global__ __launch_bounds__(kThreads)
void combine_rows_kernel(const uint8_t* __restrict__ rows, int64_t R, int64_t K, const int32_t* __restrict__ pair_row, int64_t M,
                         int topk, const float* __restrict__ weights, uint8_t* __restrict__ out)
{
    const int64_t chunks = K / 8, slices = (chunks + 63) / 64, row_bytes = K * T::kBytes;
    for (int64_t u = wave_number(); u < M * slices; u += (int64_t)gridDim.x * kWaves) {
        const int64_t t = u / slices, c = (u - t * slices) * 64 + lane_id();
        if (c >= chunks) continue;
        float acc[8] = {};
        for (int j0 = 0; j0 < topk; j0 += kBatch) {
            typename T::Raw v[kBatch];
            float w[kBatch];
            bool some[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t p = t * topk + j0 + j, r = j0 + j < topk ? row_of(pair_row, p, R) : -1;
                some[j] = r >= 0;
                if (some[j]) {
                    v[j] = load8<T, NT>(rows + r * row_bytes, c);
                    w[j] = weights ? weights[p] : 1.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (some[j]) {
                    float f[8];
                    T::unpack(v[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], f[e], acc[e]);
                }
        }
        T::store8(out + t * row_bytes, c, T::pack(acc));
    }
}

// A workgroup takes a token and kBatch of its slots.  dweights null: only drows.  A chunk of all
// the rows is read before any is written (drows may be rows).
template <class T, bool NT>
__global__ __launch_bounds__(kThreads)
void combine_rows_bwd_kernel(const uint8_t* __restrict__ dout, const uint8_t* rows, int64_t R, int64_t K,
                             const int32_t* __restrict__ pair_row, int64_t M, int topk, const float* __restrict__ weights,
                             uint8_t* drows, float* __restrict__ dweights)
{
    __shared__ float sh[kWaves][kBatch];
    const int64_t chunks = K / 8, row_bytes = K * T::kBytes;
    const int batches = (topk + kBatch - 1) / kBatch;
    for (int64_t u = blockIdx.x; u < M * batches; u += gridDim.x) {
        const int64_t t = u / batches;
        const int j0 = (int)(u - t * batches) * kBatch, n = topk - j0 < kBatch ? topk - j0 : kBatch;
        const int64_t p0 = t * topk + j0;
        float dot[kBatch] = {};
        for (int64_t c = threadIdx.x; c < chunks; c += kThreads) {
            const typename T::Raw dr = T::load8(dout + t * row_bytes, c);
            typename T::Raw v[kBatch];
            int64_t row[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                row[j] = j < n ? row_of(pair_row, p0 + j, R) : -1;
                if (dweights && row[j] >= 0) v[j] = load8<T, NT>(rows + row[j] * row_bytes, c);
            }
            float d[8];
            T::unpack(dr, d);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (row[j] < 0) continue;
                if (dweights) {
                    float f[8];
                    T::unpack(v[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = fmaf(d[e], f[e], dot[j]);
                }
                const float w = weights ? weights[p0 + j] : 1.0f;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = w * d[e];
                T::store8(drows + row[j] * row_bytes, c, T::pack(o));
            }
        }
        if (!dweights) continue;
        __syncthreads();                                  // (the last token's sums have been read)
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float s = lanes_sum<64>(dot[j]);
            if (lane_id() == 0) sh[threadIdx.x >> 6][j] = s;
        }
        __syncthreads();
        if ((int)threadIdx.x < n) {
            float s = 0.0f;
            for (int w = 0; w < kWaves; ++w) s += sh[w][threadIdx.x];
            dweights[p0 + threadIdx.x] = s;
        }
    }
}

unsigned capped(int64_t blocks) { return (unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid); }

}  // namespace

hipError_t launch_dispatch_rows(const void* x, int64_t row_bytes, int64_t M, int topk, const int32_t* pair_row,
                                const int32_t* group_end, int E, void* rows, int32_t* src_pair, hipStream_t stream)
{
    const int64_t chunks = row_bytes / 16, waves = M * ((chunks + 63) / 64);
    const dim3 grid(capped((waves + kWaves - 1) / kWaves));
    if (M * row_bytes * (1 + topk) > kCacheBytes)
        hipLaunchKernelGGL(dispatch_rows_kernel<true>, grid, dim3(kThreads), 0, stream, (const uint4*)x, chunks, M, topk, pair_row,
                           group_end, E, (uint4*)rows, src_pair);
    else
        hipLaunchKernelGGL(dispatch_rows_kernel<false>, grid, dim3(kThreads), 0, stream, (const uint4*)x, chunks, M, topk, pair_row,
                           group_end, E, (uint4*)rows, src_pair);
    return hipGetLastError();
}

hipError_t launch_pair_rows(const int32_t* src_pair, int64_t pairs, int32_t* pair_row, hipStream_t stream)
{
    const unsigned grid = capped((pairs + kThreads - 1) / kThreads);
    hipLaunchKernelGGL(fill_kernel, dim3(grid), dim3(kThreads), 0, stream, pair_row, pairs, -1);
    hipLaunchKernelGGL(pair_rows_kernel, dim3(grid), dim3(kThreads), 0, stream, src_pair, pairs, pair_row);
    return hipGetLastError();
}

#define MXQ_TYPES(CALL)                          \
    do {                                         \
        const bool nt = bytes > kCacheBytes;     \
        if (f32 && nt) CALL(F32, true);          \
        else if (f32) CALL(F32, false);          \
        else if (nt) CALL(Bf16, true);           \
        else CALL(Bf16, false);                  \
    } while (0)

hipError_t launch_combine_rows(const void* rows, bool f32, int64_t R, int64_t K, const int32_t* pair_row, int64_t M, int topk,
                               const float* weights, void* out, hipStream_t stream)
{
    const int64_t waves = M * ((K / 8 + 63) / 64), bytes = M * topk * K * (f32 ? 4 : 2);
    const dim3 grid(capped((waves + kWaves - 1) / kWaves));
#define MXQ_CALL(T, NT)                                                                                                      \
    hipLaunchKernelGGL((combine_rows_kernel<T, NT>), grid, dim3(kThreads), 0, stream, (const uint8_t*)rows, R, K, pair_row, M, \
                       topk, weights, (uint8_t*)out)
    MXQ_TYPES(MXQ_CALL);
#undef MXQ_CALL
    return hipGetLastError();
}

hipError_t launch_combine_rows_bwd(const void* dout, const void* rows, bool f32, int64_t R, int64_t K, const int32_t* pair_row,
                                   int64_t M, int topk, const float* weights, void* drows, float* dweights, hipStream_t stream)
{
    const int64_t bytes = M * topk * K * (f32 ? 4 : 2) * 2;
    const dim3 grid(capped(M * ((topk + kBatch - 1) / kBatch)));
#define MXQ_CALL(T, NT)                                                                                            \
    hipLaunchKernelGGL((combine_rows_bwd_kernel<T, NT>), grid, dim3(kThreads), 0, stream, (const uint8_t*)dout,    \
                       (const uint8_t*)rows, R, K, pair_row, M, topk, weights, (uint8_t*)drows, dweights)
    MXQ_TYPES(MXQ_CALL);
#undef MXQ_CALL
    return hipGetLastError();
}
#undef MXQ_TYPES

}  // namespace mxq
