// norm.hip -- residual addition + root-mean-square norm of token rows, with the
// row's MXFP8 encoding beside the normalised row, and its gradients (gfx950).
//
// Forward, for each row of K values:
//   h = x + r             added in fp32, rounded once to the stored type (h is the
//                         residual stream that the next layer reads, so the norm
//                         is that of the stored h and the backward pass needs
//                         nothing else);
//   rstd = 1 / sqrt(mean(h^2) + eps)        the sum in fp32, the rest in doubles,
//                         rounded once;
//   y = h * rstd * w      rounded once to the stored type;
//   q, s = the MXFP8 encoding of y rounded to bf16: the bytes mxq_quantize_mx
//          writes for y, so that the fused call replaces the two calls bit for bit.
//
// Backward, with g = dy * w and c = mean(g * h) * rstd^2:
//   dx = rstd * (g - h * c) + dh            (the gradient of x and of r alike)
//   dw_k = sum over the rows of dy * h * rstd.
//
// Both are HBM bound (a few operations a value): the row is read once and held in
// registers between its reduction and its use, LANES threads a row with C chunks
// of 8 values each.  65536 x 5120 bf16 with every output: 512 us, 5.9 TB/s; backward of
// 16640 x 5120 with dh: 119 us, 5.7 TB/s.  The sum of a row is eight short chains a lane and one
// tree, in a fixed order, so results are reproducible.
#include "device_common.hpp"
#include "internal.hpp"
#include "mx_block.hpp"

namespace mxq {

namespace {

constexpr int kNormMaxK = 16384;

// Sum over the LANES threads of a row, in all of them.  LANES == 64: a wave
// alone; else through LDS (sh: one float a wave, alternated by `turn` so that one
// barrier a row is enough).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float (*sh)[16], int turn)
{
    v = lanes_sum<64>(v);
    if constexpr (LANES > 64) {
        constexpr int W = LANES / 64;
        if ((threadIdx.x & 63) == 0) sh[turn][threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += sh[turn][w];
    }
    return v;
}

template <class T, int LANES, int C>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES)
void add_rmsnorm_kernel(const uint8_t* x, const uint8_t* r, const uint8_t* __restrict__ w, int64_t M, int K, float eps,
                        uint8_t* h, uint8_t* y, uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                        float* __restrict__ rstd)
{
    constexpr int kRows = LANES < 256 ? 256 / LANES : 1;      // rows of a workgroup
    __shared__ float sh[2][16];
    const int lane = (int)threadIdx.x % LANES;
    const int K8 = K / 8;
    const int64_t row_bytes = (int64_t)K * T::kBytes;
    typename T::Raw wr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = lane + c * LANES;
        if (i < K8) wr[c] = T::load8(w, i);
    }
    int turn = 0;
    for (int64_t m = (int64_t)blockIdx.x * kRows + (int)threadIdx.x / LANES; m < M;
         m += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const int64_t at = m * row_bytes;
        typename T::Raw xr[C], rr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                xr[c] = T::load8(x + at, i);
                if (r) rr[c] = T::load8(r + at, i);
            }
        }
        float ss[8] = {};                                 // eight short sums: an eighth of a chain's roundings
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8];
                T::unpack(xr[c], a);
                if (r) {
                    float b[8];
                    T::unpack(rr[c], b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] += b[e];
                    xr[c] = T::pack(a);
                    T::unpack(xr[c], a);
                }
                if (h) T::store8(h + at, i, xr[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss[e] += a[e] * a[e];
            }
        }
        const float sum = ((ss[0] + ss[1]) + (ss[2] + ss[3])) + ((ss[4] + ss[5]) + (ss[6] + ss[7]));
        // (in doubles, rounded once: with three roundings in floats rstd was off by 0.75 units
        // of 2^-24 in the mean square against 0.6)
        const float rs = (float)(1.0 / sqrt((double)row_sum<LANES>(sum, sh, turn) / K + (double)eps));
        if (rstd && lane == 0) rstd[m] = rs;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8], b[8];
                T::unpack(xr[c], a);
                T::unpack(wr[c], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = a[e] * rs * b[e];
                const typename T::Raw o = T::pack(a);
                if (y) T::store8(y + at, i, o);
                if (q) {                                  // whole quads are in or out (K % 32 == 0)
                    uint32_t code;
                    const uint2 e8 = quantize_chunk<false>(T::bf16_bits(o), &code);
                    store_nt(e8, (uint2*)(q + m * K) + i);
                    if ((lane & 3) == 0) s[m * (K / 32) + (i >> 2)] = (uint8_t)code;
                }
            }
        }
    }
}

// Backward.  Each workgroup walks over rows and keeps its part of dw in fp32
// registers; the parts (one row of `part` for each workgroup) are summed by
// dweight_kernel in a fixed order.
template <class T, int LANES, int C, bool NT>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES)
void add_rmsnorm_bwd_kernel(const uint8_t* __restrict__ h, const uint8_t* __restrict__ w,
                            const float* __restrict__ rstd, const uint8_t* dy, const uint8_t* dh, int64_t M, int K,
                            uint8_t* dx, float* __restrict__ part)
{
    constexpr int kRows = LANES < 256 ? 256 / LANES : 1;
    __shared__ float sh[2][16];
    const int lane = (int)threadIdx.x % LANES;
    const int sub = (int)threadIdx.x / LANES;
    const int K8 = K / 8;
    const int64_t row_bytes = (int64_t)K * T::kBytes;
    typename T::Raw wr[C];
    float acc[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = lane + c * LANES;
        if (i < K8) wr[c] = T::load8(w, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c][e] = 0.0f;
    }
    int turn = 0;
    for (int64_t m = (int64_t)blockIdx.x * kRows + sub; m < M; m += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const int64_t at = m * row_bytes;
        typename T::Raw hr[C], gr[C], dr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                hr[c] = NT ? T::load8_nt(h + at, i) : T::load8(h + at, i);
                gr[c] = NT ? T::load8_nt(dy + at, i) : T::load8(dy + at, i);
                if (dh) dr[c] = NT ? T::load8_nt(dh + at, i) : T::load8(dh + at, i);
            }
        }
        const float rs = rstd[m];
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8], g[8], b[8];
                T::unpack(hr[c], a);
                T::unpack(gr[c], g);
                T::unpack(wr[c], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = a[e] * rs;
                    dot += g[e] * b[e] * n;
                    acc[c][e] += g[e] * n;
                }
            }
        }
        const float mean = row_sum<LANES>(dot, sh, turn) / (float)K;      // mean(g * h) * rstd
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8], g[8], b[8], o[8];
                T::unpack(hr[c], a);
                T::unpack(gr[c], g);
                T::unpack(wr[c], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = rs * (g[e] * b[e] - a[e] * rs * mean);
                if (dh) {
                    float d[8];
                    T::unpack(dr[c], d);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += d[e];
                }
                T::store8(dx + at, i, T::pack(o));
            }
        }
    }
    if constexpr (kRows > 1) {                                // the waves' parts become the workgroup's, in wave order
        __shared__ float join[kRows - 1][LANES * C * 8];
        if (sub > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) join[sub - 1][(c * 8 + e) * LANES + lane] = acc[c][e];
        }
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int r = 0; r < kRows - 1; ++r) acc[c][e] += join[r][(c * 8 + e) * LANES + lane];
    }
    float* dst = part + (int64_t)blockIdx.x * K;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = lane + c * LANES;
        if (i < K8) {
            float4* p = (float4*)dst + 2 * i;
            p[0] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
            p[1] = make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]);
        }
    }
}

// dw[k] = sum over `rows` partial rows.  A workgroup owns 32 columns (8 threads
// of float4) and splits the rows over 32 slices, joined in LDS in slice order.
__global__ __launch_bounds__(256)
void dweight_kernel(const float* __restrict__ part, int rows, int K, float* __restrict__ dw)
{
    __shared__ float4 sh[32][8];
    const int col = (int)threadIdx.x & 7, slice = (int)threadIdx.x >> 3;
    const int k4 = (int)blockIdx.x * 8 + col;
    float4 a = make_float4(0, 0, 0, 0);
    if (k4 < K / 4) {
#pragma unroll 4
        for (int r = slice; r < rows; r += 32) {
            const float4 v = ((const float4*)(part + (int64_t)r * K))[k4];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
    }
    sh[slice][col] = a;
    __syncthreads();
    if (slice == 0 && k4 < K / 4) {
        for (int i = 1; i < 32; ++i) {
            const float4 v = sh[i][col];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
        ((float4*)dw)[k4] = a;
    }
}

constexpr int kNormMaxGrid = 1 << 22;
// Workgroups of the backward pass at most, and so parts of dw: two a CU, which are
// resident together up to K = 8192 (16640 x 5120: 256 / 512 / 768 / 1024 took 147 / 119 / 129 /
// 134 us; 16640 x 1024: 512 / 1024 / 2048 25.4 / 27.5 / 31.0).  Longer rows need more than half
// of the registers, so that the second half runs after the first; not timed apart.
constexpr int kBwdParts = 512;
// Up to this many rows for each of a workgroup's row slots one workgroup takes them all, and
// dw is its part: no second launch (1 to 16 rows, 64 to 5120 values: 12.3 us a call against
// 15.4; 4 rows of 16384: 15.5 both).
constexpr int kBwdOne = 4;
// Inputs that do not fit the 256 MB last-level cache are read as streams (16640 x 5120:
// 119 us, plain loads 128); smaller ones may be in it, where their writer left them
// (4096 x 8192: 47.6 us, as streams 54).  The forward pass measured no such gain.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;

// Threads a row and chunks a thread for K values: a wave while 4 chunks hold the
// row (no barrier), then 256 threads.
#define MXQ_NORM_SHAPE(K, CALL)            \
    do {                                   \
        const int k8_ = ((K) + 7) / 8;     \
        if (k8_ <= 64) CALL(64, 1);        \
        else if (k8_ <= 128) CALL(64, 2);  \
        else if (k8_ <= 256) CALL(64, 4);  \
        else if (k8_ <= 512) CALL(256, 2); \
        else if (k8_ <= 768) CALL(256, 3); \
        else if (k8_ <= 1024) CALL(256, 4);\
        else CALL(256, 8);                 \
    } while (0)

int rows_per_group(int K) { return K <= 2048 ? 4 : 1; }

int64_t bwd_grid(int64_t M, int K)
{
    const int rows = rows_per_group(K);
    const int64_t groups = (M + rows - 1) / rows;
    if (groups <= kBwdOne) return groups < 1 ? groups : 1;
    return groups < kBwdParts ? groups : kBwdParts;
}

}  // namespace

int norm_max_k() { return kNormMaxK; }

hipError_t launch_add_rmsnorm(const void* x, const void* r, const void* w, bool f32, int64_t M, int64_t K, float eps,
                              void* h, void* y, void* q, void* s, float* rstd, hipStream_t stream)
{
    const int rows = rows_per_group((int)K);
    const int64_t groups = (M + rows - 1) / rows;
    const unsigned grid = (unsigned)(groups < kNormMaxGrid ? groups : kNormMaxGrid);
#define MXQ_CALL(L, C)                                                                                              \
    do {                                                                                                            \
        const dim3 block((L) < 256 ? 256 : (L));                                                                    \
        if (f32)                                                                                                    \
            hipLaunchKernelGGL((add_rmsnorm_kernel<F32, L, C>), dim3(grid), block, 0, stream, (const uint8_t*)x,    \
                               (const uint8_t*)r, (const uint8_t*)w, M, (int)K, eps, (uint8_t*)h, (uint8_t*)y,      \
                               (uint8_t*)q, (uint8_t*)s, rstd);                                                     \
        else                                                                                                        \
            hipLaunchKernelGGL((add_rmsnorm_kernel<Bf16, L, C>), dim3(grid), block, 0, stream, (const uint8_t*)x,   \
                               (const uint8_t*)r, (const uint8_t*)w, M, (int)K, eps, (uint8_t*)h, (uint8_t*)y,      \
                               (uint8_t*)q, (uint8_t*)s, rstd);                                                     \
    } while (0)
    MXQ_NORM_SHAPE(K, MXQ_CALL);
#undef MXQ_CALL
    return hipGetLastError();
}

size_t add_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K)
{
    return (size_t)bwd_grid(M, (int)K) * (size_t)K * 4u;
}

hipError_t launch_add_rmsnorm_bwd(const void* h, const void* w, const float* rstd, const void* dy, const void* dh,
                                  bool f32, int64_t M, int64_t K, void* dx, float* dw, void* workspace,
                                  hipStream_t stream)
{
    const int64_t grid = bwd_grid(M, (int)K);
    float* part = grid == 1 ? dw : (float*)workspace;
    const bool nt = M * K * (f32 ? 4 : 2) * (dh ? 3 : 2) > kCacheBytes;
    if (grid > 0) {
#define MXQ_LAUNCH(T, L, C, NT)                                                                                     \
    hipLaunchKernelGGL((add_rmsnorm_bwd_kernel<T, L, C, NT>), dim3((unsigned)grid), dim3((L) < 256 ? 256 : (L)), 0, \
                       stream, (const uint8_t*)h, (const uint8_t*)w, rstd, (const uint8_t*)dy, (const uint8_t*)dh,  \
                       M, (int)K, (uint8_t*)dx, part)
#define MXQ_CALL(L, C)                                   \
    do {                                                 \
        if (f32 && nt) MXQ_LAUNCH(F32, L, C, true);      \
        else if (f32) MXQ_LAUNCH(F32, L, C, false);      \
        else if (nt) MXQ_LAUNCH(Bf16, L, C, true);       \
        else MXQ_LAUNCH(Bf16, L, C, false);              \
    } while (0)
        MXQ_NORM_SHAPE(K, MXQ_CALL);
#undef MXQ_CALL
#undef MXQ_LAUNCH
    }
    if (grid == 1) return hipGetLastError();
    hipLaunchKernelGGL(dweight_kernel, dim3((unsigned)((K / 4 + 7) / 8)), dim3(256), 0, stream, part,
                       (int)grid, (int)K, dw);
    return hipGetLastError();
}

}  // namespace mxq
