// layernorm.hip -- residual addition + layer norm of token rows, with the row's MXFP8
// encoding beside the normalised row, and its gradients (gfx950).
//
// Forward, for each row of K values:
//   h = x + r             added in fp32, rounded once to the stored type (the residual
//                         stream that the next layer reads; the norm is that of the stored h);
//   m = mean(h);  v = mean((h - m)^2);  rstd = 1 / sqrt(v + eps);
//   y = (h - m) * rstd * w + b      rounded once to the stored type;
//   q, s = the MXFP8 encoding of y rounded to bf16.
// The row is in registers, so the squares are those of the differences from a mean that is
// already known (mean(h^2) - m^2 loses everything when m^2 is large next to v).  That mean is
// cut to 16 bits; what it lacks is the mean of those differences, taken in the same pass: m
// gets it added, v its square taken off.
//
// Backward, with n = (h - m) * rstd and g = dy * w:
//   dx = rstd * (g - mean(g) - n * mean(g * n)) + dh      (the gradient of x and of r alike)
//   dw_k = sum over the rows of dy * n;  db_k = sum over the rows of dy.
//
// Both are HBM bound: the row is read once and held in registers between its reductions and
// its use, LANES threads a row with C chunks of 8 values each.  Sums go in a fixed order.
// 65536 x 5120 bf16 with every output: 528 us, 5.7 TB/s; backward of 16640 x 5120 with dh: 122 us,
// 5.6 TB/s.  The backward pass is near its VALU's bound too: with n and dy * w made again after
// the sums it took 136 us, with the next row's loads ahead of that 142.
#include "device_common.hpp"
#include "internal.hpp"
#include "mx_block.hpp"

#include <type_traits>

namespace mxq {

namespace {

constexpr int kWaves = 8;                                 // of a workgroup, at most
// y is rounded to bf16 (itself or for its codes) from fp32 arithmetic that is good to two units of
// 2^-24 or so; where the fp32 value is within this many of the middle between two bf16, the chunk is
// computed again in doubles, rounded to fp32 first.  Of 3.4e8 values 1300 then differ from the exact
// ones' roundings by way of fp32 and of 10^7 blocks' scales none; 3800 and one or two without it; 13000
// and one in steps of fp32 throughout (65536 x 5120: 528 us; 515 with sums in fp32, 593 all in doubles).
// Against the bf16 nearest to the exact values themselves it is 3900 and at times one: some 2600 of
// 3.4e8 roundings to fp32 land on a middle from the wrong side.  fp32 rows take this path too, so that
// their y is the same with and without codes.
constexpr uint32_t kNear = 4;

// Sums of two values over the LANES threads of a row, in all of them: a wave alone, else
// through LDS (alternated by `turn`, so that one barrier is enough).
template <int LANES>
__device__ __forceinline__ float2 row_sums(float a, float b, float2 (*sh)[kWaves], int turn)
{
    a = lanes_sum<64>(a);
    b = lanes_sum<64>(b);
    if constexpr (LANES > 64) {
        constexpr int W = LANES / 64;
        if ((threadIdx.x & 63) == 0) sh[turn][threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += sh[turn][w].x;
            b += sh[turn][w].y;
        }
    }
    return make_float2(a, b);
}

// Over the wave, by moves of the halves as lanes_sum.
__device__ __forceinline__ double wave_sum(double v)
{
    const auto moved = [](double x, auto ctrl) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const uint64_t lo = dpp_move<decltype(ctrl)::value>((uint32_t)b), hi = dpp_move<decltype(ctrl)::value>((uint32_t)(b >> 32));
        return __builtin_bit_cast(double, hi << 32 | lo);
    };
    const auto lane = [](double x, int l) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const uint64_t lo = (uint32_t)readlane((int)(uint32_t)b, l), hi = (uint32_t)readlane((int)(uint32_t)(b >> 32), l);
        return __builtin_bit_cast(double, hi << 32 | lo);
    };
    v += moved(v, std::integral_constant<int, kDppXor1>{});
    v += moved(v, std::integral_constant<int, kDppXor2>{});
    v += moved(v, std::integral_constant<int, kDppHalfMirror>{});
    v += moved(v, std::integral_constant<int, kDppMirror>{});
    return (lane(v, 0) + lane(v, 16)) + (lane(v, 32) + lane(v, 48));
}
// Sums of two doubles over the LANES threads of a row, in all of them.
template <int LANES>
__device__ __forceinline__ double2 row_sums(double a, double b, double2 (&sh)[kWaves])
{
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (LANES > 64) {
        constexpr int W = LANES / 64;
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_double2(a, b);
        __syncthreads();
        a = b = 0.0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += sh[w].x;
            b += sh[w].y;
        }
    }
    return make_double2(a, b);
}

__device__ __forceinline__ float sum8(const float (&v)[8])
{
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

template <class T, int LANES, int C, bool NT>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES, T::kBytes * C <= (NT ? 6 : 4) ? 3 : 2)
void add_layernorm_kernel(const uint8_t* x, const uint8_t* r, const uint8_t* __restrict__ w, const uint8_t* __restrict__ b,
                          int64_t M, int K, float eps, uint8_t* h, uint8_t* y, uint8_t* __restrict__ q,
                          uint8_t* __restrict__ s, float* __restrict__ mean, float* __restrict__ rstd)
{
    constexpr int kRows = LANES < 256 ? 256 / LANES : 1;      // rows of a workgroup
    __shared__ float2 sh[2][kWaves];
    __shared__ double2 shd[kWaves];
    const int lane = (int)threadIdx.x % LANES;
    const int K8 = K / 8;
    const int64_t row_bytes = (int64_t)K * T::kBytes;
    constexpr bool kHold = LANES < 512;                   // (w and b anew from the cache where registers are short)
    typename T::Raw wr[C], br[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = lane + c * LANES;
        br[c] = {};
        if (kHold && i < K8) {
            wr[c] = T::load8(w, i);
            if (b) br[c] = T::load8(b, i);
        }
    }
    for (int64_t m = (int64_t)blockIdx.x * kRows + (int)threadIdx.x / LANES; m < M; m += (int64_t)gridDim.x * kRows) {
        const int64_t at = m * row_bytes;
        typename T::Raw xr[C], rr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                xr[c] = NT ? T::load8_nt(x + at, i) : T::load8(x + at, i);
                if (r) rr[c] = NT ? T::load8_nt(r + at, i) : T::load8(r + at, i);
            }
        }
        float t[8] = {};                                  // eight short sums: an eighth of a chain's roundings
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8];
                T::unpack(xr[c], a);
                if (r) {
                    float d[8];
                    T::unpack(rr[c], d);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] += d[e];
                    xr[c] = T::pack(a);
                    T::unpack(xr[c], a);
                }
                if (h) T::store8(h + at, i, xr[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] += a[e];
            }
        }
        // (cut to 16 bits, so that the differences of bf16 values of its size from it are exact: their
        // roundings are alike over a row, and the mean lacked half a unit of them)
        const float m0 = __uint_as_float(__float_as_uint(row_sums<LANES>(sum8(t), 0.0f, sh, 0).x / (float)K) & 0xFFFFFF00u);
        double d1 = 0.0, d2 = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8];
                T::unpack(xr[c], a);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double d = a[e] - m0;
                    d1 += d;
                    d2 = fma(d, d, d2);
                }
            }
        }
        const double2 sums = row_sums<LANES>(d1, d2, shd);
        const double left = sums.x / K;                   // what the mean lacks
        const double var = sums.y / K - left * left;
        const double rstd64 = 1.0 / sqrt((var < 0.0 ? 0.0 : var) + (double)eps), mean64 = (double)m0 + left;
        const float rs = (float)rstd64, l0 = (float)left;
        if (lane == 0) {
            if (mean) mean[m] = (float)mean64;
            if (rstd) rstd[m] = rs;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float a[8], f[8], g[8], o[8];
                T::unpack(xr[c], a);
                T::unpack(kHold ? wr[c] : T::load8(w, i), f);
                T::unpack(kHold || !b ? br[c] : T::load8(b, i), g);
                uint32_t least = ~0u;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o[e] = fmaf((a[e] - m0 - l0) * rs, f[e], g[e]);
                    const uint32_t from = (__float_as_uint(o[e]) - (0x8000u - kNear)) << 16;
                    least = from < least ? from : least;
                }
                if (least <= (2u * kNear) << 16) {        // near the middle of two bf16: again in doubles
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = (float)fma(((double)a[e] - mean64) * rstd64, (double)f[e], (double)g[e]);
                }
                const typename T::Raw p = T::pack(o);
                if (y) T::store8(y + at, i, p);
                if (q) {                                  // whole quads are in or out (K % 32 == 0)
                    uint32_t code;
                    const uint2 e8 = quantize_chunk<false>(T::bf16_bits(p), &code);
                    store_nt(e8, (uint2*)(q + m * K) + i);
                    if ((lane & 3) == 0) s[m * (K / 32) + (i >> 2)] = (uint8_t)code;
                }
            }
        }
    }
}

// Backward.  Each workgroup walks over rows and keeps its parts of dw and db in fp32
// registers; the parts (a row of 2K floats for each workgroup) are summed by
// columns_kernel in a fixed order.
template <class T, int LANES, int C, bool NT>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES)
void add_layernorm_bwd_kernel(const uint8_t* __restrict__ h, const uint8_t* __restrict__ w, const float* __restrict__ mean,
                              const float* __restrict__ rstd, const uint8_t* dy, const uint8_t* dh, int64_t M, int K,
                              uint8_t* dx, float* __restrict__ part_w, float* __restrict__ part_b, int64_t part_stride)
{
    constexpr int kRows = LANES < 256 ? 256 / LANES : 1;
    __shared__ float2 sh[2][kWaves];
    const int lane = (int)threadIdx.x % LANES;
    const int sub = (int)threadIdx.x / LANES;
    const int K8 = K / 8;
    const int64_t row_bytes = (int64_t)K * T::kBytes;
    constexpr bool kHoldW = LANES < 512;                  // (a row's w anew from the cache where registers are short)
    typename T::Raw wr[C];
    float aw[C][8], ab[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = lane + c * LANES;
        if (kHoldW && i < K8) wr[c] = T::load8(w, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[c][e] = ab[c][e] = 0.0f;
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
        const float mu = mean[m], rs = rstd[m];
        // n = (h - m) * rstd and u = dy * w; held in fp32 between the passes where registers allow it
        constexpr bool kHold = C <= 3;
        float hn[kHold ? C : 1][8], hu[kHold ? C : 1][8];
        // n is left as h - m, whose product with rstd comes where it is used (with it here one variant spills)
        const auto differences = [&](int c, int i, float (&n)[8], float (&u)[8], float (&g)[8]) {
            float f[8];
            T::unpack(hr[c], n);
            T::unpack(gr[c], g);
            T::unpack(kHoldW ? wr[c] : T::load8(w, i), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] -= mu;
                u[e] = g[e] * f[e];
            }
        };
        float s1 = 0.0f, s2 = 0.0f;                       // sums of u and of u * n
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float n[8], u[8], g[8];
                differences(c, i, n, u, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[e] *= rs;
                    s1 += u[e];
                    s2 = fmaf(u[e], n[e], s2);
                    aw[c][e] = fmaf(g[e], n[e], aw[c][e]);
                    ab[c][e] += g[e];
                    if constexpr (kHold) {
                        hn[c][e] = n[e];
                        hu[c][e] = u[e];
                    }
                }
            }
        }
        const float2 sums = row_sums<LANES>(s1, s2, sh, turn);
        // dx = rstd u - rstd mean(u) - n rstd mean(u n); not with (h - m) and rstd^2, which leaves
        // fp32's range at spreads of 1e19 and 1e-19 already
        const float k1 = -rs * (sums.x / (float)K), k2 = -rs * (sums.y / (float)K);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + c * LANES;
            if (i < K8) {
                float n[8], u[8], g[8], o[8];
                if constexpr (!kHold) differences(c, i, n, u, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (kHold) {
                        n[e] = hn[c][e];
                        u[e] = hu[c][e];
                    } else {
                        n[e] *= rs;
                    }
                    o[e] = fmaf(n[e], k2, fmaf(u[e], rs, k1));
                }
                if (dh) {
                    float r[8];
                    T::unpack(dr[c], r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += r[e];
                }
                T::store8(dx + at, i, T::pack(o));
            }
        }
    }
    if constexpr (kRows > 1) {                            // the waves' parts become the workgroup's, in wave order
        __shared__ float join[kRows - 1][LANES * C * 8];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float (&acc)[C][8] = which ? ab : aw;
            if (which) __syncthreads();
            if (sub > 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) join[sub - 1][(c * 8 + e) * LANES + lane] = acc[c][e];
            }
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int r = 0; r < kRows - 1; ++r) acc[c][e] += join[r][(c * 8 + e) * LANES + lane];
            }
        }
        if (sub > 0) return;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float (&acc)[C][8] = which ? ab : aw;
        float* dst = which ? part_b : part_w;
        if (!dst) continue;
        dst += (int64_t)blockIdx.x * part_stride;
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
}

// dw and db: the sums over `rows` rows of 2K floats (dw's parts, then db's).  A workgroup
// owns 32 columns (8 threads of float4) and splits the rows over 32 slices, joined in LDS
// in slice order.
__global__ __launch_bounds__(256)
void columns_kernel(const float* __restrict__ part, int rows, int K, float* __restrict__ dw, float* __restrict__ db)
{
    __shared__ float4 sh[32][8];
    const int col = (int)threadIdx.x & 7, slice = (int)threadIdx.x >> 3;
    const int k4 = (int)blockIdx.x * 8 + col, n4 = (db ? 2 : 1) * (K / 4);
    float4 a = make_float4(0, 0, 0, 0);
    if (k4 < n4) {
#pragma unroll 4
        for (int r = slice; r < rows; r += 32) {
            const float4 v = ((const float4*)(part + (int64_t)r * 2 * K))[k4];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
    }
    sh[slice][col] = a;
    __syncthreads();
    if (slice == 0 && k4 < n4) {
        for (int i = 1; i < 32; ++i) {
            const float4 v = sh[i][col];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
        if (k4 < K / 4) ((float4*)dw)[k4] = a;
        else ((float4*)db)[k4 - K / 4] = a;
    }
}

constexpr int kMaxGrid = 1 << 22;
// Inputs that do not fit the 256 MB last-level cache are read as streams (65536 x 5120 with a
// residual 4 % less; backward 16640 x 5120 with dh 137 -> 135); smaller ones may be there.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;
// Workgroups of the backward pass at most, and so parts: two a CU, which are resident together
// (16640 x 5120: 512 / 768 119 / 141 us).
constexpr int kBwdParts = 512;
constexpr int kBwdOne = 4;                                // up to this many rows a row slot, one workgroup takes them all

// Threads a row and chunks a thread for K values (at most 16384).
#define MXQ_NORM_SHAPE(K, CALL)            \
    do {                                   \
        const int k8_ = ((K) + 7) / 8;     \
        if (k8_ <= 64) CALL(64, 1);        \
        else if (k8_ <= 128) CALL(64, 2);  \
        else if (k8_ <= 256) CALL(64, 4);  \
        else if (k8_ <= 512) CALL(256, 2); \
        else if (k8_ <= 768) CALL(256, 3); \
        else if (k8_ <= 1024) CALL(256, 4);\
        else CALL(512, 4);                 \
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

hipError_t launch_add_layernorm(const void* x, const void* r, const void* w, const void* b, bool f32, int64_t M, int64_t K,
                                float eps, void* h, void* y, void* q, void* s, float* mean, float* rstd, hipStream_t stream)
{
    const int rows = rows_per_group((int)K);
    const int64_t groups = (M + rows - 1) / rows;
    const unsigned grid = (unsigned)(groups < kMaxGrid ? groups : kMaxGrid);
    const bool nt = M * K * (f32 ? 4 : 2) * (r ? 2 : 1) > kCacheBytes;
#define MXQ_LAUNCH(T, L, C, NT)                                                                                        \
    hipLaunchKernelGGL((add_layernorm_kernel<T, L, C, NT>), dim3(grid), dim3((L) < 256 ? 256 : (L)), 0, stream,             \
                       (const uint8_t*)x, (const uint8_t*)r, (const uint8_t*)w, (const uint8_t*)b, M, (int)K, eps,      \
                       (uint8_t*)h, (uint8_t*)y, (uint8_t*)q, (uint8_t*)s, mean, rstd)
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
    return hipGetLastError();
}

size_t add_layernorm_bwd_workspace_bytes(int64_t M, int64_t K)
{
    return (size_t)bwd_grid(M, (int)K) * (size_t)K * 8u;
}

hipError_t launch_add_layernorm_bwd(const void* h, const void* w, const float* mean, const float* rstd, const void* dy,
                                    const void* dh, bool f32, int64_t M, int64_t K, void* dx, float* dw, float* db,
                                    void* workspace, hipStream_t stream)
{
    const int64_t grid = bwd_grid(M, (int)K);
    float* part = (float*)workspace;
    float* part_w = grid == 1 ? dw : part;
    float* part_b = grid == 1 || !db ? db : part + K;
    if (grid > 0) {
        const bool nt = M * K * (f32 ? 4 : 2) * (dh ? 3 : 2) > kCacheBytes;
#define MXQ_LAUNCH(T, L, C, NT)                                                                                        \
    hipLaunchKernelGGL((add_layernorm_bwd_kernel<T, L, C, NT>), dim3((unsigned)grid), dim3((L) < 256 ? 256 : (L)), 0, stream, \
                       (const uint8_t*)h, (const uint8_t*)w, mean, rstd, (const uint8_t*)dy, (const uint8_t*)dh, M,     \
                       (int)K, (uint8_t*)dx, part_w, part_b, 2 * K)
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
    const unsigned blocks = (unsigned)(((db ? 2 : 1) * K / 4 + 7) / 8);
    hipLaunchKernelGGL(columns_kernel, dim3(blocks), dim3(256), 0, stream, part, (int)grid, (int)K, dw, db);
    return hipGetLastError();
}

}  // namespace mxq
