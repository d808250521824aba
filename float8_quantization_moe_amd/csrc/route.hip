// route.hip -- expert routing on gfx950: scores, balance bias, expert groups,
// top-k selection and the selected experts' weights, and the logits' gradient.
//
// For a row of E logits l:
//   score   s_e = exp(l_e - max l) / sum_i exp(l_i - max l), or 1 / (1 + exp(-l_e));
//   key     s_e + bias_e; without a bias l_e itself (both scores grow with l, so
//           the order is the same and no two logits fall together by rounding);
//   group   E / n_groups neighbours; its value is the largest s + bias (without a
//           bias: of exp(l - max l), or of the sigmoid) in it, or the sum of its
//           two largest; the topk_groups largest groups stay;
//   ids     the topk largest keys of the groups that stay, largest first;
//   weights scale * s, or scale * s / (sum of the selected s + 1e-20).
// Ties go to the lowest index, of groups and of experts.  A logit of -inf or NaN
// (or a key of -inf or NaN) is never selected; slots that nothing is left for
// get id -1 and weight 0.
// All arithmetic is fp32 with the correctly rounded divide: the selection must
// not depend on how a row is spread over lanes, so the keys use nothing but
// operations on one value (and, for softmax with a bias, the row's sum).
//
// Forward layout: L lanes a row (16 lanes for E <= 256, so that a wave works on
// four rows and each cross-lane step serves all four; 64 beyond), each with
// 4 C values in registers: lane i holds experts 4 (i + L j) .. + 3.  A round of
// the selection is an integer maximum over the row (the keys mapped to integers
// of the same order, 0 for "not eligible"), then the lowest index that holds it;
// both finish across the lanes with DPP.  Reading the logits is the floor; the
// rounds' VALU work is what bounds it.
#include "device_common.hpp"
#include "internal.hpp"

namespace mxq {

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 64;
constexpr float kTiny = 1e-20f;
#define MXQ_NEG_INF (-__builtin_huge_valf())

// Integers of the same order as the floats; 0 is below every float.  (-0 counts
// as +0, as in a comparison of floats.)
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }

// The 4 logits of experts e0 .. e0+3 of a row; -inf past E.  `vec`: rows are
// aligned to 4 values (E % 4 == 0).
template <bool F32L>
__device__ __forceinline__ void load4(const void* row, int e0, int E, bool vec, float (&v)[4])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = MXQ_NEG_INF;
    if (vec) {
        if (e0 < E) {
            if constexpr (F32L) {
                const float4 t = *(const float4*)((const float*)row + e0);
                v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
            } else {
                const uint2 t = *(const uint2*)((const uint16_t*)row + e0);
                v[0] = bf16_lo_to_f32(t.x), v[1] = bf16_hi_to_f32(t.x);
                v[2] = bf16_lo_to_f32(t.y), v[3] = bf16_hi_to_f32(t.y);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (e0 + c < E) {
                if constexpr (F32L) v[c] = ((const float*)row)[e0 + c];
                else v[c] = bf16_lo_to_f32(((const uint16_t*)row)[e0 + c]);
            }
    }
}

template <int L>
__device__ __forceinline__ float lanes_max_f(float v)
{
    return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}

struct RouteArgs {
    int E, n_groups, topk_groups, topk;
    int group_size;              // E / n_groups
    uint32_t group_magic;        // e / group_size == mulhi(e, group_magic) for e < 1024 (group_size > 1)
    float scale;
    bool renorm, top2;
};

// LDS of one workgroup, per row: E values (groups only), n_groups values, topk
// ids and scores.
template <bool F32L, bool SIGMOID, int L, int C>
__global__ __launch_bounds__(kRouteThreads)
void route_topk_kernel(const void* __restrict__ logits, const float* __restrict__ bias, int64_t M, RouteArgs a,
                       int32_t* __restrict__ ids, float* __restrict__ weights)
{
    constexpr int kRows = kRouteThreads / L;
    constexpr int kMaxE = 4 * L * C;
    __shared__ float values[kRows][kMaxE + 4];
    __shared__ float gvalues[kRows][kMaxE + 4];
    __shared__ int32_t out_id[kRows][kRouteMaxTopk];
    __shared__ float out_s[kRows][kRouteMaxTopk];
    const int lane = (int)threadIdx.x % L, sub = (int)threadIdx.x / L;
    const int E = a.E;
    const bool vec = E % 4 == 0;
    for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < M; m0 += (int64_t)gridDim.x * kRows) {
        const int64_t m = m0 + sub;
        const bool live = m < M;
        const uint8_t* row = (const uint8_t*)logits + (live ? m : M - 1) * E * (F32L ? 4 : 2);

        // scores s, and the row's poison: a NaN anywhere, or +inf under softmax
        float l[C][4], s[C][4], v[C][4];
        bool bad = false;
        float top = MXQ_NEG_INF;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            load4<F32L>(row, 4 * (lane + L * j), E, vec, l[j]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                bad |= l[j][c] != l[j][c] || (!SIGMOID && l[j][c] == -MXQ_NEG_INF);
                top = fmaxf(top, l[j][c]);
            }
        }
        float total = 1.0f;
        if constexpr (SIGMOID) {
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[j][c] = s[j][c] = sigmoid_of(l[j][c]);
        } else {
            top = lanes_max_f<L>(top);
            top = top > MXQ_NEG_INF ? top : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    v[j][c] = expf(l[j][c] - top);
                    sum += v[j][c];
                }
            total = lanes_sum<L>(sum);
            total = total > 0.0f ? total : 1.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[j][c] = v[j][c] / total;
        }
        bad = lanes_max<L>(bad ? 1u : 0u) != 0;

        // keys
        uint32_t key[C][4];
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int e = 4 * (lane + L * j) + c;
                float k = l[j][c];
                if (bias) k = v[j][c] = s[j][c] + (e < E ? bias[e] : 0.0f);
                const bool ok = l[j][c] > MXQ_NEG_INF && k > MXQ_NEG_INF;      // (false for NaN)
                key[j][c] = ok ? order_key(k) : 0u;
                if (a.n_groups > 1 && e < E) values[sub][e] = ok ? v[j][c] : MXQ_NEG_INF;
            }

        if (a.n_groups > 1) {                                     // (uniform)
            __syncthreads();
            for (int g = lane; g < a.n_groups; g += L) {
                float v1 = MXQ_NEG_INF, v2 = MXQ_NEG_INF;
                for (int i = 0; i < a.group_size; ++i) {
                    const float t = values[sub][g * a.group_size + i];
                    v2 = fmaxf(v2, fminf(v1, t));
                    v1 = fmaxf(v1, t);
                }
                gvalues[sub][g] = a.top2 && v2 > MXQ_NEG_INF ? v1 + v2 : v1;
            }
            __syncthreads();
            // a group stays if fewer than topk_groups precede it; `values` becomes the flag
            for (int g = lane; g < a.n_groups; g += L) {
                const float t = gvalues[sub][g];
                int before = 0;
                for (int i = 0; i < a.n_groups; ++i) {
                    const float u = gvalues[sub][i];
                    before += u > t || (u == t && i < g) ? 1 : 0;
                }
                values[sub][g] = before < a.topk_groups ? 1.0f : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int e = 4 * (lane + L * j) + c;
                    const int g = a.group_size > 1 ? (int)__umulhi((uint32_t)e, a.group_magic) : e;
                    if (e < E && values[sub][g] == 0.0f) key[j][c] = 0u;
                }
        }

        // topk rounds
        float picked = 0.0f;                                      // this lane's part of the selected scores' sum
        for (int t = 0; t < a.topk; ++t) {
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) best = key[j][c] > best ? key[j][c] : best;
            best = lanes_max<L>(best);
            uint32_t id = 0xFFFFFFFFu;
#pragma unroll
            for (int j = C - 1; j >= 0; --j)
#pragma unroll
                for (int c = 3; c >= 0; --c)
                    if (key[j][c] == best) id = (uint32_t)(4 * (lane + L * j) + c);
            id = lanes_min<L>(id);
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if ((uint32_t)(4 * (lane + L * j) + c) == id) {
                        if (best != 0) {
                            out_id[sub][t] = (int32_t)id;
                            out_s[sub][t] = s[j][c];
                            picked += s[j][c];
                        }
                        key[j][c] = 0u;
                    }
            if (best == 0 && lane == 0) {
                out_id[sub][t] = -1;
                out_s[sub][t] = 0.0f;
            }
        }
        const float sum = lanes_sum<L>(picked) + kTiny;
        __syncthreads();
        for (int t = lane; t < a.topk; t += L) {
            float w = out_s[sub][t];
            if (a.renorm) w /= sum;
            w *= a.scale;
            if (bad) w = __builtin_nanf("");
            if (live) {
                ids[m * a.topk + t] = out_id[sub][t];
                weights[m * a.topk + t] = w;
            }
        }
        __syncthreads();
    }
}

// Gradient.  With u_j the incoming gradient of weight j and s the scores:
//   g_j = scale * u_j, or, renormalised with D = sum of the selected s + 1e-20,
//         (scale * u_j - sum_i scale * u_i s_i / D) / D;
//   sigmoid: dl_e = s_e (1 - s_e) g_e at the selected experts, 0 elsewhere;
//   softmax: dl_e = s_e (g_e - sum_j g_j s_j) everywhere (g = 0 where not selected).
// Softmax with renormalisation is the softmax over the selected logits alone, so
// its gradient is 0 elsewhere and the other logits are not read.
// Same layout as the forward; the selected experts' g pass through LDS.
template <bool F32L, bool SIGMOID, int L, int C>
__global__ __launch_bounds__(kRouteThreads)
void route_topk_bwd_kernel(const void* __restrict__ logits, const int32_t* __restrict__ ids,
                           const float* __restrict__ dweights, int64_t M, int E, int topk, bool renorm, float scale,
                           void* __restrict__ dlogits)
{
    constexpr int kRows = kRouteThreads / L;
    constexpr int kMaxE = 4 * L * C;
    constexpr int kSlots = (kRouteMaxTopk + L - 1) / L;           // slots a lane handles at most
    __shared__ float grad[kRows][kMaxE + 4];
    const int lane = (int)threadIdx.x % L, sub = (int)threadIdx.x / L;
    const bool vec = E % 4 == 0;
    const bool dense = !SIGMOID && !renorm;
    for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < M; m0 += (int64_t)gridDim.x * kRows) {
        const int64_t m = m0 + sub;
        const bool live = m < M;
        const int64_t mr = live ? m : M - 1;
        const uint8_t* row = (const uint8_t*)logits + mr * E * (F32L ? 4 : 2);

        float l[C][4], p[C][4];
        float top = MXQ_NEG_INF, total = 1.0f;
        if (dense) {                                              // (uniform)
#pragma unroll
            for (int j = 0; j < C; ++j) {
                load4<F32L>(row, 4 * (lane + L * j), E, vec, l[j]);
#pragma unroll
                for (int c = 0; c < 4; ++c) top = fmaxf(top, l[j][c]);
            }
            top = lanes_max_f<L>(top);
            top = top > MXQ_NEG_INF ? top : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    p[j][c] = expf(l[j][c] - top);
                    sum += p[j][c];
                }
            total = lanes_sum<L>(sum);
            total = total > 0.0f ? total : 1.0f;
        }
        for (int e = lane; e < kMaxE; e += L) grad[sub][e] = 0.0f;

        // this lane's slots: the selected expert, its logit and gradient
        int id[kSlots];
        float ls[kSlots], sc[kSlots], g[kSlots];
        float seltop = MXQ_NEG_INF;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int t = lane + L * i;
            id[i] = -1;
            ls[i] = MXQ_NEG_INF;
            g[i] = 0.0f;
            if (t < topk) {
                const int e = ids[mr * topk + t];
                if (e >= 0 && e < E) {
                    id[i] = e;
                    g[i] = scale * dweights[mr * topk + t];
                    if constexpr (F32L) ls[i] = ((const float*)row)[e];
                    else ls[i] = bf16_lo_to_f32(((const uint16_t*)row)[e]);
                }
            }
            seltop = fmaxf(seltop, ls[i]);
        }
        float sum = 0.0f, dot = 0.0f;
        if constexpr (!SIGMOID) {
            if (!dense) {
                top = lanes_max_f<L>(seltop);
                top = top > MXQ_NEG_INF ? top : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            sc[i] = 0.0f;
            if (id[i] >= 0) sc[i] = SIGMOID ? sigmoid_of(ls[i]) : expf(ls[i] - top) / total;
            sum += sc[i];
            dot += g[i] * sc[i];
        }
        sum = lanes_sum<L>(sum) + kTiny;
        dot = lanes_sum<L>(dot);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (id[i] >= 0) {
                float d = g[i];
                if (renorm) d = (d - dot / sum) / sum;
                if (SIGMOID) d *= sc[i] * (1.0f - sc[i]);
                else if (renorm) d *= sc[i];
                grad[sub][id[i]] = d;
            }
        __syncthreads();
        if (live) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int e0 = 4 * (lane + L * j);
                float d[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    d[c] = grad[sub][e0 + c];
                    if (dense) d[c] = p[j][c] / total * (d[c] - dot);
                }
                if (vec) {
                    if (e0 < E) {
                        if constexpr (F32L)
                            *(float4*)((float*)dlogits + m * E + e0) = make_float4(d[0], d[1], d[2], d[3]);
                        else
                            *(uint2*)((uint16_t*)dlogits + m * E + e0) =
                                make_uint2(f32_pair_to_bf16(d[0], d[1]), f32_pair_to_bf16(d[2], d[3]));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (e0 + c < E) {
                            if constexpr (F32L) ((float*)dlogits)[m * E + e0 + c] = d[c];
                            else ((uint16_t*)dlogits)[m * E + e0 + c] = (uint16_t)f32_pair_to_bf16(d[c], 0.0f);
                        }
                }
            }
        }
        __syncthreads();
    }
}

constexpr int64_t kRouteMaxGrid = 1 << 22;

// Lanes a row and values a lane for E experts.
#define MXQ_ROUTE_SHAPE(E, CALL)         \
    do {                                 \
        if ((E) <= 64) CALL(16, 1);      \
        else if ((E) <= 128) CALL(16, 2);\
        else if ((E) <= 256) CALL(16, 4);\
        else if ((E) <= 512) CALL(64, 2);\
        else CALL(64, 4);                \
    } while (0)

unsigned route_grid(int64_t M, int L)
{
    const int64_t rows = kRouteThreads / L;
    const int64_t n = (M + rows - 1) / rows;
    return (unsigned)(n < kRouteMaxGrid ? n : kRouteMaxGrid);
}

}  // namespace

int route_max_experts() { return kRouteMaxExperts; }
int route_max_topk() { return kRouteMaxTopk; }

hipError_t launch_route_topk(const void* logits, bool f32, int64_t M, int E, const float* bias, bool sigmoid,
                             int n_groups, int topk_groups, int topk, bool renorm, bool top2, float scale,
                             int32_t* ids, float* weights, hipStream_t stream)
{
    RouteArgs a;
    a.E = E;
    a.n_groups = topk_groups < n_groups ? n_groups : 1;           // all groups stay: no groups
    a.topk_groups = topk_groups;
    a.topk = topk;
    a.group_size = E / n_groups;
    a.group_magic = a.group_size > 1 ? (uint32_t)((((uint64_t)1 << 32) + (uint32_t)a.group_size - 1) / (uint32_t)a.group_size) : 0u;
    a.scale = scale;
    a.renorm = renorm;
    a.top2 = top2;
#define MXQ_LAUNCH(F, S, L, C)                                                                                      \
    hipLaunchKernelGGL((route_topk_kernel<F, S, L, C>), dim3(route_grid(M, L)), dim3(kRouteThreads), 0, stream,     \
                       logits, bias, M, a, ids, weights)
#define MXQ_CALL(L, C)                                                       \
    do {                                                                     \
        if (f32 && sigmoid) MXQ_LAUNCH(true, true, L, C);                    \
        else if (f32) MXQ_LAUNCH(true, false, L, C);                         \
        else if (sigmoid) MXQ_LAUNCH(false, true, L, C);                     \
        else MXQ_LAUNCH(false, false, L, C);                                 \
    } while (0)
    MXQ_ROUTE_SHAPE(E, MXQ_CALL);
#undef MXQ_CALL
#undef MXQ_LAUNCH
    return hipGetLastError();
}

hipError_t launch_route_topk_bwd(const void* logits, bool f32, int64_t M, int E, bool sigmoid, const int32_t* ids,
                                 int topk, bool renorm, float scale, const float* dweights, void* dlogits,
                                 hipStream_t stream)
{
#define MXQ_LAUNCH(F, S, L, C)                                                                                        \
    hipLaunchKernelGGL((route_topk_bwd_kernel<F, S, L, C>), dim3(route_grid(M, L)), dim3(kRouteThreads), 0, stream,   \
                       logits, ids, dweights, M, E, topk, renorm, scale, dlogits)
#define MXQ_CALL(L, C)                                                       \
    do {                                                                     \
        if (f32 && sigmoid) MXQ_LAUNCH(true, true, L, C);                    \
        else if (f32) MXQ_LAUNCH(true, false, L, C);                         \
        else if (sigmoid) MXQ_LAUNCH(false, true, L, C);                     \
        else MXQ_LAUNCH(false, false, L, C);                                 \
    } while (0)
    MXQ_ROUTE_SHAPE(E, MXQ_CALL);
#undef MXQ_CALL
#undef MXQ_LAUNCH
    return hipGetLastError();
}

}  // namespace mxq
