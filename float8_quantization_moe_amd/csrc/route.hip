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
// All arithmetic is fp32.  The selection must not depend on how a row is spread over
// lanes, so a key uses nothing but correctly rounded operations on its own value
// and expf (and, for softmax with a bias, the row's sum).
//
// Forward layout: L lanes a row (8 lanes for E <= 64, so that a wave works on
// eight rows and each cross-lane step serves all eight; 16 up to 256; 64 beyond), each with
// 4 C values in registers: lane i holds experts 4 (i + L j) .. + 3.  A key and its
// index become one 64-bit number, ordered as the keys and then by falling index (a
// key of -inf: not eligible).  Each lane sorts its numbers once (a fixed network of f64 minima
// and maxima: the bit patterns compare as doubles) and keeps the list in LDS; a
// round of the selection is then the maximum of the lists' heads over the row's
// lanes, with DPP, and the winner steps to its next.  Reading the logits is the
// floor; VALU work is what bounds it (scores 17 and keys 10 instructions a value,
// the sort 5, a round 20 for four rows).
// 65536 x 128, sigmoid, bias, 4 of 8 groups, top-8: 26 us (8 lanes a row two more;
// rounds that searched the registers instead of sorted lists 33).
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

// 1 / x for x >= 1, correctly rounded: one Newton step from the hardware's
// reciprocal is exact for every float from 1 to 2^126 (checked one by one); past
// that the quotient is subnormal and takes the divide, and 1 / inf is 0.
__device__ __forceinline__ float reciprocal_step(float x)
{
    const float y = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, y, 1.0f), y, y);
}
__device__ __forceinline__ float sigmoid_of(float l)
{
    const float x = 1.0f + expf(-l);
    return x < 0x1p126f ? reciprocal_step(x) : 1.0f / x;
}
// The same for N values, with one branch.
template <int N>
__device__ __forceinline__ void sigmoids_of(const float (&l)[N], float (&s)[N])
{
    float x[N], most = 1.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = 1.0f + expf(-l[i]);
        most = fmaxf(most, x[i]);
        s[i] = reciprocal_step(x[i]);
    }
    if (most >= 0x1p126f) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (x[i] >= 0x1p126f) s[i] = 1.0f / x[i];
    }
}

// A sigmoid's derivative s (1 - s), in a form that does not cancel where s rounds to 1.
__device__ __forceinline__ float sigmoid_slope(float l)
{
    const float e = expf(-fabsf(l)), r = reciprocal_step(1.0f + e);
    return e * r * r;
}

// Key and index as one number; doubles of these bits are finite and in their order.
__device__ __forceinline__ double ranked(uint32_t key, uint32_t id)
{
    return __hiloint2double((int)(key >> 1), (int)((key << 31) | (1023u - id)));
}

constexpr uint32_t kNoKey = 0x007FFFFFu >> 1;             // the high word of -inf: not eligible

// Sorts v in falling order (odd-even merge network).
template <int N>
__device__ __forceinline__ void sort_falling(double (&v)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const double a = v[i + j], b = v[i + j + k];
                        v[i + j] = __builtin_fmax(a, b);
                        v[i + j + k] = __builtin_fmin(a, b);
                    }
}

// The LDS operations of one wave run in order: this keeps the compiler's order too.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The 4 logits of experts e0 .. e0+3 of a row; -inf past E.  `vec`: rows are
// aligned to 4 values (E % 4 == 0).
template <bool F32L>
__device__ __forceinline__ void load4(const void* row, int e0, int E, bool vec, float* v)
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
    int lanes_log2;              // log2 of the lanes that find one group's value
    float scale;
    bool renorm, top2;
};

// Rows are the work of single waves: no workgroup barrier.  A wave's LDS holds the
// groups' values first, then the lanes' sorted lists.
template <bool F32L, bool SIGMOID, int L, int C>
__global__ __launch_bounds__(kRouteThreads, C == 4 ? 3 : 5)      // (workgroups a CU; one more would spill)
void route_topk_kernel(const void* __restrict__ logits, const float* __restrict__ bias, int64_t M, RouteArgs a,
                       int32_t* __restrict__ ids, float* __restrict__ weights)
{
    constexpr int kRows = kRouteThreads / L;
    constexpr int NE = 4 * C, kMaxE = L * NE;
    constexpr int kSlots = (kRouteMaxTopk + L - 1) / L;          // slots a lane finishes at most
    __shared__ double lds[kRouteThreads * (NE + 1)];
    const int lane = (int)threadIdx.x % L, sub = (int)threadIdx.x / L;
    double* list = lds + threadIdx.x * (NE + 1);
    float* values = (float*)(lds + sub * L * (NE + 1));          // kMaxE values of the row, then of its groups
    float* gvalues = values + kMaxE;
    const int E = a.E;
    const bool vec = E % 4 == 0, bias_vec = ((uintptr_t)bias & 15u) == 0;
    const bool groups = a.n_groups > 1;
    // what all values of a row are needed for; the selected ones' scores are made again at the end
    const bool all_scores = bias != nullptr || groups, total_needed = !SIGMOID && (all_scores || !a.renorm);
    for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < M; m0 += (int64_t)gridDim.x * kRows) {
        const int64_t m = m0 + sub;
        const bool live = m < M;
        const uint8_t* row = (const uint8_t*)logits + (live ? m : M - 1) * E * (F32L ? 4 : 2);

        float l[NE], v[NE];
        bool bad = false;                                        // a NaN anywhere, or +inf under softmax
        float top = MXQ_NEG_INF;
#pragma unroll
        for (int j = 0; j < C; ++j) load4<F32L>(row, 4 * (lane + L * j), E, vec, l + 4 * j);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            bad |= l[i] != l[i] || (!SIGMOID && l[i] == -MXQ_NEG_INF);
            if constexpr (!SIGMOID) top = fmaxf(top, l[i]);
        }
        bad = lanes_max<L>(bad ? 1u : 0u) != 0;
        float total = 1.0f;
        if constexpr (SIGMOID) {
            if (all_scores) sigmoids_of<NE>(l, v);
        } else {
            top = lanes_max_f<L>(top);
            top = top > MXQ_NEG_INF ? top : 0.0f;
            if (total_needed) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    v[i] = expf(l[i] - top);
                    sum += v[i];
                }
                total = lanes_sum<L>(sum);
                total = total > 0.0f ? total : 1.0f;
            }
        }

        float key[NE];                                           // -inf: not eligible
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = l[i];
        if (bias) {                                              // (uniform)
            const float unit = SIGMOID ? 1.0f : 1.0f / total;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float b4[4];
                load4<true>(bias, 4 * (lane + L * j), E, vec && bias_vec, b4);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = 4 * j + c;
                    v[i] = (SIGMOID ? v[i] : v[i] * unit) + b4[c];
                    key[i] = v[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = l[i] > MXQ_NEG_INF && key[i] > MXQ_NEG_INF ? key[i] : MXQ_NEG_INF;   // (NaN too)

        if (groups) {                                            // (uniform)
            // each lane's four neighbours are of one group if that has a multiple of 4: then
            // their two largest go to LDS, else all four
            const bool quads = a.group_size % 4 == 0;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] = key[4 * j + c] > MXQ_NEG_INF ? v[4 * j + c] : MXQ_NEG_INF;
                if (quads) {
                    const float a1 = fmaxf(w[0], w[1]), a2 = fminf(w[0], w[1]), b1 = fmaxf(w[2], w[3]), b2 = fminf(w[2], w[3]);
                    ((float2*)values)[lane + L * j] = make_float2(fmaxf(a1, b1), fmaxf(fminf(a1, b1), fmaxf(a2, b2)));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) values[4 * (lane + L * j) + c] = w[c];
                }
            }
            wave_order();
            // 2^lg lanes a group, each every 2^lg-th of its entries, from a place of its own on:
            // groups of 16 or more floats start in the same few banks (32768 x 256, 8 groups:
            // 34.7 -> 27.2 us; 16384 x 512: 31.0 -> 27.9)
            const int lg = a.lanes_log2, P = 1 << lg, entries = quads ? a.group_size / 4 : a.group_size;
            for (int g0 = lane >> lg; g0 - (lane >> lg) < a.n_groups; g0 += L >> lg) {
                const int g = g0 < a.n_groups ? g0 : 0, p = lane & (P - 1);
                const int n = (entries - p + P - 1) >> lg;
                float v1 = MXQ_NEG_INF, v2 = MXQ_NEG_INF;
                int at = n > 0 ? lane_id() % n : 0;
#pragma unroll 2
                for (int i = 0; i < n; ++i) {
                    const int k = g * entries + p + (at << lg);
                    const float2 t = quads ? ((const float2*)values)[k] : make_float2(values[k], MXQ_NEG_INF);
                    at = at + 1 < n ? at + 1 : 0;
                    v2 = fmaxf(fmaxf(v2, t.y), fminf(v1, t.x));
                    v1 = fmaxf(v1, t.x);
                }
                for (int d = 1; d < P; d *= 2) {
                    const float o1 = __shfl_xor(v1, d), o2 = __shfl_xor(v2, d);
                    v2 = fmaxf(fmaxf(v2, o2), fminf(v1, o1));
                    v1 = fmaxf(v1, o1);
                }
                if (p == 0 && g0 < a.n_groups) gvalues[g] = a.top2 && v2 > MXQ_NEG_INF ? v1 + v2 : v1;
            }
            wave_order();
            // a group stays if fewer than topk_groups precede it; `values` becomes the flag
            for (int g = lane; g < a.n_groups; g += L) {
                const float t = gvalues[g];
                int before = 0;
#pragma unroll 4
                for (int i = 0; i < a.n_groups; ++i) {
                    const float u = gvalues[i];
                    before += u > t || (u == t && i < g) ? 1 : 0;
                }
                values[g] = before < a.topk_groups ? 1.0f : 0.0f;
            }
            wave_order();
            // (experts past E look at a group past the last: they are not eligible anyway)
            if (a.group_size % 4 == 0) {                         // four neighbours are of one group
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const bool out = values[__umulhi((uint32_t)(4 * (lane + L * j)), a.group_magic)] == 0.0f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) key[4 * j + c] = out ? MXQ_NEG_INF : key[4 * j + c];
                }
            } else {
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    const uint32_t e = (uint32_t)(4 * (lane + L * (i / 4)) + i % 4);
                    const uint32_t g = a.group_size > 1 ? __umulhi(e, a.group_magic) : e;
                    key[i] = values[g] == 0.0f ? MXQ_NEG_INF : key[i];
                }
            }
            wave_order();
        }

        double r[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) r[i] = ranked(order_key(key[i]), (uint32_t)(4 * (lane + L * (i / 4)) + i % 4));
        sort_falling<NE>(r);
#pragma unroll
        for (int i = 1; i < NE; ++i) list[i] = r[i];
        list[NE] = 0.0;
        wave_order();

        int slot[kSlots];
        uint32_t hi = (uint32_t)__double2hiint(r[0]), lo = (uint32_t)__double2loint(r[0]);
        int at = 0;
#pragma unroll
        for (int tb = 0; tb < kSlots; ++tb) {
            slot[tb] = -1;
            const int n = a.topk - tb * L < L ? a.topk - tb * L : L;
            for (int t = 0; t < n; ++t) {
                const uint32_t best = lanes_max<L>(hi);
                const uint32_t which = lanes_max<L>(hi == best ? lo : 0u);
                if (lane == t && best > kNoKey) slot[tb] = (int)(1023u - (which & 1023u));
                if (hi == best && lo == which) {             // (the list's end is 0, and 0 wins over nothing)
                    ++at;
                    const double next = list[at];
                    hi = (uint32_t)__double2hiint(next);
                    lo = (uint32_t)__double2loint(next);
                }
            }
        }

        float s[kSlots], sum = 0.0f;
#pragma unroll
        for (int tb = 0; tb < kSlots; ++tb) {
            s[tb] = 0.0f;
            if (slot[tb] >= 0) {
                float x;
                if constexpr (F32L) x = ((const float*)row)[slot[tb]];
                else x = bf16_lo_to_f32(((const uint16_t*)row)[slot[tb]]);
                s[tb] = SIGMOID ? sigmoid_of(x) : expf(x - top) / total;
            }
            sum += s[tb];
        }
        sum = lanes_sum<L>(sum) + kTiny;
#pragma unroll
        for (int tb = 0; tb < kSlots; ++tb) {
            const int t = lane + L * tb;
            float w = s[tb];
            if (a.renorm) w /= sum;
            w *= a.scale;
            if (bad) w = __builtin_nanf("");
            if (live && t < a.topk) {
                ids[m * a.topk + t] = slot[tb];
                weights[m * a.topk + t] = w;
            }
        }
        wave_order();
    }
}

// Gradient.  With u_j the incoming gradient of weight j and s the scores:
//   g_j = scale * u_j, or, renormalised with D = sum of the selected s + 1e-20,
//         (scale * u_j - sum_i scale * u_i s_i / D) / D;
//   sigmoid: dl_e = s_e (1 - s_e) g_e at the selected experts, 0 elsewhere;
//   softmax: dl_e = s_e (g_e - sum_j g_j s_j) everywhere (g = 0 where not selected).
// Softmax with renormalisation, in terms that do not cancel: q = the softmax over the
// selected logits alone, S = the sum of their s, D = S + 1e-20, m = sum_j scale u_j q_j;
// then sum_j g_j s_j = m (S / D) (1e-20 / D) and
//   dl_e = q_e (S / D) (scale u_e - m + m 1e-20 / D)  where selected, and everywhere
//          - s_e m (S / D) (1e-20 / D).
// That is q's own gradient unless S is as small as 1e-20, which takes a bias or groups
// that keep a row's large logits out.
// Bound by a row's dependent steps rather than its bytes: 65536 x 64 bf16, top-6, softmax
// 8.0 us (bytes 3.4), renormalised 8.7; 65536 x 128 fp32, top-8, renormalised softmax 15.8
// (11.4), sigmoid 12.0.
// Same layout as the forward, rows are the work of single waves; the selected experts'
// g pass through LDS.
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
    for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < M; m0 += (int64_t)gridDim.x * kRows) {
        const int64_t m = m0 + sub;
        const bool live = m < M;
        const int64_t mr = live ? m : M - 1;
        const uint8_t* row = (const uint8_t*)logits + mr * E * (F32L ? 4 : 2);

        float l[C][4], p[C][4];
        float top = MXQ_NEG_INF, total = 1.0f;
        if constexpr (!SIGMOID) {
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
            total = total == 0.0f ? 1.0f : total;                 // (a NaN stays: the whole row's gradient is NaN)
        }
        const float unit = 1.0f / total;                          // (one rounding more than dividing: 2^-24 of the value)
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
            if (L * i < topk && t < topk) {                       // (the first is uniform)
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
        // softmax, renormalised: the selected scores are q times their sum, and `first` is the
        // score of the largest of them
        float sum = 0.0f, dot = 0.0f, first = 0.0f;
        float seltotal = total;
        if constexpr (!SIGMOID) {
            if (renorm) {                                         // (uniform)
                seltop = lanes_max_f<L>(seltop);
                if (seltop > MXQ_NEG_INF) first = expf(seltop - top) * unit;
                top = seltop > MXQ_NEG_INF ? seltop : 0.0f;
                seltotal = 1.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            sc[i] = 0.0f;
            if (L * i < topk && id[i] >= 0) sc[i] = SIGMOID ? sigmoid_of(ls[i]) : expf(ls[i] - top) / seltotal;
            sum += sc[i];
            dot += g[i] * sc[i];
        }
        sum = lanes_sum<L>(sum) + kTiny;
        dot = lanes_sum<L>(dot);
        float kept = 1.0f, tiny = 0.0f, rest = dot;               // rest: what s_e is multiplied by everywhere
        if constexpr (!SIGMOID) {
            if (renorm) {                                         // (uniform)
                const float D = first * sum + kTiny;
                kept = first * sum / D;
                tiny = dot / sum * (kTiny / D);
                rest = tiny * kept;
            }
        }
        wave_order();
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (L * i < topk && id[i] >= 0) {
                float d = g[i];
                if (renorm) d = (d - dot / sum + tiny) / sum;
                if (SIGMOID) d *= sigmoid_slope(ls[i]);
                else if (renorm) d *= sc[i] * kept;
                grad[sub][id[i]] = d;
            }
        wave_order();
        if (live) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int e0 = 4 * (lane + L * j);
                float d[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    d[c] = grad[sub][e0 + c];
                    if constexpr (!SIGMOID) d[c] = renorm ? d[c] - p[j][c] * unit * rest : p[j][c] * unit * (d[c] - rest);
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
        wave_order();
    }
}

constexpr int64_t kRouteMaxGrid = 1 << 22;

// Lanes a row and values a lane for E experts.
#define MXQ_ROUTE_SHAPE(E, CALL)         \
    do {                                 \
        if ((E) <= 32) CALL(8, 1);       \
        else if ((E) <= 64) CALL(8, 2);  \
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
        a.lanes_log2 = 0;                                                    \
        while ((2 << a.lanes_log2) * a.n_groups <= L) ++a.lanes_log2;        \
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
