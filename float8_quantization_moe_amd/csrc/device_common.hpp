// device_common.hpp -- small device helpers shared by the libmxq kernels (gfx950).
//
// Conversions used by the kernels (their rounding was checked exhaustively
// against the reference encoder: every bf16 pattern x every E8M0 scale code for
// quantization, every E4M3 code x every scale code for dequantization):
//   v_cvt_scalef32_pk_fp8_bf16  bf16 pair / 2^e  -> E4M3 pair, nearest-even, no saturation
//   v_cvt_pk_fp8_f32            fp32 pair        -> E4M3 pair, nearest-even, no saturation
//   v_cvt_scalef32_pk_bf16_fp8  E4M3 pair * 2^e  -> bf16 pair, nearest-even, subnormals kept
// "No saturation" means a magnitude that rounds past 448 becomes NaN, so every
// quantizing path clamps to +-448 (times the block scale) before converting.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

typedef short v2i16 __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));

constexpr int kWave = 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Streaming (non-temporal) 16- and 8-byte global accesses.
__device__ __forceinline__ uint4 load_nt(const uint4* p)
{
    const u32x4 v = __builtin_nontemporal_load((const u32x4*)p);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 load_nt(const uint2* p)
{
    const u32x2 v = __builtin_nontemporal_load((const u32x2*)p);
    return make_uint2(v.x, v.y);
}
__device__ __forceinline__ void store_nt(uint4 v, uint4* p)
{
    const u32x4 w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, (u32x4*)p);
}
__device__ __forceinline__ void store_nt(uint2 v, uint2* p)
{
    const u32x2 w = {v.x, v.y};
    __builtin_nontemporal_store(w, (u32x2*)p);
}

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b)
{
    v2u16 r = __builtin_elementwise_max(__builtin_bit_cast(v2u16, a), __builtin_bit_cast(v2u16, b));
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint32_t pk_min_u16(uint32_t a, uint32_t b)
{
    v2u16 r = __builtin_elementwise_min(__builtin_bit_cast(v2u16, a), __builtin_bit_cast(v2u16, b));
    return __builtin_bit_cast(uint32_t, r);
}

// binary32 with the biased exponent e (1..254) and zero mantissa; e == 0 gives 2^-127.
__device__ __forceinline__ float pow2_from_biased(uint32_t e)
{
    return __uint_as_float(e ? (e << 23) : 0x00400000u);
}

// E8M0 code of a block whose largest |bf16| bit pattern is amax (finite).  E is
// amax's biased exponent, so floor(log2 amax) = E - 127 for normal amax.
//   floor rule (OCP MX v1.0): floor(log2 amax) - 8, i.e. code E - 8.
//   RCEIL: the smallest e with amax <= 448 * 2^e.  448 * 2^(E-127-8) is 1.75 *
//     2^(E-127), so e is E - 135 when amax's significand is at most 1.75
//     (mantissa bits <= 0x60) and one more otherwise: code E - 8 + (m > 0x60).
// Both clamp at code 0 (amax zero, subnormal or below the smallest scale).
template <bool RCEIL>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax)
{
    const uint32_t E = (amax >> 7) + (RCEIL && (amax & 0x7Fu) > 0x60u ? 1u : 0u);
    return E > 8u ? E - 8u : 0u;
}

__device__ __forceinline__ float bf16_lo_to_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi_to_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Max over each aligned quad of lanes (DPP quad permutations).
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v)
{
    uint32_t t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);  // [1,0,3,2]
    v = v > t ? v : t;
    t = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);           // [2,3,0,1]
    return v > t ? v : t;
}

// ------------------------------------------------- reductions across lanes --
// One DPP move of all 64 lanes (every lane must be active).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;               // quad permutations
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;     // reversed within 8 and within 16 lanes

// Reduction over each aligned run of L lanes (L = 8, 16 or 64), the result in all
// of them.  A fixed order, so floating sums are reproducible; no LDS.
template <int L, class F>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, F op)
{
    static_assert(L == 8 || L == 16 || L == 64, "");
    v = op(v, dpp_move<kDppXor1>(v));
    v = op(v, dpp_move<kDppXor2>(v));
    v = op(v, dpp_move<kDppHalfMirror>(v));
    if constexpr (L > 8) v = op(v, dpp_move<kDppMirror>(v));
    if constexpr (L == 64) {
        const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
        const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
        const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
        const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
        v = op(op(a, b), op(c, d));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// --------------------------------------------- 8 values of bf16 or fp32 --
// kBytes of one value; load8 / store8 move values 8i .. 8i+7 of a row.
__device__ __forceinline__ uint32_t f32_pair_to_bf16(float lo, float hi)
{
    const v2bf16 t = {(__bf16)lo, (__bf16)hi};        // nearest even
    return __builtin_bit_cast(uint32_t, t);
}
struct Bf16 {
    static constexpr int kBytes = 2;
    struct Raw { uint4 a; };
    static __device__ __forceinline__ Raw load8(const void* row, int64_t i) { return {((const uint4*)row)[i]}; }
    static __device__ __forceinline__ Raw load8_nt(const void* row, int64_t i) { return {load_nt((const uint4*)row + i)}; }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[8])
    {
        const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo_to_f32(w[i]);
            v[2 * i + 1] = bf16_hi_to_f32(w[i]);
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[8])
    {
        return {make_uint4(f32_pair_to_bf16(v[0], v[1]), f32_pair_to_bf16(v[2], v[3]), f32_pair_to_bf16(v[4], v[5]),
                           f32_pair_to_bf16(v[6], v[7]))};
    }
    static __device__ __forceinline__ void store8(void* row, int64_t i, const Raw& r) { store_nt(r.a, (uint4*)row + i); }
    // the bf16 values of a packed chunk
    static __device__ __forceinline__ uint4 bf16_bits(const Raw& r) { return r.a; }
};
struct F32 {
    static constexpr int kBytes = 4;
    struct Raw { uint4 a, b; };
    static __device__ __forceinline__ Raw load8(const void* row, int64_t i)
    {
        return {((const uint4*)row)[2 * i], ((const uint4*)row)[2 * i + 1]};
    }
    static __device__ __forceinline__ Raw load8_nt(const void* row, int64_t i)
    {
        return {load_nt((const uint4*)row + 2 * i), load_nt((const uint4*)row + 2 * i + 1)};
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[8])
    {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ Raw pack(const float (&v)[8])
    {
        return {make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])),
                make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]))};
    }
    static __device__ __forceinline__ void store8(void* row, int64_t i, const Raw& r)
    {
        store_nt(r.a, (uint4*)row + 2 * i);
        store_nt(r.b, (uint4*)row + 2 * i + 1);
    }
    static __device__ __forceinline__ uint4 bf16_bits(const Raw& r)
    {
        float v[8];
        unpack(r, v);
        return Bf16::pack(v).a;
    }
};

// Non-zero in each byte lane of the result whose input byte is 0x7F or 0xFF.
__device__ __forceinline__ uint32_t nan_code_bytes(uint32_t q)
{
    uint32_t t = q & 0x7F7F7F7Fu;
    return (t + 0x01010101u) & 0x80808080u;
}

// ------------------------------------------------------------------ scans --
__device__ __forceinline__ int lane_id() { return (int)(threadIdx.x & (kWave - 1)); }

__device__ __forceinline__ int wave_incl_max(int v)
{
    const int lane = lane_id();
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        int t = __shfl_up(v, d, kWave);
        if (lane >= d) v = v > t ? v : t;
    }
    return v;
}

__device__ __forceinline__ int wave_incl_sum(int v)
{
    const int lane = lane_id();
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        int t = __shfl_up(v, d, kWave);
        if (lane >= d) v += t;
    }
    return v;
}

// wave_incl_max of non-negative values with DPP alone (no LDS round trips).
__device__ __forceinline__ int wave_incl_max_dpp(int v)
{
    auto up = [](int x, int moved) { return moved > x ? moved : x; };      // (lanes with no source get 0)
    v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
    v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
    v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
    v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
    v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));   // lane 15 of rows 0, 2 to rows 1, 3
    v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));   // lane 31 to rows 2 and 3
    return v;
}

__device__ __forceinline__ int readlane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

}  // namespace mxq
