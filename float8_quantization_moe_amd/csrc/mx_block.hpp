// mx_block.hpp -- the MXFP8 encoder of one 16-byte chunk of bf16, shared by the
// codec, the dispatch pack and the norm (all three write the same bytes).
#pragma once

#include "device_common.hpp"

namespace mxq {

// One 16-byte chunk (8 bf16) -> 8 E4M3 codes; returns the block's E8M0 code in *scode.
// RCEIL selects the round-up scale rule (see mx_scale_code).
template <bool RCEIL>
__device__ __forceinline__ uint2 quantize_chunk(uint4 v, uint32_t* scode)
{
    const uint32_t m0 = v.x & 0x7FFF7FFFu, m1 = v.y & 0x7FFF7FFFu;
    const uint32_t m2 = v.z & 0x7FFF7FFFu, m3 = v.w & 0x7FFF7FFFu;
    const uint32_t pm = pk_max_u16(pk_max_u16(m0, m1), pk_max_u16(m2, m3));
    uint32_t amax = (pm & 0xFFFFu) > (pm >> 16) ? (pm & 0xFFFFu) : (pm >> 16);
    amax = quad_max_u32(amax);

    const uint32_t code = mx_scale_code<RCEIL>(amax);
    if (amax >= 0x7F80u) {                       // Inf or NaN in the block
        *scode = 0xFFu;
        return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    *scode = code;
    // Saturation bound 448 * 2^(code-127) as a bf16 magnitude, in both halves.
    const uint32_t L = ((code + 8u) << 7) | 0x60u;
    const uint32_t LL = L | (L << 16);
    const float scale = pow2_from_biased(code);
    const uint32_t t0 = (v.x & 0x80008000u) | pk_min_u16(m0, LL);
    const uint32_t t1 = (v.y & 0x80008000u) | pk_min_u16(m1, LL);
    const uint32_t t2 = (v.z & 0x80008000u) | pk_min_u16(m2, LL);
    const uint32_t t3 = (v.w & 0x80008000u) | pk_min_u16(m3, LL);
    v2i16 lo = {0, 0}, hi = {0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(v2bf16, t0), scale, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(v2bf16, t1), scale, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(v2bf16, t2), scale, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(v2bf16, t3), scale, true);
    return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

}  // namespace mxq
