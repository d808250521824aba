// mxfp4_codec.hip -- MXFP4 quantize / dequantize of a bf16 tensor on gfx950.
//
// MXFP4 (OCP Microscaling v1.0): blocks of 32 consecutive elements of a row share
// one E8M0 scale; an element is an E2M1 code (sign, two exponent bits of bias 1,
// one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the even element
// in the low nibble.
//
//   scale code  floor rule: floor(log2 amax) - 2, so amax / scale lies in [4, 8);
//               round-up rule: the smallest e with amax <= 6 * 2^e.
//   element     x / scale (exact), rounded once to the nearest E2M1 value, ties
//               to even, saturating at 6.  This is the one rounding to 4 bits.
//
// Both kernels are flat streaming passes (HBM bound, no reuse), built as the
// MXFP8 codec's: a lane owns one 16-byte chunk of bf16 (8 elements) a step, four
// consecutive lanes own one block, so a wave reads 1 KB and writes 256 B in
// whole runs; the block maximum is an integer maximum finished across the quad
// with DPP.  The hardware converters take the scale as an operand; they round to
// nearest even and saturate.
#include "device_common.hpp"
#include "internal.hpp"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;        // independent chunks in flight per lane

// E8M0 code of a block whose largest |bf16| bit pattern is amax (finite).  With E
// its biased exponent, 6 * 2^(E-127-2) is 1.5 * 2^(E-127): the round-up rule
// needs one more when the significand passes 1.5 (mantissa bits > 0x40).  Both
// rules clamp at code 0 (zero, subnormal or tiny maxima).
template <bool RCEIL>
__device__ __forceinline__ uint32_t fp4_scale_code(uint32_t amax)
{
    const uint32_t E = (amax >> 7) + (RCEIL && (amax & 0x7Fu) > 0x40u ? 1u : 0u);
    return E > 2u ? E - 2u : 0u;
}

// 8 bf16 -> 8 E2M1 codes; the block's E8M0 code in *scode.
template <bool RCEIL>
__device__ __forceinline__ uint32_t quantize_chunk4(uint4 v, uint32_t* scode)
{
    const uint32_t m0 = v.x & 0x7FFF7FFFu, m1 = v.y & 0x7FFF7FFFu;
    const uint32_t m2 = v.z & 0x7FFF7FFFu, m3 = v.w & 0x7FFF7FFFu;
    const uint32_t pm = pk_max_u16(pk_max_u16(m0, m1), pk_max_u16(m2, m3));
    uint32_t amax = (pm & 0xFFFFu) > (pm >> 16) ? (pm & 0xFFFFu) : (pm >> 16);
    amax = quad_max_u32(amax);
    if (amax >= 0x7F80u) {                       // Inf or NaN in the block
        *scode = 0xFFu;
        return 0u;
    }
    const uint32_t code = fp4_scale_code<RCEIL>(amax);
    *scode = code;
    const float scale = pow2_from_biased(code);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf16, v.x), scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf16, v.y), scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf16, v.z), scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf16, v.w), scale, 3);
    return q;
}

template <bool RCEIL>
__global__ __launch_bounds__(kThreads)
void mxfp4_quantize_kernel(const uint4* __restrict__ x, uint32_t* __restrict__ q, uint8_t* __restrict__ s,
                           int64_t nchunks)
{
    const int64_t per_block = (int64_t)kThreads * kUnroll;
    for (int64_t base = (int64_t)blockIdx.x * per_block + threadIdx.x; base < nchunks;
         base += (int64_t)gridDim.x * per_block) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = base + (int64_t)u * kThreads;
            v[u] = c < nchunks ? load_nt(x + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = base + (int64_t)u * kThreads;
            uint32_t code;
            const uint32_t out = quantize_chunk4<RCEIL>(v[u], &code);   // whole quads are in or out of range
            if (c < nchunks) {
                __builtin_nontemporal_store(out, q + c);
                if ((threadIdx.x & 3) == 0) s[c >> 2] = (uint8_t)code;
            }
        }
    }
}

// 8 E2M1 codes of one block (scale code sc) -> 8 bf16.  code * 2^(sc-127) is
// exact in bf16 except past its largest value (6 * 2^126 and up: Inf); a NaN
// scale makes every element NaN.
__device__ __forceinline__ uint4 dequantize_chunk4(uint32_t q, uint32_t sc)
{
    const float scale = pow2_from_biased(sc);
    const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
    const uint32_t c = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
    const uint32_t d = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
    return sc == 0xFFu ? make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u) : make_uint4(a, b, c, d);
}

__global__ __launch_bounds__(kThreads)
void mxfp4_dequantize_kernel(const uint32_t* __restrict__ q, const uint8_t* __restrict__ s, uint4* __restrict__ y,
                             int64_t nchunks)
{
    const int64_t per_block = (int64_t)kThreads * kUnroll;
    for (int64_t base = (int64_t)blockIdx.x * per_block + threadIdx.x; base < nchunks;
         base += (int64_t)gridDim.x * per_block) {
        uint32_t qv[kUnroll], sc[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = base + (int64_t)u * kThreads;
            const bool in = c < nchunks;
            qv[u] = in ? __builtin_nontemporal_load(q + c) : 0u;
            sc[u] = in ? (uint32_t)s[c >> 2] : 0u;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = base + (int64_t)u * kThreads;
            if (c < nchunks) store_nt(dequantize_chunk4(qv[u], sc[u]), y + c);
        }
    }
}

unsigned flat_grid(int64_t nchunks)
{
    const int64_t per_block = (int64_t)kThreads * kUnroll;
    const int64_t blocks = (nchunks + per_block - 1) / per_block;
    const int64_t cap = 1 << 22;
    return (unsigned)(blocks < cap ? blocks : cap);
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int64_t M, int64_t K, void* q, void* s, bool rceil,
                                 hipStream_t stream)
{
    const int64_t nchunks = M * K / 8;
    if (rceil)
        hipLaunchKernelGGL(mxfp4_quantize_kernel<true>, dim3(flat_grid(nchunks)), dim3(kThreads), 0, stream,
                           (const uint4*)x, (uint32_t*)q, (uint8_t*)s, nchunks);
    else
        hipLaunchKernelGGL(mxfp4_quantize_kernel<false>, dim3(flat_grid(nchunks)), dim3(kThreads), 0, stream,
                           (const uint4*)x, (uint32_t*)q, (uint8_t*)s, nchunks);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const void* q, const void* s, int64_t M, int64_t K, void* y, hipStream_t stream)
{
    const int64_t nchunks = M * K / 8;
    hipLaunchKernelGGL(mxfp4_dequantize_kernel, dim3(flat_grid(nchunks)), dim3(kThreads), 0, stream,
                       (const uint32_t*)q, (const uint8_t*)s, (uint4*)y, nchunks);
    return hipGetLastError();
}

}  // namespace mxq
