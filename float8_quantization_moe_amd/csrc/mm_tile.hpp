// mm_tile.hpp -- what the products' tile kernels share (gfx950): loads straight into LDS and
// the barrier that waits for them, a scan over a workgroup, and the lane order of whole-line
// stores.  A workgroup is four waves.
#pragma once

#include "device_common.hpp"

#include <type_traits>

namespace mxq {

constexpr int kTileThreads = 256;

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t* LdsPtr;

template <int V>
using Int = std::integral_constant<int, V>;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Buffer resource: base, stride 0, size in bytes (loads past it return zeros).
__device__ __forceinline__ v4i resource(const void* base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    v4i r = {uniform((int)(uint32_t)b), uniform((int)(uint32_t)(b >> 32)), uniform((int)bytes), 0x00020000};
    return r;
}

// Buffer load straight into LDS: lane l's 16 bytes land at lds + 16 l.  Counted by
// vmcnt, which slot_barrier waits on; in asm so that the compiler adds no wait of
// its own before later LDS reads.  Nor does it add the wait states that such a load
// needs inside an asm block: one after M0 is written, and five after a vector
// instruction (a v_readlane that fetches a spilled resource) has written a scalar
// register that the load reads.  s_mov and s_nop WAIT are WAIT + 2 of them.  MXFP4 scales,
// whose resources the compiler spills, take all five; five at every load took 1 % longer
// (16640 rows in 16 groups 558 / 396 us against 553 / 393).  A test reads the assembly.
template <int WAIT = 0>
__device__ __forceinline__ void load_to_lds(const v4i& srd, uint32_t lds, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop %3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(srd),
                 "n"(WAIT)
                 : "memory");
}

// At most N of this wave's loads are still under way (the last ones issued) and its
// LDS reads are done; then meet the other waves.
template <int N>
__device__ __forceinline__ void slot_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Inclusive scan over the workgroup's threads (maximum or sum) through sh.
template <bool MAX>
__device__ int block_scan(int v, int* sh)
{
    const int t = (int)threadIdx.x;
    v = MAX ? wave_incl_max(v) : wave_incl_sum(v);
    if ((t & 63) == 63) sh[t >> 6] = v;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < (t >> 6); ++w) before = MAX ? (sh[w] > before ? sh[w] : before) : before + sh[w];
    __syncthreads();
    return MAX ? (v > before ? v : before) : v + before;
}

// Four 16-byte pieces a lane, piece s of lane (r, h) at byte 32 s + 16 h of row r of a
// 32-row, 128-byte block, change lanes so that piece s lies in row 16 (s % 2) +
// 8 (s / 2) + r % 8 at byte 64 (r / 8 % 2) + 32 (r / 16) + 16 h: a store then covers
// whole lines.  (Pieces 0 and 1, 2 and 3 swap between rows of 16 lanes, then 0 and 2,
// 1 and 3 between halves of 16.)
__device__ __forceinline__ void join_lines(v4i (&p)[4])
{
    constexpr int kRor8 = 0x128;                         // lane ^ 8, within 16 lanes
#pragma unroll
    for (int s = 0; s < 4; s += 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const auto v = __builtin_amdgcn_permlane16_swap((uint32_t)p[s][k], (uint32_t)p[s + 1][k], false, false);
            p[s][k] = (int)v[0];
            p[s + 1][k] = (int)v[1];
        }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int lo = p[s][k], hi = p[s + 2][k];
            p[s][k] = __builtin_amdgcn_update_dpp(lo, hi, kRor8, 0xf, 0xc, false);
            p[s + 2][k] = __builtin_amdgcn_update_dpp(hi, lo, kRor8, 0xf, 0x3, false);
        }
}

}  // namespace mxq
