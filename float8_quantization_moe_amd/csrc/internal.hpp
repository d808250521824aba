// internal.hpp -- launchers shared between the kernel files and the C ABI layer.
// Arguments reaching these functions have already been validated by api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxq {

hipError_t launch_mx_quantize(const void* x, int64_t M, int64_t K, void* q, void* s, bool rceil, hipStream_t stream);
hipError_t launch_mx_dispatch_pack(const void* x, int64_t K, int32_t* src_pair, int topk, const int32_t* group_end,
                                   int E, void* packed, int64_t nrows, hipStream_t stream);
int dispatch_max_experts();
size_t dispatch_workspace_bytes(int64_t P, int32_t E);
// pair_row may be null.
hipError_t launch_dispatch_order(const int32_t* ids, int64_t P, int E, int32_t* src_pair, int32_t* pair_row,
                                 int32_t* group_end, void* workspace, hipStream_t stream);
hipError_t launch_mx_quantize_dim0(const void* x, int64_t M, int64_t K, void* q, void* s, bool rceil,
                                   hipStream_t stream);
hipError_t launch_mx_dequantize_dim0(const void* q, const void* s, int64_t M, int64_t K, void* y,
                                     hipStream_t stream);
hipError_t launch_mx_dequantize(const void* q, const void* s, int64_t M, int64_t K, void* y, hipStream_t stream);

bool group_scale_sizes_ok(int64_t M, int64_t K, int64_t G);
size_t group_scale_workspace_bytes(int64_t M, int64_t K, int32_t G);
bool group_split_sizes_ok(int64_t M, int64_t K, int64_t G);
size_t group_split_workspace_bytes(int64_t M, int64_t K, int32_t G);
hipError_t launch_group_split(const void* x, int M, int K, const int32_t* offs, int G, int layout, int flags, void* q,
                              float* scales, void* workspace, hipStream_t stream);
// Route overrides for tests (process-wide): method 0 auto, 1 hold, 2 two-pass, 3 split;
// hold_tiles < 0, wait_us < 0 and strip_block <= 0 select the defaults.
void set_group_scale_knobs(int method, int hold_tiles, long wait_us, int strip_block);
// The allocation-free variant's scratch: a static device array of this many
// bytes per device, its address on the current device.
constexpr size_t kNoAllocScratchBytes = (size_t)16 << 20;
hipError_t group_scale_scratch(void** ptr);
// The hold method's route counters of the last call that used this workspace
// (synchronises the stream).
hipError_t group_scale_route_counters(const void* workspace, int64_t M, int64_t K, int64_t G, int layout,
                                     uint32_t* out, hipStream_t stream);
hipError_t launch_group_scale(const void* x, int M, int K, const int32_t* offs, int G, int layout, int flags,
                              void* q, float* scales, void* workspace, hipStream_t stream);

int grouped_mm_max_groups();
bool grouped_mm_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t G);
size_t grouped_mm_workspace_bytes(int64_t M, int64_t N, int32_t G);
hipError_t launch_grouped_mm(const void* xq, const void* xs, const void* wq, const void* ws,
                             const int32_t* offs, int M, int N, int K, int G, void* y, bool f32_out,
                             void* workspace, hipStream_t stream);
// Token operand with explicit row strides in bytes (codes ldx, scales ldxs; both multiples of 16).
hipError_t launch_grouped_mm_strided(const void* xq, const void* xs, uint32_t ldx, uint32_t ldxs, const void* wq,
                                     const void* ws, const int32_t* offs, int M, int N, int K, int G, void* y,
                                     bool f32_out, void* workspace, hipStream_t stream);

// MXFP4: codec and grouped product.
hipError_t launch_mxfp4_quantize(const void* x, int64_t M, int64_t K, void* q, void* s, bool rceil,
                                 hipStream_t stream);
hipError_t launch_mxfp4_dequantize(const void* q, const void* s, int64_t M, int64_t K, void* y, hipStream_t stream);
bool mxfp4_mm_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t G);
// ldx, ldxs: row strides in bytes of the token codes (a multiple of 16) and scales (of 4).
hipError_t launch_mxfp4_mm(const void* xq, const void* xs, bool x8, int64_t ldx, int64_t ldxs, const void* wq,
                           const void* wsc, const int32_t* offs, int M, int N, int K, int G, void* y, bool f32_out,
                           hipStream_t stream);
// Its part for groups of many rows.
hipError_t launch_mxfp4_mm_tile(const void* xq, const void* xs, bool x8, int64_t ldx, int64_t ldxs, const void* wq,
                                const void* wsc, const int32_t* offs, int M, int N, int K, int G, void* y, bool f32_out,
                                hipStream_t stream);

// Norm: K at most norm_max_k(), a multiple of 8 (of 32 with q).
int norm_max_k();
hipError_t launch_add_rmsnorm(const void* x, const void* r, const void* w, bool f32, int64_t M, int64_t K, float eps,
                              void* h, void* y, void* q, void* s, float* rstd, hipStream_t stream);
size_t add_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K);
hipError_t launch_add_rmsnorm_bwd(const void* h, const void* w, const float* rstd, const void* dy, const void* dh,
                                  bool f32, int64_t M, int64_t K, void* dx, float* dw, void* workspace,
                                  hipStream_t stream);

// Layer norm, in the norm's sizes.
hipError_t launch_add_layernorm(const void* x, const void* r, const void* w, const void* b, bool f32, int64_t M, int64_t K,
                                float eps, void* h, void* y, void* q, void* s, float* mean, float* rstd, hipStream_t stream);
size_t add_layernorm_bwd_workspace_bytes(int64_t M, int64_t K);
hipError_t launch_add_layernorm_bwd(const void* h, const void* w, const float* mean, const float* rstd, const void* dy,
                                    const void* dh, bool f32, int64_t M, int64_t K, void* dx, float* dw, float* db,
                                    void* workspace, hipStream_t stream);

// Rows to their experts and back; row_bytes is a multiple of 16.
hipError_t launch_dispatch_rows(const void* x, int64_t row_bytes, int64_t M, int topk, const int32_t* pair_row,
                                const int32_t* group_end, int E, void* rows, int32_t* src_pair, hipStream_t stream);
hipError_t launch_pair_rows(const int32_t* src_pair, int64_t pairs, int32_t* pair_row, hipStream_t stream);
hipError_t launch_combine_rows(const void* rows, bool f32, int64_t R, int64_t K, const int32_t* pair_row, int64_t M, int topk,
                               const float* weights, void* out, hipStream_t stream);
hipError_t launch_combine_rows_bwd(const void* dout, const void* rows, bool f32, int64_t R, int64_t K, const int32_t* pair_row,
                                   int64_t M, int topk, const float* weights, void* drows, float* dweights,
                                   hipStream_t stream);

// Grouped products in bf16; product is an mxq_product.
bool bf16_mm_sizes_ok(int product, int64_t M, int64_t N, int64_t K, int64_t G);
size_t bf16_mm_workspace_bytes(int product, int64_t M, int64_t N, int64_t K, int64_t G);
hipError_t launch_bf16_mm(int product, const void* rows, const void* other, const int32_t* offs, int M, int N, int K, int G,
                          void* out, bool f32_out, bool accumulate, void* workspace, hipStream_t stream);

// Their part for few rows and small results.  With a split above 1 out takes that many fp32 arrays of results, to be added.
int bf16_mm_few_split(int product, int M, int N, int K, int G);
hipError_t launch_bf16_mm_few(int product, const void* rows, const void* other, const int32_t* offs, int M, int N, int K, int G,
                              int split, void* out, bool f32_out, bool add, hipStream_t stream);

// Routing.
int route_max_experts();
int route_max_topk();
hipError_t launch_route_topk(const void* logits, bool f32, int64_t M, int E, const float* bias, bool sigmoid,
                             int n_groups, int topk_groups, int topk, bool renorm, bool top2, float scale,
                             int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_route_topk_bwd(const void* logits, bool f32, int64_t M, int E, bool sigmoid, const int32_t* ids,
                                 int topk, bool renorm, float scale, const float* dweights, void* dlogits,
                                 hipStream_t stream);

hipError_t launch_transpose_u8(const void* in, int64_t R, int64_t C, void* out, hipStream_t stream);

}  // namespace mxq
