"""Python binding of libmxq (ctypes): argument marshalling only.

Every function has the name of the C entry point it calls (see include/mxq.h)
and takes torch tensors for the device buffers; torch is used for device memory
and streams only.  All arithmetic runs in the HIP kernels of libmxq.so.  There
is no fallback: if the library is missing or a call fails, an exception is
raised.

Sources of the operations: "[mxfp8 MoE training] Support mxfp8 all to all in
expert parallel" (Summary) for the MXFP8 codec, "[moe training] fix
uncoalesced global accesses in per group rowwise scaling kernel" (Summary) for
the group scaling and the layout transform, and "[float8] add float8 rowwise
MoE prototype" (Summary) for the scaled grouped GEMM.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxq.so")

MXQ_LAYOUT_ROW = 0
MXQ_LAYOUT_COL = 1
MXQ_OK = 0
MXQ_ERR_NULL, MXQ_ERR_SHAPE, MXQ_ERR_ALIGN, MXQ_ERR_LAYOUT, MXQ_ERR_WORKSPACE, MXQ_ERR_HIP = 1, 2, 3, 4, 5, 6
MXQ_ERR_DTYPE = 8
MXQ_ERR_RULE = 9
MXQ_OUT_BF16 = 0
MXQ_OUT_F32 = 1
MXQ_SCALE_FLOOR = 0
MXQ_SCALE_RCEIL = 1
MXQ_GROUP_POW2_SCALE = 1
MXQ_GROUP_INVERSE_SCALE = 2
MXQ_FMT_E4M3 = 0
MXQ_FMT_E2M1 = 1
MXQ_SCORE_SOFTMAX = 0
MXQ_SCORE_SIGMOID = 1
MXQ_PRODUCT_Y, MXQ_PRODUCT_DX, MXQ_PRODUCT_DW = 0, 1, 2
MXQ_ROUTE_RENORM = 1
MXQ_ROUTE_GROUP_TOP2 = 2

EXPORTED = ("mxq_abi_version", "mxq_status_string", "mxq_last_hip_error", "mxq_quantize_mx",
            "mxq_dequantize_mx", "mxq_group_scale_workspace_bytes", "mxq_group_scale_fp8",
            "mxq_transpose_u8", "mxq_grouped_mm_workspace_bytes", "mxq_scaled_grouped_mm",
            "mxq_quantize_mx_ex", "mxq_dequantize_mx_ex", "mxq_group_scale_fp8_ex",
            "mxq_dispatch_pack_workspace_bytes", "mxq_dispatch_pack_mx", "mxq_scaled_grouped_mm_packed",
            "mxq_set_group_scale_knobs", "mxq_group_scale_fp8_noalloc", "mxq_group_scale_route_counters",
            "mxq_add_rmsnorm", "mxq_add_rmsnorm_bwd_workspace_bytes", "mxq_add_rmsnorm_bwd", "mxq_route_topk",
            "mxq_route_topk_bwd", "mxq_quantize_mxfp4", "mxq_dequantize_mxfp4",
            "mxq_mxfp4_grouped_mm", "mxq_mxfp4_grouped_mm_packed", "mxq_bf16_grouped_mm_workspace_bytes",
            "mxq_bf16_grouped_mm", "mxq_bf16_grouped_mm_dx", "mxq_bf16_grouped_mm_dw", "mxq_add_layernorm",
            "mxq_add_layernorm_bwd_workspace_bytes", "mxq_add_layernorm_bwd", "mxq_dispatch_rows_workspace_bytes",
            "mxq_dispatch_rows", "mxq_pair_rows", "mxq_combine_rows", "mxq_combine_rows_bwd")

GROUP_METHODS = {"auto": 0, "hold": 1, "twopass": 2, "split": 3}


class MxqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().mxq_status_string(status).decode()
        if status == MXQ_ERR_HIP:
            msg += f" (hipError {lib().mxq_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmxq.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmxq.so not found at {LIB_PATH}; build it with "
                              "`python -m float8_quantization_moe_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i32, i64, P, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        L.mxq_abi_version.restype = ctypes.c_int
        L.mxq_abi_version.argtypes = []
        L.mxq_status_string.restype = ctypes.c_char_p
        L.mxq_status_string.argtypes = [ctypes.c_int]
        L.mxq_last_hip_error.restype = ctypes.c_int
        L.mxq_last_hip_error.argtypes = []
        L.mxq_quantize_mx.restype = ctypes.c_int
        L.mxq_quantize_mx.argtypes = [P, i64, i64, P, P, P]
        L.mxq_dequantize_mx.restype = ctypes.c_int
        L.mxq_dequantize_mx.argtypes = [P, P, i64, i64, P, P]
        L.mxq_quantize_mx_ex.restype = ctypes.c_int
        L.mxq_quantize_mx_ex.argtypes = [P, i64, i64, ctypes.c_int, ctypes.c_int, P, P, P]
        L.mxq_dequantize_mx_ex.restype = ctypes.c_int
        L.mxq_dequantize_mx_ex.argtypes = [P, P, i64, i64, ctypes.c_int, P, P]
        L.mxq_group_scale_workspace_bytes.restype = sz
        L.mxq_group_scale_workspace_bytes.argtypes = [i64, i64, i32]
        L.mxq_group_scale_fp8.restype = ctypes.c_int
        L.mxq_group_scale_fp8.argtypes = [P, i64, i64, P, i32, ctypes.c_int, P, P, P, sz, P]
        L.mxq_group_scale_fp8_ex.restype = ctypes.c_int
        L.mxq_group_scale_fp8_ex.argtypes = [P, i64, i64, P, i32, ctypes.c_int, ctypes.c_int, P, P, P, sz, P]
        L.mxq_transpose_u8.restype = ctypes.c_int
        L.mxq_transpose_u8.argtypes = [P, i64, i64, P, P]
        L.mxq_grouped_mm_workspace_bytes.restype = sz
        L.mxq_grouped_mm_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.mxq_dispatch_pack_workspace_bytes.restype = sz
        L.mxq_dispatch_pack_workspace_bytes.argtypes = [i64, i64, i32, i32]
        L.mxq_dispatch_pack_mx.restype = ctypes.c_int
        L.mxq_dispatch_pack_mx.argtypes = [P, i64, i64, P, i32, i32, P, P, P, P, sz, P]
        L.mxq_scaled_grouped_mm_packed.restype = ctypes.c_int
        L.mxq_scaled_grouped_mm_packed.argtypes = [P, P, P, P, i64, i64, i64, i32, ctypes.c_int, P, P, sz, P]
        L.mxq_group_scale_fp8_noalloc.restype = ctypes.c_int
        L.mxq_group_scale_fp8_noalloc.argtypes = [P, i64, i64, P, i32, ctypes.c_int, ctypes.c_int, P, P, P]
        L.mxq_set_group_scale_knobs.restype = ctypes.c_int
        L.mxq_set_group_scale_knobs.argtypes = [ctypes.c_int, ctypes.c_int, i64, ctypes.c_int]
        L.mxq_group_scale_route_counters.restype = ctypes.c_int
        L.mxq_group_scale_route_counters.argtypes = [P, sz, i64, i64, i32, ctypes.c_int, P, P]
        L.mxq_scaled_grouped_mm.restype = ctypes.c_int
        L.mxq_scaled_grouped_mm.argtypes = [P, P, P, P, P, i64, i64, i64, i32, ctypes.c_int, P, P, sz, P]
        f32, ci = ctypes.c_float, ctypes.c_int
        L.mxq_add_rmsnorm.restype = ci
        L.mxq_add_rmsnorm.argtypes = [P, P, P, ci, i64, i64, f32, P, P, P, P, P, P]
        L.mxq_add_rmsnorm_bwd_workspace_bytes.restype = sz
        L.mxq_add_rmsnorm_bwd_workspace_bytes.argtypes = [i64, i64]
        L.mxq_add_rmsnorm_bwd.restype = ci
        L.mxq_add_rmsnorm_bwd.argtypes = [P, P, P, P, P, ci, i64, i64, P, P, P, sz, P]
        L.mxq_route_topk.restype = ci
        L.mxq_route_topk.argtypes = [P, ci, i64, i32, P, ci, i32, i32, i32, ci, f32, P, P, P]
        L.mxq_route_topk_bwd.restype = ci
        L.mxq_route_topk_bwd.argtypes = [P, ci, i64, i32, ci, P, i32, ci, f32, P, P, P]
        L.mxq_quantize_mxfp4.restype = ci
        L.mxq_quantize_mxfp4.argtypes = [P, i64, i64, ci, P, P, P]
        L.mxq_dequantize_mxfp4.restype = ci
        L.mxq_dequantize_mxfp4.argtypes = [P, P, i64, i64, P, P]
        L.mxq_mxfp4_grouped_mm.restype = ci
        L.mxq_mxfp4_grouped_mm.argtypes = [P, P, ci, P, P, P, i64, i64, i64, i32, ci, P, P]
        L.mxq_mxfp4_grouped_mm_packed.restype = ci
        L.mxq_mxfp4_grouped_mm_packed.argtypes = [P, P, P, P, i64, i64, i64, i32, ci, P, P]
        L.mxq_bf16_grouped_mm_workspace_bytes.restype = sz
        L.mxq_bf16_grouped_mm_workspace_bytes.argtypes = [ci, i64, i64, i64, i32]
        L.mxq_bf16_grouped_mm.restype = ci
        L.mxq_bf16_grouped_mm.argtypes = [P, P, P, i64, i64, i64, i32, ci, P, P, sz, P]
        L.mxq_bf16_grouped_mm_dx.restype = ci
        L.mxq_bf16_grouped_mm_dx.argtypes = [P, P, P, i64, i64, i64, i32, ci, P, P, sz, P]
        L.mxq_bf16_grouped_mm_dw.restype = ci
        L.mxq_bf16_grouped_mm_dw.argtypes = [P, P, P, i64, i64, i64, i32, ci, ci, P, P, sz, P]
        L.mxq_add_layernorm.restype = ci
        L.mxq_add_layernorm.argtypes = [P, P, P, P, ci, i64, i64, f32, P, P, P, P, P, P, P]
        L.mxq_add_layernorm_bwd_workspace_bytes.restype = sz
        L.mxq_add_layernorm_bwd_workspace_bytes.argtypes = [i64, i64]
        L.mxq_add_layernorm_bwd.restype = ci
        L.mxq_add_layernorm_bwd.argtypes = [P, P, P, P, P, P, ci, i64, i64, P, P, P, P, sz, P]
        L.mxq_dispatch_rows_workspace_bytes.restype = sz
        L.mxq_dispatch_rows_workspace_bytes.argtypes = [i64, i32, i32]
        L.mxq_dispatch_rows.restype = ci
        L.mxq_dispatch_rows.argtypes = [P, ci, i64, i64, P, i32, i32, P, P, P, P, P, sz, P]
        L.mxq_pair_rows.restype = ci
        L.mxq_pair_rows.argtypes = [P, i64, P, P]
        L.mxq_combine_rows.restype = ci
        L.mxq_combine_rows.argtypes = [P, ci, i64, i64, P, i64, i32, P, P, P]
        L.mxq_combine_rows_bwd.restype = ci
        L.mxq_combine_rows_bwd.argtypes = [P, P, ci, i64, i64, P, i64, i32, P, P, P, P]
        _lib = L
    return _lib


def mxq_set_group_scale_knobs(method: str = "auto", hold_tiles: int = -1, wait_us: int = -1,
                              strip_block: int = 0) -> None:
    """Test hook: force the group-scaling route (see include/mxq.h).  Defaults restore the automatic choice."""
    _check(lib().mxq_set_group_scale_knobs(GROUP_METHODS[method], int(hold_tiles), int(wait_us), int(strip_block)),
           "mxq_set_group_scale_knobs")


def mxq_group_scale_route_counters(workspace: torch.Tensor, M: int, K: int, G: int, out_layout: int,
                                   stream=None) -> tuple:
    """Test hook: the hold method's (timed-out tiles, strips re-read from X) of the
    last call that used `workspace` (see include/mxq.h).  Synchronises the stream."""
    out = (ctypes.c_uint32 * 2)()
    pw = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_group_scale_route_counters(pw, wbytes, int(M), int(K), int(G), int(out_layout), out,
                                                _stream(stream)), "mxq_group_scale_route_counters")
    return int(out[0]), int(out[1])


@contextlib.contextmanager
def group_scale_knobs(**kw):
    """Context manager around mxq_set_group_scale_knobs that restores the defaults on exit."""
    mxq_set_group_scale_knobs(**kw)
    try:
        yield
    finally:
        mxq_set_group_scale_knobs()


# The current stream's handle without building a torch.cuda.Stream object (0.1 us
# instead of 2.9 us a call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, name: str, dtype=None, numel=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _check(status: int, where: str) -> None:
    if status != MXQ_OK:
        raise MxqError(status, where)


def mxq_abi_version() -> int:
    return lib().mxq_abi_version()


def mxq_quantize_mx(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """x (M, K) bf16 -> q (M, K) uint8 E4M3 codes, s (M, K/32) uint8 E8M0 codes."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    px = _dev(x, "x", torch.bfloat16)
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(s, "s", torch.uint8, M * (K // 32) if K % 32 == 0 else None)
    _check(lib().mxq_quantize_mx(px, M, K, pq, ps, _stream(stream)), "mxq_quantize_mx")


def mxq_dequantize_mx(q: torch.Tensor, s: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """q (M, K) uint8 E4M3 + s (M, K/32) uint8 E8M0 -> y (M, K) bf16."""
    if y.dim() != 2:
        raise ValueError("y must be 2-D (M, K)")
    M, K = y.shape
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(s, "s", torch.uint8, M * (K // 32) if K % 32 == 0 else None)
    py = _dev(y, "y", torch.bfloat16)
    _check(lib().mxq_dequantize_mx(pq, ps, M, K, py, _stream(stream)), "mxq_dequantize_mx")


def _mx_scale_numel(M: int, K: int, axis: int):
    if axis == 1:
        return M * (K // 32) if K % 32 == 0 else None
    if axis == 0:
        return (M // 32) * K if M % 32 == 0 else None
    return None


def mxq_quantize_mx_ex(x: torch.Tensor, axis: int, rule: int, q: torch.Tensor, s: torch.Tensor,
                       stream=None) -> None:
    """MX variants: x (M, K) bf16 -> q (M, K) uint8 E4M3 and s E8M0 codes, (M, K/32) for
    axis 1 or (M/32, K) for axis 0; rule MXQ_SCALE_FLOOR or MXQ_SCALE_RCEIL."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    px = _dev(x, "x", torch.bfloat16)
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(s, "s", torch.uint8, _mx_scale_numel(M, K, axis))
    _check(lib().mxq_quantize_mx_ex(px, M, K, int(axis), int(rule), pq, ps, _stream(stream)), "mxq_quantize_mx_ex")


def mxq_dequantize_mx_ex(q: torch.Tensor, s: torch.Tensor, axis: int, y: torch.Tensor, stream=None) -> None:
    """Inverse of mxq_quantize_mx_ex for either axis -> y (M, K) bf16."""
    if y.dim() != 2:
        raise ValueError("y must be 2-D (M, K)")
    M, K = y.shape
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(s, "s", torch.uint8, _mx_scale_numel(M, K, axis))
    py = _dev(y, "y", torch.bfloat16)
    _check(lib().mxq_dequantize_mx_ex(pq, ps, M, K, int(axis), py, _stream(stream)), "mxq_dequantize_mx_ex")


def mxq_group_scale_workspace_bytes(M: int, K: int, G: int) -> int:
    return int(lib().mxq_group_scale_workspace_bytes(int(M), int(K), int(G)))


def mxq_group_scale_fp8(x: torch.Tensor, group_end_offs: torch.Tensor, out_layout: int,
                        q: torch.Tensor, scales: torch.Tensor, workspace: torch.Tensor,
                        stream=None) -> None:
    """x (M, K) bf16, group_end_offs int32[G] (device) -> q uint8 ((M, K) for ROW,
    (K, M) for COL) and scales float32 (G, K)."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    G = group_end_offs.numel()
    px = _dev(x, "x", torch.bfloat16)
    po = _dev(group_end_offs, "group_end_offs", torch.int32)
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(scales, "scales", torch.float32, G * K)
    pw = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_group_scale_fp8(px, M, K, po, G, int(out_layout), pq, ps, pw, wbytes, _stream(stream)),
           "mxq_group_scale_fp8")


def mxq_group_scale_fp8_ex(x: torch.Tensor, group_end_offs: torch.Tensor, out_layout: int, flags: int,
                           q: torch.Tensor, scales: torch.Tensor, workspace: torch.Tensor,
                           stream=None) -> None:
    """mxq_group_scale_fp8 with flags MXQ_GROUP_POW2_SCALE / MXQ_GROUP_INVERSE_SCALE."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    G = group_end_offs.numel()
    px = _dev(x, "x", torch.bfloat16)
    po = _dev(group_end_offs, "group_end_offs", torch.int32)
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(scales, "scales", torch.float32, G * K)
    pw = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_group_scale_fp8_ex(px, M, K, po, G, int(out_layout), int(flags), pq, ps, pw, wbytes,
                                        _stream(stream)), "mxq_group_scale_fp8_ex")


def mxq_group_scale_fp8_noalloc(x: torch.Tensor, group_end_offs: torch.Tensor, out_layout: int, flags: int,
                                q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """mxq_group_scale_fp8_ex with the library's static per-GPU scratch instead of a workspace."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    G = group_end_offs.numel()
    px = _dev(x, "x", torch.bfloat16)
    po = _dev(group_end_offs, "group_end_offs", torch.int32)
    pq = _dev(q, "q", torch.uint8, M * K)
    ps = _dev(scales, "scales", torch.float32, G * K)
    _check(lib().mxq_group_scale_fp8_noalloc(px, M, K, po, G, int(out_layout), int(flags), pq, ps,
                                             _stream(stream)), "mxq_group_scale_fp8_noalloc")


def mxq_transpose_u8(inp: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out (C, R) = inp (R, C)^T for uint8 tensors."""
    if inp.dim() != 2:
        raise ValueError("inp must be 2-D")
    R, C = inp.shape
    pi = _dev(inp, "inp", torch.uint8)
    po = _dev(out, "out", torch.uint8, R * C)
    _check(lib().mxq_transpose_u8(pi, R, C, po, _stream(stream)), "mxq_transpose_u8")


def mxq_grouped_mm_workspace_bytes(M: int, N: int, K: int, G: int) -> int:
    return int(lib().mxq_grouped_mm_workspace_bytes(int(M), int(N), int(K), int(G)))


def mxq_scaled_grouped_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                          group_end_offs: torch.Tensor, y: torch.Tensor, workspace: torch.Tensor,
                          stream=None) -> None:
    """xq (M, K) / xs (M, K/32) and wq (G, N, K) / ws (G, N, K/32) uint8 MXFP8
    operands, group_end_offs int32[G] (device) -> y (M, N) bf16 or float32."""
    if xq.dim() != 2 or wq.dim() != 3 or y.dim() != 2:
        raise ValueError("xq must be (M, K), wq (G, N, K) and y (M, N)")
    M, K = xq.shape
    G, N, Kw = wq.shape
    if Kw != K or tuple(y.shape) != (M, N):
        raise ValueError("operand shapes do not match")
    if group_end_offs.numel() != G:
        raise ValueError("need one end offset per group")
    if y.dtype == torch.bfloat16:
        out_dtype = MXQ_OUT_BF16
    elif y.dtype == torch.float32:
        out_dtype = MXQ_OUT_F32
    else:
        raise TypeError("y must be bfloat16 or float32")
    kb = K // 32 if K % 32 == 0 else None
    pxq = _dev(xq, "xq", torch.uint8)
    pxs = _dev(xs, "xs", torch.uint8, M * kb if kb is not None else None)
    pwq = _dev(wq, "wq", torch.uint8)
    pws = _dev(ws, "ws", torch.uint8, G * N * kb if kb is not None else None)
    po = _dev(group_end_offs, "group_end_offs", torch.int32)
    py = _dev(y, "y")
    pw = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_scaled_grouped_mm(pxq, pxs, pwq, pws, po, M, N, K, G, out_dtype, py, pw, wbytes,
                                       _stream(stream)), "mxq_scaled_grouped_mm")


# ---------------------------------------------------------------- helpers ---
# Allocate outputs and workspaces with torch and call the entry points above.  A helper
# given a stream (a torch stream or a raw handle) runs as it would under
# `with torch.cuda.stream(stream):`, its allocations included: torch hands out memory that
# is free in the order of the current stream's work, so a block taken on another stream
# could still be in use there, and a dropped one be handed out again before this stream
# is done with it.  The caller orders the stream after the work that makes the inputs.

def _stream_of(stream, t: torch.Tensor) -> torch.cuda.Stream:
    """`stream` as a torch stream; a raw handle is one of the tensor's device."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    device = t.device if t.is_cuda else None
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)


def quantize_mx(x: torch.Tensor, stream=None):
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, x)):
            return quantize_mx(x)
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    mxq_quantize_mx(x, q, s)
    return q, s


def dequantize_mx(q: torch.Tensor, s: torch.Tensor, stream=None) -> torch.Tensor:
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, q)):
            return dequantize_mx(q, s)
    y = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    mxq_dequantize_mx(q, s, y)
    return y


def group_scale_fp8(x: torch.Tensor, group_end_offs: torch.Tensor, out_layout: int = MXQ_LAYOUT_ROW,
                    stream=None):
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, x)):
            return group_scale_fp8(x, group_end_offs, out_layout)
    M, K = x.shape
    G = group_end_offs.numel()
    q = torch.empty((M, K) if out_layout == MXQ_LAYOUT_ROW else (K, M), dtype=torch.uint8, device=x.device)
    scales = torch.empty((G, K), dtype=torch.float32, device=x.device)
    ws = torch.empty(max(mxq_group_scale_workspace_bytes(M, K, G), 16), dtype=torch.uint8, device=x.device)
    mxq_group_scale_fp8(x, group_end_offs, out_layout, q, scales, ws)
    return q, scales


def transpose_u8(inp: torch.Tensor, stream=None) -> torch.Tensor:
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, inp)):
            return transpose_u8(inp)
    R, C = inp.shape
    out = torch.empty((C, R), dtype=torch.uint8, device=inp.device)
    mxq_transpose_u8(inp, out)
    return out


def scaled_grouped_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                      group_end_offs: torch.Tensor, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, xq)):
            return scaled_grouped_mm(xq, xs, wq, ws, group_end_offs, out_dtype)
    M, K = xq.shape
    G, N, _ = wq.shape
    y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    wsp = torch.empty(max(mxq_grouped_mm_workspace_bytes(M, N, K, G), 16), dtype=torch.uint8,
                      device=xq.device)
    mxq_scaled_grouped_mm(xq, xs, wq, ws, group_end_offs, y, wsp)
    return y


def mxq_dispatch_pack_workspace_bytes(M: int, K: int, topk: int, E: int) -> int:
    return int(lib().mxq_dispatch_pack_workspace_bytes(int(M), int(K), int(topk), int(E)))


def mxq_dispatch_pack_mx(x: torch.Tensor, expert_ids: torch.Tensor, E: int, packed: torch.Tensor,
                         group_end_offs: torch.Tensor, src_pair: torch.Tensor, workspace: torch.Tensor,
                         stream=None) -> None:
    """x (M, K) bf16, expert_ids (M, topk) int32 -> packed (M*topk, K + K/32) uint8 rows
    [e4m3 | e8m0] sorted stably by expert, group_end_offs int32[E], src_pair int32[M*topk]."""
    if x.dim() != 2 or expert_ids.dim() != 2 or expert_ids.shape[0] != x.shape[0]:
        raise ValueError("x must be (M, K) and expert_ids (M, topk)")
    M, K = x.shape
    topk = expert_ids.shape[1]
    px = _dev(x, "x", torch.bfloat16)
    pi = _dev(expert_ids, "expert_ids", torch.int32)
    pp = _dev(packed, "packed", torch.uint8, M * topk * (K + K // 32))
    pe = _dev(group_end_offs, "group_end_offs", torch.int32, int(E))
    ps = _dev(src_pair, "src_pair", torch.int32, M * topk)
    pw = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_dispatch_pack_mx(px, M, K, pi, topk, int(E), pp, pe, ps, pw, wbytes, _stream(stream)),
           "mxq_dispatch_pack_mx")


def mxq_scaled_grouped_mm_packed(packed: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                                 group_end_offs: torch.Tensor, y: torch.Tensor, workspace: torch.Tensor,
                                 stream=None) -> None:
    """packed (M, K + K/32) uint8 token rows [e4m3 | e8m0], wq (G, N, K) / ws (G, N, K/32) ->
    y (M, N), bf16 or float32 by y's dtype."""
    if packed.dim() != 2 or wq.dim() != 3 or y.dim() != 2:
        raise ValueError("packed must be 2-D, wq 3-D (G, N, K), y 2-D (M, N)")
    G, N, K = wq.shape
    M = packed.shape[0]
    if packed.shape[1] != K + K // 32 or tuple(y.shape) != (M, N):
        raise ValueError("shapes do not match")
    dt = {torch.bfloat16: MXQ_OUT_BF16, torch.float32: MXQ_OUT_F32}.get(y.dtype)
    if dt is None:
        raise TypeError("y must be bfloat16 or float32")
    pp = _dev(packed, "packed", torch.uint8)
    pwq = _dev(wq, "wq", torch.uint8)
    pws = _dev(ws, "ws", torch.uint8, G * N * (K // 32))
    po = _dev(group_end_offs, "group_end_offs", torch.int32, G)
    py = _dev(y, "y")
    pw = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_scaled_grouped_mm_packed(pp, pwq, pws, po, M, N, K, G, dt, py, pw, wbytes, _stream(stream)),
           "mxq_scaled_grouped_mm_packed")


# ------------------------------------------------------------------- norm ---
def _float_code(t: torch.Tensor, name: str) -> int:
    """mxq_out_dtype of a bf16 or float32 tensor."""
    if t.dtype == torch.bfloat16:
        return MXQ_OUT_BF16
    if t.dtype == torch.float32:
        return MXQ_OUT_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _opt(t, name: str, dtype=None, numel=None) -> int:
    """_dev of a tensor that may be None (a NULL pointer)."""
    return 0 if t is None else _dev(t, name, dtype, numel)


def mxq_add_rmsnorm(x: torch.Tensor, residual, weight: torch.Tensor, eps: float, h=None, y=None, q=None, s=None,
                    rstd=None, stream=None) -> None:
    """x (+ residual) (M, K) and weight (K), bf16 or float32 -> h = x + residual, y = rmsnorm(h) * weight
    (their type), q (M, K) / s (M, K/32) uint8 = MXFP8 of y, rstd (M) float32; outputs may be None."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    code, dt, n = _float_code(x, "x"), x.dtype, M * K
    px = _dev(x, "x")
    pr = _opt(residual, "residual", dt, n)
    pw = _dev(weight, "weight", dt, K)
    ph = _opt(h, "h", dt, n)
    py = _opt(y, "y", dt, n)
    pq = _opt(q, "q", torch.uint8, n)
    ps = _opt(s, "s", torch.uint8, M * (K // 32) if K % 32 == 0 else None)
    pd = _opt(rstd, "rstd", torch.float32, M)
    _check(lib().mxq_add_rmsnorm(px, pr, pw, code, M, K, float(eps), ph, py, pq, ps, pd, _stream(stream)),
           "mxq_add_rmsnorm")


def mxq_add_rmsnorm_bwd_workspace_bytes(M: int, K: int) -> int:
    return int(lib().mxq_add_rmsnorm_bwd_workspace_bytes(int(M), int(K)))


def mxq_add_rmsnorm_bwd(h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor, dh,
                        dx: torch.Tensor, dweight: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """h, rstd of mxq_add_rmsnorm and the gradients dy, dh (or None) -> dx (M, K) and dweight (K) float32."""
    if h.dim() != 2:
        raise ValueError("h must be 2-D (M, K)")
    M, K = h.shape
    code, dt, n = _float_code(h, "h"), h.dtype, M * K
    ph = _dev(h, "h")
    pw = _dev(weight, "weight", dt, K)
    pr = _dev(rstd, "rstd", torch.float32, M)
    pg = _dev(dy, "dy", dt, n)
    pd = _opt(dh, "dh", dt, n)
    px = _dev(dx, "dx", dt, n)
    pk = _dev(dweight, "dweight", torch.float32, K)
    pws = _dev(workspace, "workspace")
    wbytes = workspace.numel() * workspace.element_size()
    _check(lib().mxq_add_rmsnorm_bwd(ph, pw, pr, pg, pd, code, M, K, px, pk, pws, wbytes, _stream(stream)),
           "mxq_add_rmsnorm_bwd")


def add_rmsnorm(x: torch.Tensor, residual, weight: torch.Tensor, eps: float, stream=None):
    """(h, y, q, s, rstd) of mxq_add_rmsnorm; h is x itself when there is no residual."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, x)):
            return add_rmsnorm(x, residual, weight, eps)
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    code, dt = _float_code(x, "x"), x.dtype
    px, pr, pw = _dev(x, "x"), _opt(residual, "residual", dt, M * K), _dev(weight, "weight", dt, K)
    # (outputs made here need no checks: a token's norm is host time)
    h = x if residual is None else torch.empty_like(x)
    y = torch.empty_like(x)
    q = torch.empty_like(x, dtype=torch.uint8)
    s = x.new_empty((M, K // 32), dtype=torch.uint8)
    rstd = x.new_empty(M, dtype=torch.float32)
    _check(lib().mxq_add_rmsnorm(px, pr, pw, code, M, K, eps, 0 if residual is None else h.data_ptr(), y.data_ptr(),
                                 q.data_ptr(), s.data_ptr(), rstd.data_ptr(), _stream(None)), "mxq_add_rmsnorm")
    return h, y, q, s, rstd


def add_rmsnorm_bwd(h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor, dh=None, stream=None):
    """(dx, dweight) of mxq_add_rmsnorm_bwd."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, h)):
            return add_rmsnorm_bwd(h, weight, rstd, dy, dh)
    if h.dim() != 2:
        raise ValueError("h must be 2-D (M, K)")
    M, K = h.shape
    dx = torch.empty_like(h)
    dweight = h.new_empty(K, dtype=torch.float32)
    ws = h.new_empty(max(mxq_add_rmsnorm_bwd_workspace_bytes(M, K), 16), dtype=torch.uint8)
    mxq_add_rmsnorm_bwd(h, weight, rstd, dy, dh, dx, dweight, ws)
    return dx, dweight


# ---------------------------------------------------------------- routing ---
SCORES = {"softmax": MXQ_SCORE_SOFTMAX, "sigmoid": MXQ_SCORE_SIGMOID}


def mxq_route_topk(logits: torch.Tensor, bias, score: int, n_groups: int, topk_groups: int, flags: int, scale: float,
                   expert_ids: torch.Tensor, weights: torch.Tensor, stream=None) -> None:
    """logits (M, E) bf16 or float32, bias float32 (E) or None -> expert_ids int32 and weights float32, (M, topk)."""
    if logits.dim() != 2 or expert_ids.dim() != 2 or expert_ids.shape[0] != logits.shape[0]:
        raise ValueError("logits must be (M, E) and expert_ids (M, topk)")
    M, E = logits.shape
    topk = expert_ids.shape[1]
    code = _float_code(logits, "logits")
    pl = _dev(logits, "logits")
    pb = _opt(bias, "bias", torch.float32, E)
    pi = _dev(expert_ids, "expert_ids", torch.int32)
    pw = _dev(weights, "weights", torch.float32, M * topk)
    _check(lib().mxq_route_topk(pl, code, M, E, pb, int(score), int(n_groups), int(topk_groups), topk, int(flags),
                                float(scale), pi, pw, _stream(stream)), "mxq_route_topk")


def mxq_route_topk_bwd(logits: torch.Tensor, score: int, expert_ids: torch.Tensor, flags: int, scale: float,
                       dweights: torch.Tensor, dlogits: torch.Tensor, stream=None) -> None:
    """logits (M, E), expert_ids and dweights (M, topk) -> dlogits (M, E), the type of logits."""
    if logits.dim() != 2 or expert_ids.dim() != 2 or expert_ids.shape[0] != logits.shape[0]:
        raise ValueError("logits must be (M, E) and expert_ids (M, topk)")
    M, E = logits.shape
    topk = expert_ids.shape[1]
    code = _float_code(logits, "logits")
    pl = _dev(logits, "logits")
    pi = _dev(expert_ids, "expert_ids", torch.int32)
    pw = _dev(dweights, "dweights", torch.float32, M * topk)
    pd = _dev(dlogits, "dlogits", logits.dtype, M * E)
    _check(lib().mxq_route_topk_bwd(pl, code, M, E, int(score), pi, topk, int(flags), float(scale), pw, pd,
                                    _stream(stream)), "mxq_route_topk_bwd")


def route_topk(logits: torch.Tensor, topk: int, bias=None, score: str = "softmax", n_groups: int = 1,
               topk_groups: int = 1, renormalize: bool = False, group_top2: bool = False, scale: float = 1.0,
               stream=None):
    """(expert_ids, weights), each (M, topk), of mxq_route_topk."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, logits)):
            return route_topk(logits, topk, bias, score, n_groups, topk_groups, renormalize, group_top2, scale)
    M = logits.shape[0]
    ids = logits.new_empty((M, topk), dtype=torch.int32)
    weights = logits.new_empty((M, topk), dtype=torch.float32)
    flags = (MXQ_ROUTE_RENORM if renormalize else 0) | (MXQ_ROUTE_GROUP_TOP2 if group_top2 else 0)
    mxq_route_topk(logits, bias, SCORES[score], n_groups, topk_groups, flags, scale, ids, weights)
    return ids, weights


def route_topk_bwd(logits: torch.Tensor, expert_ids: torch.Tensor, dweights: torch.Tensor, score: str = "softmax",
                   renormalize: bool = False, scale: float = 1.0, stream=None) -> torch.Tensor:
    """dlogits of mxq_route_topk_bwd."""
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, logits)):
            return route_topk_bwd(logits, expert_ids, dweights, score, renormalize, scale)
    dlogits = torch.empty_like(logits)
    mxq_route_topk_bwd(logits, SCORES[score], expert_ids, MXQ_ROUTE_RENORM if renormalize else 0, scale, dweights,
                       dlogits)
    return dlogits


# ------------------------------------------------------------------ MXFP4 ---
def mxq_quantize_mxfp4(x: torch.Tensor, rule: int, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """x (M, K) bf16 -> q (M, K/2) uint8 pairs of E2M1 codes, s (M, K/32) uint8 E8M0 codes."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    px = _dev(x, "x", torch.bfloat16)
    pq = _dev(q, "q", torch.uint8, M * (K // 2) if K % 32 == 0 else None)
    ps = _dev(s, "s", torch.uint8, M * (K // 32) if K % 32 == 0 else None)
    _check(lib().mxq_quantize_mxfp4(px, M, K, int(rule), pq, ps, _stream(stream)), "mxq_quantize_mxfp4")


def mxq_dequantize_mxfp4(q: torch.Tensor, s: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """q (M, K/2) uint8 + s (M, K/32) uint8 -> y (M, K) bf16."""
    if y.dim() != 2:
        raise ValueError("y must be 2-D (M, K)")
    M, K = y.shape
    pq = _dev(q, "q", torch.uint8, M * (K // 2) if K % 32 == 0 else None)
    ps = _dev(s, "s", torch.uint8, M * (K // 32) if K % 32 == 0 else None)
    py = _dev(y, "y", torch.bfloat16)
    _check(lib().mxq_dequantize_mxfp4(pq, ps, M, K, py, _stream(stream)), "mxq_dequantize_mxfp4")


def quantize_mxfp4(x: torch.Tensor, rule: int = MXQ_SCALE_FLOOR, stream=None):
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, x)):
            return quantize_mxfp4(x, rule)
    M, K = x.shape
    q = x.new_empty((M, K // 2), dtype=torch.uint8)
    s = x.new_empty((M, K // 32), dtype=torch.uint8)
    mxq_quantize_mxfp4(x, rule, q, s)
    return q, s


def dequantize_mxfp4(q: torch.Tensor, s: torch.Tensor, stream=None) -> torch.Tensor:
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, q)):
            return dequantize_mxfp4(q, s)
    y = q.new_empty((q.shape[0], 2 * q.shape[1]), dtype=torch.bfloat16)
    mxq_dequantize_mxfp4(q, s, y)
    return y


def mxq_mxfp4_grouped_mm(xq: torch.Tensor, xs: torch.Tensor, x_format: int, wq: torch.Tensor, ws: torch.Tensor,
                         group_end_offs: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """xq (M, K) E4M3 or (M, K/2) E2M1 by x_format, xs (M, K/32), wq (G, N, K/2) E2M1, ws (G, N, K/32),
    group_end_offs int32[G] (device) -> y (M, N) bf16 or float32."""
    if xq.dim() != 2 or wq.dim() != 3 or y.dim() != 2:
        raise ValueError("xq must be 2-D, wq (G, N, K/2) and y (M, N)")
    M = xq.shape[0]
    G, N, half = wq.shape
    K = 2 * half
    if xq.shape[1] != (half if x_format == MXQ_FMT_E2M1 else K) or tuple(y.shape) != (M, N):
        raise ValueError("operand shapes do not match")
    kb = K // 32 if K % 32 == 0 else None
    pxq = _dev(xq, "xq", torch.uint8)
    pxs = _dev(xs, "xs", torch.uint8, M * kb if kb is not None else None)
    pwq = _dev(wq, "wq", torch.uint8)
    pws = _dev(ws, "ws", torch.uint8, G * N * kb if kb is not None else None)
    po = _dev(group_end_offs, "group_end_offs", torch.int32, G)
    code = _float_code(y, "y")
    py = _dev(y, "y")
    _check(lib().mxq_mxfp4_grouped_mm(pxq, pxs, int(x_format), pwq, pws, po, M, N, K, G, code, py,
                                      _stream(stream)), "mxq_mxfp4_grouped_mm")


def mxq_mxfp4_grouped_mm_packed(packed: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                                group_end_offs: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """packed (M, K + K/32) uint8 MXFP8 token rows, wq (G, N, K/2) / ws (G, N, K/32) -> y (M, N) bf16 or float32."""
    if packed.dim() != 2 or wq.dim() != 3 or y.dim() != 2:
        raise ValueError("packed must be 2-D, wq 3-D (G, N, K/2), y 2-D (M, N)")
    G, N, half = wq.shape
    K, M = 2 * half, packed.shape[0]
    if packed.shape[1] != K + K // 32 or tuple(y.shape) != (M, N):
        raise ValueError("shapes do not match")
    pp = _dev(packed, "packed", torch.uint8)
    pwq = _dev(wq, "wq", torch.uint8)
    pws = _dev(ws, "ws", torch.uint8, G * N * (K // 32))
    po = _dev(group_end_offs, "group_end_offs", torch.int32, G)
    code = _float_code(y, "y")
    py = _dev(y, "y")
    _check(lib().mxq_mxfp4_grouped_mm_packed(pp, pwq, pws, po, M, N, K, G, code, py, _stream(stream)),
           "mxq_mxfp4_grouped_mm_packed")


def mxfp4_grouped_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                     group_end_offs: torch.Tensor, x_format: int = MXQ_FMT_E4M3, out_dtype=torch.bfloat16,
                     stream=None) -> torch.Tensor:
    if stream is not None:
        with torch.cuda.stream(_stream_of(stream, xq)):
            return mxfp4_grouped_mm(xq, xs, wq, ws, group_end_offs, x_format, out_dtype)
    M = xq.shape[0]
    G, N, half = wq.shape
    y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    mxq_mxfp4_grouped_mm(xq, xs, x_format, wq, ws, group_end_offs, y)
    return y


# ------------------------------------------------------- products in bf16 ---
# (Their helpers, which allocate, are in training.py.)
def mxq_bf16_grouped_mm_workspace_bytes(product: int, M: int, N: int, K: int, G: int) -> int:
    return int(lib().mxq_bf16_grouped_mm_workspace_bytes(int(product), int(M), int(N), int(K), int(G)))


def _bytes(t) -> int:
    """Size of a workspace that may be None."""
    return 0 if t is None else t.numel() * t.element_size()


def mxq_bf16_grouped_mm(x: torch.Tensor, w: torch.Tensor, group_end_offs: torch.Tensor, y: torch.Tensor, workspace=None,
                        stream=None) -> None:
    """x (M, K), w (G, N, K) bf16, group_end_offs int32[G] (device) -> y (M, N) bf16 or float32."""
    if x.dim() != 2 or w.dim() != 3 or y.dim() != 2:
        raise ValueError("x must be (M, K), w (G, N, K) and y (M, N)")
    M, K = x.shape
    G, N, Kw = w.shape
    if Kw != K or tuple(y.shape) != (M, N):
        raise ValueError("operand shapes do not match")
    px, pw = _dev(x, "x", torch.bfloat16), _dev(w, "w", torch.bfloat16)
    po = _dev(group_end_offs, "group_end_offs", torch.int32, G)
    code, py = _float_code(y, "y"), _dev(y, "y")
    _check(lib().mxq_bf16_grouped_mm(px, pw, po, M, N, K, G, code, py, _opt(workspace, "workspace"), _bytes(workspace),
                                     _stream(stream)), "mxq_bf16_grouped_mm")


def mxq_bf16_grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, group_end_offs: torch.Tensor, dx: torch.Tensor,
                           workspace=None, stream=None) -> None:
    """dy (M, N), w (G, N, K) bf16, group_end_offs int32[G] (device) -> dx (M, K) bf16 or float32."""
    if dy.dim() != 2 or w.dim() != 3 or dx.dim() != 2:
        raise ValueError("dy must be (M, N), w (G, N, K) and dx (M, K)")
    G, N, K = w.shape
    M = dy.shape[0]
    if dy.shape[1] != N or tuple(dx.shape) != (M, K):
        raise ValueError("operand shapes do not match")
    pd, pw = _dev(dy, "dy", torch.bfloat16), _dev(w, "w", torch.bfloat16)
    po = _dev(group_end_offs, "group_end_offs", torch.int32, G)
    code, px = _float_code(dx, "dx"), _dev(dx, "dx")
    _check(lib().mxq_bf16_grouped_mm_dx(pd, pw, po, M, N, K, G, code, px, _opt(workspace, "workspace"), _bytes(workspace),
                                        _stream(stream)), "mxq_bf16_grouped_mm_dx")


def mxq_bf16_grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, group_end_offs: torch.Tensor, dw: torch.Tensor,
                           accumulate: bool = False, workspace=None, stream=None) -> None:
    """dy (M, N), x (M, K) bf16, group_end_offs int32[G] (device) -> dw (G, N, K) bf16 or float32; with accumulate
    the sums are added to the float32 dw."""
    if dy.dim() != 2 or x.dim() != 2 or dw.dim() != 3:
        raise ValueError("dy must be (M, N), x (M, K) and dw (G, N, K)")
    G, N, K = dw.shape
    M = dy.shape[0]
    if dy.shape[1] != N or tuple(x.shape) != (M, K):
        raise ValueError("operand shapes do not match")
    pd, px = _dev(dy, "dy", torch.bfloat16), _dev(x, "x", torch.bfloat16)
    po = _dev(group_end_offs, "group_end_offs", torch.int32, G)
    code, pw = _float_code(dw, "dw"), _dev(dw, "dw")
    _check(lib().mxq_bf16_grouped_mm_dw(pd, px, po, M, N, K, G, code, int(bool(accumulate)), pw,
                                        _opt(workspace, "workspace"), _bytes(workspace), _stream(stream)),
           "mxq_bf16_grouped_mm_dw")


# ------------------------------------------------------------- layer norm ---
def mxq_add_layernorm(x: torch.Tensor, residual, weight: torch.Tensor, bias, eps: float, h=None, y=None, q=None, s=None,
                      mean=None, rstd=None, stream=None) -> None:
    """x (+ residual) (M, K), weight (K) and bias (K) or None, bf16 or float32 -> h = x + residual, y = the layer norm of
    h (their type), q (M, K) / s (M, K/32) uint8 = MXFP8 of y, mean and rstd (M) float32; outputs may be None."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    code, dt, n = _float_code(x, "x"), x.dtype, M * K
    px = _dev(x, "x")
    pr = _opt(residual, "residual", dt, n)
    pw = _dev(weight, "weight", dt, K)
    pb = _opt(bias, "bias", dt, K)
    ph = _opt(h, "h", dt, n)
    py = _opt(y, "y", dt, n)
    pq = _opt(q, "q", torch.uint8, n)
    ps = _opt(s, "s", torch.uint8, M * (K // 32) if K % 32 == 0 else None)
    pm = _opt(mean, "mean", torch.float32, M)
    pd = _opt(rstd, "rstd", torch.float32, M)
    _check(lib().mxq_add_layernorm(px, pr, pw, pb, code, M, K, float(eps), ph, py, pq, ps, pm, pd, _stream(stream)),
           "mxq_add_layernorm")


def mxq_add_layernorm_bwd_workspace_bytes(M: int, K: int) -> int:
    return int(lib().mxq_add_layernorm_bwd_workspace_bytes(int(M), int(K)))


def mxq_add_layernorm_bwd(h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor,
                          dh, dx: torch.Tensor, dweight: torch.Tensor, dbias, workspace: torch.Tensor, stream=None) -> None:
    """h, mean, rstd of mxq_add_layernorm and the gradients dy, dh (or None) -> dx (M, K), dweight (K) and dbias (K, or
    None) float32."""
    if h.dim() != 2:
        raise ValueError("h must be 2-D (M, K)")
    M, K = h.shape
    code, dt, n = _float_code(h, "h"), h.dtype, M * K
    ph = _dev(h, "h")
    pw = _dev(weight, "weight", dt, K)
    pm = _dev(mean, "mean", torch.float32, M)
    pr = _dev(rstd, "rstd", torch.float32, M)
    pg = _dev(dy, "dy", dt, n)
    pd = _opt(dh, "dh", dt, n)
    px = _dev(dx, "dx", dt, n)
    pk = _dev(dweight, "dweight", torch.float32, K)
    pb = _opt(dbias, "dbias", torch.float32, K)
    pws = _dev(workspace, "workspace")
    _check(lib().mxq_add_layernorm_bwd(ph, pw, pm, pr, pg, pd, code, M, K, px, pk, pb, pws, _bytes(workspace),
                                       _stream(stream)), "mxq_add_layernorm_bwd")


# --------------------------------------------- rows to the experts and back ---
def mxq_dispatch_rows_workspace_bytes(M: int, topk: int, E: int) -> int:
    return int(lib().mxq_dispatch_rows_workspace_bytes(int(M), int(topk), int(E)))


def mxq_dispatch_rows(x: torch.Tensor, expert_ids: torch.Tensor, E: int, rows: torch.Tensor, group_end_offs: torch.Tensor,
                      src_pair: torch.Tensor, pair_row: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """x (M, K) bf16 or float32, expert_ids (M, topk) int32 -> rows (M*topk, K) sorted stably by expert,
    group_end_offs int32[E], src_pair int32[M*topk], pair_row int32 (M, topk)."""
    if x.dim() != 2 or expert_ids.dim() != 2 or expert_ids.shape[0] != x.shape[0]:
        raise ValueError("x must be (M, K) and expert_ids (M, topk)")
    M, K = x.shape
    topk = expert_ids.shape[1]
    code = _float_code(x, "x")
    px = _dev(x, "x")
    pi = _dev(expert_ids, "expert_ids", torch.int32)
    pr = _dev(rows, "rows", x.dtype, M * topk * K)
    pe = _dev(group_end_offs, "group_end_offs", torch.int32, int(E))
    ps = _dev(src_pair, "src_pair", torch.int32, M * topk)
    pp = _dev(pair_row, "pair_row", torch.int32, M * topk)
    pw = _dev(workspace, "workspace")
    _check(lib().mxq_dispatch_rows(px, code, M, K, pi, topk, int(E), pr, pe, ps, pp, pw, _bytes(workspace),
                                   _stream(stream)), "mxq_dispatch_rows")


def mxq_pair_rows(src_pair: torch.Tensor, pair_row: torch.Tensor, stream=None) -> None:
    """src_pair int32 (a dispatch's) -> pair_row int32, its inverse, as many elements."""
    n = src_pair.numel()
    ps = _dev(src_pair, "src_pair", torch.int32)
    pp = _dev(pair_row, "pair_row", torch.int32, n)
    _check(lib().mxq_pair_rows(ps, n, pp, _stream(stream)), "mxq_pair_rows")


def mxq_combine_rows(rows: torch.Tensor, pair_row: torch.Tensor, weights, out: torch.Tensor, stream=None) -> None:
    """rows (R, K) bf16 or float32, pair_row (M, topk) int32, weights (M, topk) float32 or None -> out (M, K)."""
    if rows.dim() != 2 or pair_row.dim() != 2:
        raise ValueError("rows must be (R, K) and pair_row (M, topk)")
    R, K = rows.shape
    M, topk = pair_row.shape
    code = _float_code(rows, "rows")
    pr = _dev(rows, "rows")
    pp = _dev(pair_row, "pair_row", torch.int32)
    pw = _opt(weights, "weights", torch.float32, M * topk)
    po = _dev(out, "out", rows.dtype, M * K)
    _check(lib().mxq_combine_rows(pr, code, R, K, pp, M, topk, pw, po, _stream(stream)), "mxq_combine_rows")


def mxq_combine_rows_bwd(dout: torch.Tensor, rows, pair_row: torch.Tensor, weights, drows: torch.Tensor, dweights=None,
                         stream=None) -> None:
    """dout (M, K), rows (R, K) or None (without dweights), pair_row (M, topk) int32, weights (M, topk) float32 or None
    -> drows (R, K) of dout's type, dweights (M, topk) float32 or None."""
    if dout.dim() != 2 or drows.dim() != 2 or pair_row.dim() != 2:
        raise ValueError("dout must be (M, K), drows (R, K) and pair_row (M, topk)")
    R, K = drows.shape
    M, topk = pair_row.shape
    code, dt = _float_code(dout, "dout"), dout.dtype
    pd = _dev(dout, "dout", dt, M * K)
    pr = _opt(rows, "rows", dt, R * K)
    pp = _dev(pair_row, "pair_row", torch.int32)
    pw = _opt(weights, "weights", torch.float32, M * topk)
    px = _dev(drows, "drows", dt)
    pk = _opt(dweights, "dweights", torch.float32, M * topk)
    _check(lib().mxq_combine_rows_bwd(pd, pr, code, R, K, pp, M, topk, pw, px, pk, _stream(stream)),
           "mxq_combine_rows_bwd")
