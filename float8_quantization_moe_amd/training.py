"""Helpers of a training step of routed experts: the bf16 products and their gradients, the layer norm,
and the rows' way to their experts and back.

They allocate outputs and workspaces with torch and call the entry points of ``mxq``, as the helpers
there do; given a stream (a torch stream or a raw handle) they run as they would under
``with torch.cuda.stream(stream):``, allocations included, and the caller orders that stream after the
work that makes the inputs.  A ``stream`` of None is the current one.
"""
from __future__ import annotations

import torch

from . import mxq


def _on(stream, t: torch.Tensor):
    """The context in which a helper given `stream` runs."""
    return torch.cuda.stream(mxq._stream_of(stream, t))


def _workspace(like: torch.Tensor, size: int):
    """Scratch of `size` bytes on like's device; None for none."""
    return like.new_empty(size, dtype=torch.uint8) if size else None


# ------------------------------------------------------------- products ---
def bf16_grouped_mm(x: torch.Tensor, w: torch.Tensor, group_end_offs: torch.Tensor, out_dtype=torch.bfloat16,
                    stream=None) -> torch.Tensor:
    """y (M, N) = each row of x (M, K) times its group's w (G, N, K) transposed."""
    if stream is not None:
        with _on(stream, x):
            return bf16_grouped_mm(x, w, group_end_offs, out_dtype)
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x must be (M, K) and w (G, N, K)")
    M, (G, N, K) = x.shape[0], w.shape
    y = x.new_empty((M, N), dtype=out_dtype)
    ws = _workspace(x, mxq.mxq_bf16_grouped_mm_workspace_bytes(mxq.MXQ_PRODUCT_Y, M, N, K, G))
    mxq.mxq_bf16_grouped_mm(x, w, group_end_offs, y, ws)
    return y


def bf16_grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, group_end_offs: torch.Tensor, out_dtype=torch.bfloat16,
                       stream=None) -> torch.Tensor:
    """dx (M, K) = each row of dy (M, N) times its group's w (G, N, K)."""
    if stream is not None:
        with _on(stream, dy):
            return bf16_grouped_mm_dx(dy, w, group_end_offs, out_dtype)
    if dy.dim() != 2 or w.dim() != 3:
        raise ValueError("dy must be (M, N) and w (G, N, K)")
    M, (G, N, K) = dy.shape[0], w.shape
    dx = dy.new_empty((M, K), dtype=out_dtype)
    ws = _workspace(dy, mxq.mxq_bf16_grouped_mm_workspace_bytes(mxq.MXQ_PRODUCT_DX, M, N, K, G))
    mxq.mxq_bf16_grouped_mm_dx(dy, w, group_end_offs, dx, ws)
    return dx


def bf16_grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, group_end_offs: torch.Tensor, out_dtype=torch.float32, dw=None,
                       stream=None) -> torch.Tensor:
    """dw (G, N, K) = each group's sum of dy (M, N)'s rows times x (M, K)'s; a float32 dw that is given is added to,
    in place, and returned."""
    if stream is not None:
        with _on(stream, dy):
            return bf16_grouped_mm_dw(dy, x, group_end_offs, out_dtype, dw)
    if dy.dim() != 2 or x.dim() != 2:
        raise ValueError("dy must be (M, N) and x (M, K)")
    (M, N), K, G = dy.shape, x.shape[1], group_end_offs.numel()
    add = dw is not None
    if add and tuple(dw.shape) != (G, N, K):
        raise ValueError("dw must be (G, N, K)")
    if not add:
        dw = dy.new_empty((G, N, K), dtype=out_dtype)
    ws = _workspace(dy, mxq.mxq_bf16_grouped_mm_workspace_bytes(mxq.MXQ_PRODUCT_DW, M, N, K, G))
    mxq.mxq_bf16_grouped_mm_dw(dy, x, group_end_offs, dw, add, ws)
    return dw


# ----------------------------------------------------------- layer norm ---
def add_layernorm(x: torch.Tensor, residual, weight: torch.Tensor, bias, eps: float, stream=None):
    """(h, y, q, s, mean, rstd) of mxq_add_layernorm; h is x itself when there is no residual."""
    if stream is not None:
        with _on(stream, x):
            return add_layernorm(x, residual, weight, bias, eps)
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    code, dt = mxq._float_code(x, "x"), x.dtype
    px, pr = mxq._dev(x, "x"), mxq._opt(residual, "residual", dt, M * K)
    pw, pb = mxq._dev(weight, "weight", dt, K), mxq._opt(bias, "bias", dt, K)
    # (outputs made here need no checks: a token's norm is host time)
    h = x if residual is None else torch.empty_like(x)
    y = torch.empty_like(x)
    q = torch.empty_like(x, dtype=torch.uint8)
    s = x.new_empty((M, K // 32), dtype=torch.uint8)
    mean = x.new_empty(M, dtype=torch.float32)
    rstd = x.new_empty(M, dtype=torch.float32)
    mxq._check(mxq.lib().mxq_add_layernorm(px, pr, pw, pb, code, M, K, eps, 0 if residual is None else h.data_ptr(),
                                           y.data_ptr(), q.data_ptr(), s.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                           mxq._stream(None)), "mxq_add_layernorm")
    return h, y, q, s, mean, rstd


def add_layernorm_bwd(h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor,
                      dh=None, stream=None):
    """(dx, dweight, dbias) of mxq_add_layernorm_bwd."""
    if stream is not None:
        with _on(stream, h):
            return add_layernorm_bwd(h, weight, mean, rstd, dy, dh)
    if h.dim() != 2:
        raise ValueError("h must be 2-D (M, K)")
    M, K = h.shape
    dx = torch.empty_like(h)
    dweight = h.new_empty(K, dtype=torch.float32)
    dbias = h.new_empty(K, dtype=torch.float32)
    ws = h.new_empty(max(mxq.mxq_add_layernorm_bwd_workspace_bytes(M, K), 16), dtype=torch.uint8)
    mxq.mxq_add_layernorm_bwd(h, weight, mean, rstd, dy, dh, dx, dweight, dbias, ws)
    return dx, dweight, dbias


# ----------------------------------------------------------------- rows ---
def dispatch_rows(x: torch.Tensor, expert_ids: torch.Tensor, E: int, stream=None):
    """(rows, group_end_offs, src_pair, pair_row) of mxq_dispatch_rows."""
    if stream is not None:
        with _on(stream, x):
            return dispatch_rows(x, expert_ids, E)
    if x.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("x must be (M, K) and expert_ids (M, topk)")
    K, (M, topk) = x.shape[1], expert_ids.shape
    rows = x.new_empty((M * topk, K))
    ends = x.new_empty(int(E), dtype=torch.int32)
    src = x.new_empty(M * topk, dtype=torch.int32)
    place = x.new_empty((M, topk), dtype=torch.int32)
    ws = x.new_empty(max(mxq.mxq_dispatch_rows_workspace_bytes(M, topk, E), 16), dtype=torch.uint8)
    mxq.mxq_dispatch_rows(x, expert_ids, E, rows, ends, src, place, ws)
    return rows, ends, src, place


def pair_rows(src_pair: torch.Tensor, topk: int, stream=None) -> torch.Tensor:
    """pair_row (M, topk) of a dispatch's src_pair (M*topk)."""
    if stream is not None:
        with _on(stream, src_pair):
            return pair_rows(src_pair, topk)
    place = src_pair.new_empty((src_pair.numel() // topk, topk), dtype=torch.int32)
    mxq.mxq_pair_rows(src_pair, place)
    return place


def combine_rows(rows: torch.Tensor, pair_row: torch.Tensor, weights=None, stream=None) -> torch.Tensor:
    """out (M, K) of mxq_combine_rows."""
    if stream is not None:
        with _on(stream, rows):
            return combine_rows(rows, pair_row, weights)
    if rows.dim() != 2 or pair_row.dim() != 2:
        raise ValueError("rows must be (R, K) and pair_row (M, topk)")
    out = rows.new_empty((pair_row.shape[0], rows.shape[1]))
    mxq.mxq_combine_rows(rows, pair_row, weights, out)
    return out


def combine_rows_bwd(dout: torch.Tensor, rows: torch.Tensor, pair_row: torch.Tensor, weights=None, stream=None):
    """(drows, dweights) of mxq_combine_rows_bwd; rows that no pair names are left as allocated."""
    if stream is not None:
        with _on(stream, dout):
            return combine_rows_bwd(dout, rows, pair_row, weights)
    if rows.dim() != 2 or pair_row.dim() != 2:
        raise ValueError("rows must be (R, K) and pair_row (M, topk)")
    drows = torch.empty_like(rows)
    dweights = dout.new_empty(pair_row.shape, dtype=torch.float32)
    mxq.mxq_combine_rows_bwd(dout, rows, pair_row, weights, drows, dweights)
    return drows, dweights
