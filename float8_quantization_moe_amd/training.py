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


def _scratch(like: torch.Tensor, size: int):
    """(tensor to keep, address, bytes) of a workspace on like's device."""
    if size == 0:
        return None, 0, 0
    t = like.new_empty(size, dtype=torch.uint8)
    return t, t.data_ptr(), size


# (Outputs and workspaces made here need no checks, so the helpers call the library themselves:
# a small call is host time.)

# ------------------------------------------------------------- products ---
def _out_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return mxq.MXQ_OUT_BF16
    if dtype == torch.float32:
        return mxq.MXQ_OUT_F32
    raise TypeError(f"out_dtype must be bfloat16 or float32, got {dtype}")


def bf16_grouped_mm(x: torch.Tensor, w: torch.Tensor, group_end_offs: torch.Tensor, out_dtype=torch.bfloat16,
                    stream=None) -> torch.Tensor:
    """y (M, N) = each row of x (M, K) times its group's w (G, N, K) transposed."""
    if stream is not None:
        with _on(stream, x):
            return bf16_grouped_mm(x, w, group_end_offs, out_dtype)
    if x.dim() != 2 or w.dim() != 3 or x.shape[1] != w.shape[2]:
        raise ValueError("x must be (M, K) and w (G, N, K)")
    M, (G, N, K) = x.shape[0], w.shape
    code, L = _out_code(out_dtype), mxq.lib()
    px, pw = mxq._dev(x, "x", torch.bfloat16), mxq._dev(w, "w", torch.bfloat16)
    po = mxq._dev(group_end_offs, "group_end_offs", torch.int32, G)
    y = x.new_empty((M, N), dtype=out_dtype)
    ws, at, size = _scratch(x, L.mxq_bf16_grouped_mm_workspace_bytes(mxq.MXQ_PRODUCT_Y, M, N, K, G))
    mxq._check(L.mxq_bf16_grouped_mm(px, pw, po, M, N, K, G, code, y.data_ptr(), at, size, mxq._stream(None)),
               "mxq_bf16_grouped_mm")
    return y


def bf16_grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, group_end_offs: torch.Tensor, out_dtype=torch.bfloat16,
                       stream=None) -> torch.Tensor:
    """dx (M, K) = each row of dy (M, N) times its group's w (G, N, K)."""
    if stream is not None:
        with _on(stream, dy):
            return bf16_grouped_mm_dx(dy, w, group_end_offs, out_dtype)
    if dy.dim() != 2 or w.dim() != 3 or dy.shape[1] != w.shape[1]:
        raise ValueError("dy must be (M, N) and w (G, N, K)")
    M, (G, N, K) = dy.shape[0], w.shape
    code, L = _out_code(out_dtype), mxq.lib()
    pd, pw = mxq._dev(dy, "dy", torch.bfloat16), mxq._dev(w, "w", torch.bfloat16)
    po = mxq._dev(group_end_offs, "group_end_offs", torch.int32, G)
    dx = dy.new_empty((M, K), dtype=out_dtype)
    ws, at, size = _scratch(dy, L.mxq_bf16_grouped_mm_workspace_bytes(mxq.MXQ_PRODUCT_DX, M, N, K, G))
    mxq._check(L.mxq_bf16_grouped_mm_dx(pd, pw, po, M, N, K, G, code, dx.data_ptr(), at, size, mxq._stream(None)),
               "mxq_bf16_grouped_mm_dx")
    return dx


def bf16_grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, group_end_offs: torch.Tensor, out_dtype=torch.float32, dw=None,
                       stream=None) -> torch.Tensor:
    """dw (G, N, K) = each group's sum of dy (M, N)'s rows times x (M, K)'s; a float32 dw that is given is added to,
    in place, and returned."""
    if stream is not None:
        with _on(stream, dy):
            return bf16_grouped_mm_dw(dy, x, group_end_offs, out_dtype, dw)
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be (M, N) and x (M, K)")
    (M, N), K, G = dy.shape, x.shape[1], group_end_offs.numel()
    add = dw is not None
    if add and tuple(dw.shape) != (G, N, K):
        raise ValueError("dw must be (G, N, K)")
    L = mxq.lib()
    pd, px = mxq._dev(dy, "dy", torch.bfloat16), mxq._dev(x, "x", torch.bfloat16)
    po = mxq._dev(group_end_offs, "group_end_offs", torch.int32)
    if add:
        code, pw = mxq._float_code(dw, "dw"), mxq._dev(dw, "dw")
    else:
        code, dw = _out_code(out_dtype), dy.new_empty((G, N, K), dtype=out_dtype)
        pw = dw.data_ptr()
    ws, at, size = _scratch(dy, L.mxq_bf16_grouped_mm_workspace_bytes(mxq.MXQ_PRODUCT_DW, M, N, K, G))
    mxq._check(L.mxq_bf16_grouped_mm_dw(pd, px, po, M, N, K, G, code, int(add), pw, at, size, mxq._stream(None)),
               "mxq_bf16_grouped_mm_dw")
    return dw


# ----------------------------------------------------------- layer norm ---
def add_layernorm(x: torch.Tensor, residual, weight: torch.Tensor, bias, eps: float, stream=None):
    """(h, y, q, s, mean, rstd) of mxq_add_layernorm; h is x itself when there is no residual.  The codes need K % 32 == 0:
    other widths, and rows without codes, go to mxq.mxq_add_layernorm."""
    if stream is not None:
        with _on(stream, x):
            return add_layernorm(x, residual, weight, bias, eps)
    if x.dim() != 2:
        raise ValueError("x must be 2-D (M, K)")
    M, K = x.shape
    code, dt = mxq._float_code(x, "x"), x.dtype
    px, pr = mxq._dev(x, "x"), mxq._opt(residual, "residual", dt, M * K)
    pw, pb = mxq._dev(weight, "weight", dt, K), mxq._opt(bias, "bias", dt, K)
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
    code, dt, n, L = mxq._float_code(h, "h"), h.dtype, M * K, mxq.lib()
    ph, pw = mxq._dev(h, "h"), mxq._dev(weight, "weight", dt, K)
    pm, pr = mxq._dev(mean, "mean", torch.float32, M), mxq._dev(rstd, "rstd", torch.float32, M)
    pg, pd = mxq._dev(dy, "dy", dt, n), mxq._opt(dh, "dh", dt, n)
    dx = torch.empty_like(h)
    dweight = h.new_empty(K, dtype=torch.float32)
    dbias = h.new_empty(K, dtype=torch.float32)
    ws, at, size = _scratch(h, L.mxq_add_layernorm_bwd_workspace_bytes(M, K))
    mxq._check(L.mxq_add_layernorm_bwd(ph, pw, pm, pr, pg, pd, code, M, K, dx.data_ptr(), dweight.data_ptr(),
                                       dbias.data_ptr(), at, size, mxq._stream(None)), "mxq_add_layernorm_bwd")
    return dx, dweight, dbias


# ----------------------------------------------------------------- rows ---
def dispatch_rows(x: torch.Tensor, expert_ids: torch.Tensor, E: int, stream=None):
    """(rows, group_end_offs, src_pair, pair_row) of mxq_dispatch_rows."""
    if stream is not None:
        with _on(stream, x):
            return dispatch_rows(x, expert_ids, E)
    if x.dim() != 2 or expert_ids.dim() != 2 or x.shape[0] != expert_ids.shape[0]:
        raise ValueError("x must be (M, K) and expert_ids (M, topk)")
    K, (M, topk), E = x.shape[1], expert_ids.shape, int(E)
    code, L = mxq._float_code(x, "x"), mxq.lib()
    px, pi = mxq._dev(x, "x"), mxq._dev(expert_ids, "expert_ids", torch.int32)
    rows = x.new_empty((M * topk, K))
    ends = x.new_empty(E, dtype=torch.int32)
    src = x.new_empty(M * topk, dtype=torch.int32)
    place = x.new_empty((M, topk), dtype=torch.int32)
    ws, at, size = _scratch(x, L.mxq_dispatch_rows_workspace_bytes(M, topk, E))
    mxq._check(L.mxq_dispatch_rows(px, code, M, K, pi, topk, E, rows.data_ptr(), ends.data_ptr(), src.data_ptr(),
                                   place.data_ptr(), at, size, mxq._stream(None)), "mxq_dispatch_rows")
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
    (R, K), (M, topk) = rows.shape, pair_row.shape
    code, pr = mxq._float_code(rows, "rows"), mxq._dev(rows, "rows")
    pp, pw = mxq._dev(pair_row, "pair_row", torch.int32), mxq._opt(weights, "weights", torch.float32, M * topk)
    out = rows.new_empty((M, K))
    mxq._check(mxq.lib().mxq_combine_rows(pr, code, R, K, pp, M, topk, pw, out.data_ptr(), mxq._stream(None)),
               "mxq_combine_rows")
    return out


def combine_rows_bwd(dout: torch.Tensor, rows: torch.Tensor, pair_row: torch.Tensor, weights=None, stream=None):
    """(drows, dweights) of mxq_combine_rows_bwd; rows that no pair names are left as allocated.  drows alone, without reading
    rows: mxq.mxq_combine_rows_bwd."""
    if stream is not None:
        with _on(stream, dout):
            return combine_rows_bwd(dout, rows, pair_row, weights)
    if dout.dim() != 2 or rows.dim() != 2 or pair_row.dim() != 2:
        raise ValueError("dout must be (M, K), rows (R, K) and pair_row (M, topk)")
    (R, K), (M, topk), dt = rows.shape, pair_row.shape, dout.dtype
    code, pd, pr = mxq._float_code(dout, "dout"), mxq._dev(dout, "dout", dt, M * K), mxq._dev(rows, "rows", dt)
    pp, pw = mxq._dev(pair_row, "pair_row", torch.int32), mxq._opt(weights, "weights", torch.float32, M * topk)
    drows = torch.empty_like(rows)
    dweights = dout.new_empty((M, topk), dtype=torch.float32)
    mxq._check(mxq.lib().mxq_combine_rows_bwd(pd, pr, code, R, K, pp, M, topk, pw, drows.data_ptr(), dweights.data_ptr(),
                                              mxq._stream(None)), "mxq_combine_rows_bwd")
    return drows, dweights
