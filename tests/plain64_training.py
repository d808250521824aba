"""The operators of a training step of routed experts in plain numpy, 64 bits, straight from
their definitions: what the GPU tests compare the kernels with."""
import numpy as np

from plain64 import group_spans


# --------------------------------------------------------------- layer norm --
def layernorm_fwd(h, w, b, eps):
    """(y, mean, rstd) of rows h; b may be None."""
    mean = h.mean(-1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[:, None] * w
    return y + (0 if b is None else b), mean, rstd


def layernorm_bwd(h, w, mean, rstd, dy, dh):
    """(dx, dw, db)."""
    n = (h - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * n).sum(0), dy.sum(0)


# --------------------------------------------------------------------- rows --
def dispatch_order(ids, E):
    """(ends (E), src_pair (P), pair_row like ids) of a stable counting sort; ids outside [0, E) are dropped."""
    flat = ids.reshape(-1)
    kept = [p for e in range(E) for p in np.nonzero(flat == e)[0]]
    src = np.full(flat.size, -1, np.int32)
    src[:len(kept)] = kept
    row = np.full(flat.size, -1, np.int32)
    row[kept] = np.arange(len(kept))
    ends = np.cumsum([(flat == e).sum() for e in range(E)]).astype(np.int32)
    return ends, src, row.reshape(ids.shape)


def combine(rows, pair_row, weights):
    """(out, sum of magnitudes); entries of pair_row outside the rows add nothing."""
    M, topk = pair_row.shape
    out = np.zeros((M, rows.shape[1]))
    size = np.zeros_like(out)
    for t in range(M):
        for j in range(topk):
            r = pair_row[t, j]
            if 0 <= r < rows.shape[0]:
                term = (1.0 if weights is None else weights[t, j]) * rows[r]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_bwd(dout, rows, pair_row, weights):
    """(drows with NaN in rows that no pair names, dweights, sum of dweights' magnitudes)."""
    drows = np.full(rows.shape, np.nan)
    dw, size = np.zeros(pair_row.shape), np.zeros(pair_row.shape)
    for (t, j), r in np.ndenumerate(pair_row):
        if 0 <= r < rows.shape[0]:
            drows[r] = (1.0 if weights is None else weights[t, j]) * dout[t]
            dw[t, j] = (dout[t] * rows[r]).sum()
            size[t, j] = np.abs(dout[t] * rows[r]).sum()
    return drows, dw, size


# ----------------------------------------------------------------- products --
def product_dx(dy, w, ends):
    """(dx, sum of magnitudes), rows past the last end zero."""
    dx = np.zeros((dy.shape[0], w.shape[2]))
    a = np.zeros_like(dx)
    for g, (p, q) in enumerate(group_spans(ends, dy.shape[0])):
        dx[p:q] = dy[p:q] @ w[g]
        a[p:q] = np.abs(dy[p:q]) @ np.abs(w[g])
    return dx, a


def product_dw(dy, x, ends):
    """(dw (G, N, K), sum of magnitudes)."""
    dw = np.zeros((len(ends), dy.shape[1], x.shape[1]))
    a = np.zeros_like(dw)
    for g, (p, q) in enumerate(group_spans(ends, dy.shape[0])):
        dw[g] = dy[p:q].T @ x[p:q]
        a[g] = np.abs(dy[p:q]).T @ np.abs(x[p:q])
    return dw, a
