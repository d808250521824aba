"""The routed-expert operators in plain numpy, 64 bits, straight from their
definitions: what the GPU tests compare the kernels with."""
import numpy as np

TINY = 1e-20


# ------------------------------------------------------------------ formats --
def bf16_round(x):
    """float64 -> the nearest bf16 (ties to even) as float64; finite inputs in bf16's normal range."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def half_step(x, dtype):
    """Half the distance between neighbouring values of "bf16" at x (8 significant bits); 0 for "f32" (whose
    rounding the callers count with the fp32 arithmetic)."""
    if dtype != "bf16":
        return 0.0
    return np.where(x == 0, 0.0, np.ldexp(1.0, np.frexp(np.abs(x))[1] - 9))


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3_value(q):
    q = np.asarray(q, np.uint8).astype(np.int64)
    e, m = (q >> 3) & 15, (q & 7).astype(np.float64)
    v = np.where(e > 0, np.ldexp(1 + m / 8, e - 7), np.ldexp(m, -9))
    return np.where(q & 0x80, -v, v)


def mxfp4_encode(x, rule):
    """x (M, K) float64 values of bf16 -> (q (M, K/2), s (M, K/32)) uint8; rule 0 floor, 1 round up."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    z = np.where(np.isfinite(b), b, 0.0)
    amax = np.abs(z).max(-1)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)
    if rule:
        e = e + (amax > np.ldexp(6.0, e))
    e = np.maximum(e, -127)
    a = np.abs(z) / np.ldexp(1.0, e)[..., None]
    # nearest of the eight magnitudes, ties to the even code
    mid = (E2M1[1:8] + E2M1[:7]) / 2
    up = np.array([False, True] * 4)[:7]                 # the upper neighbour of midpoint i is code i + 1: even for odd i
    code = sum(((a > mid[i]) | ((a == mid[i]) & up[i])).astype(np.int64) for i in range(7))
    code = code + 8 * np.signbit(z)
    code = np.where(bad[..., None], 0, code).reshape(M, K)
    s = np.where(bad, 255, e + 127)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), s.astype(np.uint8)


def mxfp4_decode(q, s):
    """(rows, K/2), (rows, K/32) -> float64 (rows, K); scale 0xFF gives NaN."""
    q = np.asarray(q, np.uint8)
    v = E2M1[np.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)]
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return v * np.repeat(f, 32, axis=1)


def past_bf16_is_inf(v):
    """Values past bf16's largest become infinities (the values here have few digits: nothing else is rounded)."""
    return np.where(np.abs(v) >= 2.0 ** 128, np.sign(v) * np.inf, v)


def mxfp8_decode(q, s):
    return e4m3_value(q) * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, axis=1)


# --------------------------------------------------------------------- norm --
def norm_fwd(h, w, eps):
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * w, rstd


def norm_bwd(h, w, rstd, dy, dh):
    n = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(-1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * n).sum(0)


# ------------------------------------------------------------------ routing --
def scores(l, sigmoid):
    with np.errstate(all="ignore"):
        if sigmoid:
            return np.where(l > -np.inf, 1.0 / (1.0 + np.exp(-l)), 0.0)
        m = l.max(-1, keepdims=True)
        e = np.where(l > -np.inf, np.exp(l - np.where(m > -np.inf, m, 0.0)), 0.0)
        t = e.sum(-1, keepdims=True)
        return e / np.where(t > 0, t, 1.0)


def route(l, bias, sigmoid, n_groups, topk_groups, topk, renorm, top2, scale):
    """(ids, weights, decided): `decided` marks the rows whose selection no rounding of 1e-5 (of the largest
    key in size) can change; equal keys are decided by their index when they are equal logits."""
    M, E = l.shape
    s = scores(l, sigmoid)
    key = l if bias is None else s + bias
    val = s if bias is None else key
    ids = np.full((M, topk), -1, np.int64)
    w = np.zeros((M, topk))
    decided = np.ones(M, bool)
    gs = E // n_groups
    for m in range(M):
        ok = (l[m] > -np.inf) & (key[m] > -np.inf)
        if topk_groups < n_groups:
            gv = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                t = np.sort(val[m, g * gs:(g + 1) * gs][ok[g * gs:(g + 1) * gs]])[::-1]
                if len(t):
                    gv[g] = t[0] + t[1] if top2 and len(t) > 1 else t[0]
            order = np.argsort(-gv, kind="stable")
            if abs(gv[order[topk_groups - 1]] - gv[order[topk_groups]]) <= 1e-5 * max(1e-300, np.abs(gv[gv > -np.inf]).max(initial=0.0)):
                decided[m] = False
            keep = np.zeros(n_groups, bool)
            keep[order[:topk_groups]] = True
            ok = ok & np.repeat(keep, gs)
        k = np.where(ok, key[m], -np.inf)
        order = np.argsort(-k, kind="stable")
        n = min(topk, int(ok.sum()))
        sel = order[:n]
        ids[m, :n] = sel
        if bias is not None:
            top = k[order[:min(n + 1, int(ok.sum()))]]
            if len(top) > 1 and (np.abs(np.diff(top)) <= 1e-5 * np.abs(top).max()).any():
                decided[m] = False
        ws = s[m, sel]
        w[m, :n] = scale * (ws / (ws.sum() + TINY) if renorm else ws)
    return ids, w, decided


def route_bwd(l, ids, dw, sigmoid, renorm, scale):
    s = scores(l, sigmoid)
    d = np.zeros_like(s)
    for m in range(l.shape[0]):
        at = np.nonzero(ids[m] >= 0)[0]
        e = ids[m, at]
        g = scale * dw[m, at]
        if renorm:
            t = s[m, e].sum() + TINY
            g = g / t - (g * s[m, e]).sum() / t ** 2
        up = np.zeros(l.shape[1])
        up[e] = g
        d[m] = up * s[m] * (1 - s[m]) if sigmoid else s[m] * (up - (up * s[m]).sum())
    return d


# ------------------------------------------------------------------ product --
def group_spans(ends, M):
    """Clamped rows [a, b) of each group: running maximum of the ends, cut to [0, M]."""
    spans, prev = [], 0
    for e in ends:
        end = min(max(int(e), prev), M)
        spans.append((prev, end))
        prev = end
    return spans


def product(x, w, ends):
    """x (M, K), w (G, N, K) float64 -> (y, sum of magnitudes), rows past the last end zero."""
    y = np.zeros((x.shape[0], w.shape[1]))
    a = np.zeros_like(y)
    for g, (p, q) in enumerate(group_spans(ends, x.shape[0])):
        y[p:q] = x[p:q] @ w[g].T
        a[p:q] = np.abs(x[p:q]) @ np.abs(w[g]).T
    return y, a
