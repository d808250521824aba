"""Cases of the routed-expert operators around the float8 buffers, for measurement.

Four operators, each as a user's program calls it:

  norm     residual addition + root-mean-square norm with the row's MXFP8 codes beside the normalised
           row (forward), and its gradients (backward);
  route    expert routing: scores, balance bias, groups, top-k, weights (forward), and the logits'
           gradient (backward);
  mxfp4    MXFP4 codes and scales of a bf16 tensor, and their decoding (one exchange's two ends);
  product  grouped product of MXFP8 or MXFP4 token rows with MXFP4 expert weights.

`own` selects the framework's kernels; otherwise the same results come from elementary torch
operations in 32 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-5            # of the norm
TINY = 1e-20          # added to a sum of selected scores before dividing by it
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MAX_ELEMS = 65536 * 5120
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one generated token through the norm of a layer: latency
        {"name": "norm_one_token", "op": "norm", "dir": "fwd", "M": 1, "K": 5120, "dtype": "bf16", "residual": True},
        # a rank's whole dispatch payload (sequence 8192 x local batch 8)
        {"name": "norm_payload", "op": "norm", "dir": "fwd", "M": 65536, "K": 5120, "dtype": "bf16", "residual": True},
        # training step on the tokens of one expert-parallel rank
        {"name": "norm_backward", "op": "norm", "dir": "bwd", "M": 16640, "K": 5120, "dtype": "bf16", "residual": True},
        # a small decode batch over many experts in groups, with a balance bias
        {"name": "route_decode", "op": "route", "dir": "fwd", "M": 33, "E": 128, "dtype": "f32", "score": "sigmoid",
         "bias": True, "n_groups": 8, "topk_groups": 4, "topk": 8, "renorm": True, "top2": True, "scale": 2.5},
        # the same router over a rank's payload
        {"name": "route_payload", "op": "route", "dir": "fwd", "M": 65536, "E": 128, "dtype": "f32", "score": "sigmoid",
         "bias": True, "n_groups": 8, "topk_groups": 4, "topk": 8, "renorm": True, "top2": True, "scale": 2.5},
        # training: the gradient of softmax weights that are not renormalised reaches every logit
        {"name": "route_backward", "op": "route", "dir": "bwd", "M": 65536, "E": 64, "dtype": "bf16", "score": "softmax",
         "bias": False, "n_groups": 1, "topk_groups": 1, "topk": 6, "renorm": False, "top2": False, "scale": 1.0},
        # the tiny tensor of the tests
        {"name": "mxfp4_tiny", "op": "mxfp4", "M": 512, "K": 256, "rule": "floor"},
        # the payload in 4 bits, out and back
        {"name": "mxfp4_payload", "op": "mxfp4", "M": 65536, "K": 5120, "rule": "rceil"},
        # 8 tokens decoded at once, top-1 over 16 experts: the chosen experts' weights are the traffic
        {"name": "product_decode", "op": "product", "M": 8, "N": 8192, "K": 5120, "G": 16, "tokens": "mxfp8", "out": "bf16",
         "route": 1},
        # small ragged groups of a mid-sized layer, odd column count, an fp32 result
        {"name": "product_ragged", "op": "product", "M": 777, "N": 1736, "K": 1408, "G": 16, "tokens": "mxfp4", "out": "f32",
         "route": 2},
        # the tokens of a rank against 16 experts, as received (MXFP8) and in 4 bits
        {"name": "product_tokens_mxfp8", "op": "product", "M": 16640, "N": 8192, "K": 5120, "G": 16, "tokens": "mxfp8",
         "out": "bf16", "route": 1},
        {"name": "product_tokens_mxfp4", "op": "product", "M": 16640, "N": 8192, "K": 5120, "G": 16, "tokens": "mxfp4",
         "out": "bf16", "route": 1},
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer multiple of `step` in [lo, hi], uniform in its logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "route", "mxfp4", "product", "product"])
    if op == "norm":
        K = _log_int(rng, 64, 16384, 32)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "M": _log_int(rng, 1, min(65536, MAX_ELEMS // 2 // K)), "K": K,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.75}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, 8, 512 // groups)
        kept = groups if groups == 1 else rng.randint(1, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "M": _log_int(rng, 1, min(65536, 65536 * 128 // E)), "E": E,
                "dtype": rng.choice(["f32", "bf16"]), "score": score, "bias": score == "sigmoid" and rng.random() < 0.7,
                "n_groups": groups, "topk_groups": kept, "topk": rng.randint(1, min(10, kept * (E // groups))),
                "renorm": rng.random() < 0.6, "top2": groups > 1 and rng.random() < 0.5, "scale": rng.choice([1.0, 2.5])}
    if op == "mxfp4":
        K = _log_int(rng, 32, 16384, 32)
        return {"op": op, "M": _log_int(rng, 1, min(65536, MAX_ELEMS // K)), "K": K, "rule": rng.choice(["floor", "rceil"])}
    tokens = rng.choice(["mxfp8", "mxfp4"])
    return {"op": op, "M": _log_int(rng, 1, 16640), "N": _log_int(rng, 64, 8192, 8), "K": _log_int(rng, 256, 5120, 128),
            "G": _log_int(rng, 1, 16), "tokens": tokens, "out": rng.choice(["bf16", "f32"]) if tokens == "mxfp4" else "bf16",
            "route": rng.randint(1, 1 << 20)}


def _sizes(case):
    """Rows of each expert: every row drawn with probability proportional to (g + 1) ** -1.1."""
    r, G = random.Random(case["route"]), case["G"]
    sizes = [0] * G
    for g in r.choices(range(G), weights=[(g + 1) ** -1.1 for g in range(G)], k=case["M"]):
        sizes[g] += 1
    return sizes


# ------------------------------------------------------------------ inputs --
def _rows(M, K, g):
    """N(0, 1) times a factor of each row, lognormal(0, 1)."""
    return torch.randn((M, K), generator=g, device="cuda") * torch.exp(torch.randn((M, 1), generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "norm":
        dt, M, K = DTYPES[case["dtype"]], case["M"], case["K"]
        st["w"] = (1.0 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(dt)
        if case["dir"] == "fwd":
            st["x"] = torch.randn((M, K), generator=g, device="cuda").to(dt)
            st["r"] = _rows(M, K, g).to(dt) if case["residual"] else None
        else:
            st["h"] = _rows(M, K, g).to(dt)
            st["rstd"] = torch.rsqrt(st["h"].float().square().mean(-1) + EPS)
            st["dy"] = (1e-2 * torch.randn((M, K), generator=g, device="cuda")).to(dt)
            st["dh"] = (1e-2 * torch.randn((M, K), generator=g, device="cuda")).to(dt) if case["residual"] else None
    elif case["op"] == "route":
        M, E = case["M"], case["E"]
        lg = 2.0 * torch.randn((M, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        lg[torch.rand(M, generator=g, device="cuda") < 0.005] = -math.inf       # padding rows: nothing to select
        st["logits"] = lg.to(DTYPES[case["dtype"]])
        st["bias"] = 0.05 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        if case["dir"] == "bwd":
            st["ids"] = _route(st["logits"], st["bias"], case)[0]
            st["dw"] = torch.randn((M, case["topk"]), generator=g, device="cuda")
    elif case["op"] == "mxfp4":
        x = _rows(case["M"], case["K"], g)
        x[torch.rand(case["M"], generator=g, device="cuda") < 0.01] = 0.0
        st["x"] = x.to(torch.bfloat16)
    else:
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        sizes = _sizes(case)
        st["ends_host"] = [sum(sizes[:i + 1]) for i in range(G)]
        st["ends"] = torch.tensor(st["ends_host"], dtype=torch.int32, device="cuda")
        x = _rows(M, K, g).to(torch.bfloat16)
        if case["tokens"] == "mxfp8":
            st["xq"], st["xs"] = _mxfp8(x.float())
        else:
            st["xq"], st["xs"] = _mxfp4(x, "floor")
        w = [_mxfp4((0.02 * torch.randn((N, K), generator=g, device="cuda")).to(torch.bfloat16), "rceil") for _ in range(G)]
        st["wq"] = torch.stack([q for q, _ in w])
        st["ws"] = torch.stack([s for _, s in w])
    return st


# --------------------------------------------------------------- plain forms --
def _exponent(amax):
    """floor(log2 amax) of non-negative floats, -127 for zero (their bits' exponent field)."""
    return (amax.float().contiguous().view(torch.int32) >> 23) - 127


def _pow2(e):
    """2 ** e for int32 e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _mxfp8(y):
    """E4M3 codes and E8M0 scales of y's bf16 rounding, blocks of 32 along the rows."""
    b = y.to(torch.bfloat16).float().view(y.shape[0], -1, 32)
    e = (_exponent(b.abs().amax(-1)) - 8).clamp(min=-127)
    q = (b * _pow2(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(y.shape), (e + 127).to(torch.uint8)


def _mxfp4(x, rule):
    """E2M1 codes (two a byte, the even element low) and E8M0 scales of x."""
    b = x.float().view(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = _exponent(amax) - 2
    if rule == "rceil":
        e = e + (amax > 6.0 * _pow2(e.clamp(min=-127))).int()
    e = e.clamp(min=-127)
    a = b.abs() * _pow2(-e).unsqueeze(-1)
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
         + 8 * torch.signbit(b).to(torch.uint8)).view(x.shape)
    return c[:, 0::2] | (c[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _decode4(q, s):
    """fp32 values of packed E2M1 codes (rows, K/2) with scales (rows, K/32)."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    v = t[torch.stack((q & 15, q >> 4), -1).int()].view(q.shape[0], -1, 32)
    return (v * _pow2(s.int() - 127).unsqueeze(-1)).view(q.shape[0], -1)


def _decode8(q, s):
    v = q.view(torch.float8_e4m3fn).float().view(q.shape[0], -1, 32)
    return (v * _pow2(s.int() - 127).unsqueeze(-1)).view(q.shape[0], -1)


def _norm_fwd(x, r, w):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1) + EPS)
    y = (hf * rstd.unsqueeze(-1) * w.float()).to(x.dtype)
    q, s = _mxfp8(y)
    return h, y, q, s, rstd


def _norm_bwd(h, w, rstd, dy, dh):
    hf, g, rs = h.float(), dy.float(), rstd.unsqueeze(-1)
    gw = g * w.float()
    dx = rs * (gw - hf * ((gw * hf).mean(-1, keepdim=True) * rs * rs))
    if dh is not None:
        dx = dx + dh.float()
    return dx.to(h.dtype), (g * hf * rs).sum(0)


def _scores(l, score):
    """Scores of logits l, and values in the same order that need no sum over the row; 0 where l is masked."""
    ok = l > -math.inf
    if score == "sigmoid":
        s = torch.where(ok, 1.0 / (1.0 + torch.exp(-l)), torch.zeros_like(l))
        return s, s
    m = l.amax(-1, keepdim=True)
    e = torch.where(ok, torch.exp(l - torch.where(m > -math.inf, m, torch.zeros_like(m))), torch.zeros_like(l))
    return e / e.sum(-1, keepdim=True).clamp(min=TINY), e


def _select(l, s, v, bias, c):
    """ids (rows, topk) of the selected experts, -1 past the last: stable sorts, so ties go to the lowest index."""
    ok = l > -math.inf
    key, val = (l, v) if bias is None else (s + bias, s + bias)
    if c["n_groups"] > 1:
        gv = torch.where(ok, val, torch.full_like(val, -math.inf)).view(l.shape[0], c["n_groups"], -1)
        top = torch.sort(gv, dim=-1, descending=True).values
        gval = top[..., 0]
        if c["top2"] and top.shape[-1] > 1:
            gval = torch.where(top[..., 1] > -math.inf, top[..., 0] + top[..., 1], top[..., 0])
        order = torch.sort(gval, dim=-1, descending=True, stable=True).indices
        kept = torch.zeros_like(gval, dtype=torch.bool).scatter_(1, order[:, :c["topk_groups"]], True)
        ok = ok & kept.repeat_interleave(l.shape[1] // c["n_groups"], 1)
    key = torch.where(ok, key, torch.full_like(key, -math.inf))
    top, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    top, ids = top[:, :c["topk"]], ids[:, :c["topk"]]
    return torch.where(top > -math.inf, ids, torch.full_like(ids, -1))


def _weights(s, ids, c):
    sel = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), torch.zeros_like(s[:, :1]))
    if c["renorm"]:
        sel = sel / (sel.sum(-1, keepdim=True) + TINY)
    return sel * c["scale"]


def _route(logits, bias, c):
    l = logits.float()
    s, v = _scores(l, c["score"])
    ids = _select(l, s, v, bias, c)
    return ids.to(torch.int32), _weights(s, ids, c)


def _route_bwd(logits, ids, dw, c, wide=torch.float32):
    l = logits.to(wide)
    s, _ = _scores(l, c["score"])
    at = ids.long()
    some = at >= 0
    sel = torch.where(some, s.gather(1, at.clamp(min=0)), torch.zeros_like(s[:, :1]))
    g = torch.where(some, dw.to(wide), torch.zeros_like(sel)) * c["scale"]
    if c["renorm"]:
        d = sel.sum(-1, keepdim=True) + TINY
        g = torch.where(some, (g - (g * sel).sum(-1, keepdim=True) / d) / d, torch.zeros_like(g))
    ds = torch.zeros_like(s).scatter_add_(1, at.clamp(min=0), g)
    if c["score"] == "sigmoid":
        return s * (1.0 - s) * ds
    return s * (ds - (g * sel).sum(-1, keepdim=True))


def _product(st, c):
    """Each expert's rows times its decoded weight; the experts that have rows only."""
    decode = _decode8 if c["tokens"] == "mxfp8" else _decode4
    x = decode(st["xq"], st["xs"])
    ends = st["ends_host"]
    spans = [(g, a, b) for g, (a, b) in enumerate(zip([0] + ends[:-1], ends)) if b > a]
    return torch.cat([x[a:b] @ _decode4(st["wq"][g], st["ws"][g]).t() for g, a, b in spans]).to(DTYPES[c["out"]])


# -------------------------------------------------------------------- a pass --
def _codes8(q, s):
    """E4M3 and E8M0 bytes as the values they stand for."""
    return {"q": q.view(torch.float8_e4m3fn), "s": s.view(torch.float8_e8m0fnu)}


def run(st):
    c = st["case"]
    if own:
        from float8_quantization_moe_amd import mxq
    if c["op"] == "norm" and c["dir"] == "fwd":
        if own:
            h, y, q, s, rstd = mxq.add_rmsnorm(st["x"], st["r"], st["w"], EPS)
        else:
            h, y, q, s, rstd = _norm_fwd(st["x"], st["r"], st["w"])
        return {"h": h, "y": y, "rstd": rstd, **_codes8(q, s)}
    if c["op"] == "norm":
        if own:
            dx, dw = mxq.add_rmsnorm_bwd(st["h"], st["w"], st["rstd"], st["dy"], st["dh"])
        else:
            dx, dw = _norm_bwd(st["h"], st["w"], st["rstd"], st["dy"], st["dh"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "route" and c["dir"] == "fwd":
        if own:
            ids, w = mxq.route_topk(st["logits"], c["topk"], bias=st["bias"], score=c["score"], n_groups=c["n_groups"],
                                    topk_groups=c["topk_groups"], renormalize=c["renorm"], group_top2=c["top2"],
                                    scale=c["scale"])
        else:
            ids, w = _route(st["logits"], st["bias"], c)
        return {"ids": ids, "weights": w}
    if c["op"] == "route":
        if own:
            d = mxq.route_topk_bwd(st["logits"], st["ids"], st["dw"], score=c["score"], renormalize=c["renorm"],
                                   scale=c["scale"])
        else:
            d = _route_bwd(st["logits"], st["ids"], st["dw"], c).to(st["logits"].dtype)
        return {"dlogits": d}
    if c["op"] == "mxfp4":
        if own:
            q, s = mxq.quantize_mxfp4(st["x"], mxq.MXQ_SCALE_RCEIL if c["rule"] == "rceil" else mxq.MXQ_SCALE_FLOOR)
            y = mxq.dequantize_mxfp4(q, s)
        else:
            q, s = _mxfp4(st["x"], c["rule"])
            y = _decode4(q, s).to(torch.bfloat16)
        return {"y": y, "s": s.view(torch.float8_e8m0fnu)}
    if own:
        return {"y": mxq.mxfp4_grouped_mm(st["xq"], st["xs"], st["wq"], st["ws"], st["ends"],
                                          x_format=mxq.MXQ_FMT_E4M3 if c["tokens"] == "mxfp8" else mxq.MXQ_FMT_E2M1,
                                          out_dtype=DTYPES[c["out"]])}
    return {"y": _product(st, c)}


def work(case):
    """Each input read once, each output written once; the arithmetic of the formulas."""
    op, M = case["op"], case["M"]
    if op == "norm":
        n, z = M * case["K"], 2 if case["dtype"] == "bf16" else 4
        if case["dir"] == "fwd":       # x (and r) in; y (and h) and 33/32 bytes of codes out
            return {"bytes": n * (z * (4 if case["residual"] else 2) + 33 / 32) + 4 * M + z * case["K"], "flops": 6 * n}
        return {"bytes": n * z * (4 if case["residual"] else 3) + 4 * M + (z + 4) * case["K"], "flops": 12 * n}
    if op == "route":
        n, z = M * case["E"], 2 if case["dtype"] == "bf16" else 4
        if case["dir"] == "fwd":
            return {"bytes": n * z + 8 * M * case["topk"], "flops": 8 * n}
        reads = n if case["score"] == "softmax" and not case["renorm"] else min(n, M * case["topk"])
        return {"bytes": z * (reads + n) + 8 * M * case["topk"], "flops": 8 * n}
    if op == "mxfp4":
        return {"bytes": M * case["K"] * 2 * (2 + 17 / 32), "flops": 4 * M * case["K"]}
    N, K = case["N"], case["K"]
    experts = sum(1 for s in _sizes(case) if s)
    x = M * K * (33 / 32 if case["tokens"] == "mxfp8" else 17 / 32)
    return {"bytes": x + experts * N * K * 17 / 32 + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# ---------------------------------------------------------- the definitions in 64 bits --
def _exact_scale(amax, top, up):
    """Power-of-two scale of a block maximum: its exponent less `top`, or rounded up so that nothing passes the format's largest."""
    m, e = torch.frexp(amax)                                     # amax = m 2^e, m in [1/2, 1)
    e = (e - 1 - top).double()
    if up:
        e = e + (m > up / 2.0 ** (top + 1)).double()
    return torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -127.0)).clamp(min=-127.0))


def _exact_grid(a, lowest, digits, most):
    """Non-negative a on the grid of a float with `digits` bits after the point and least exponent `lowest`, ties to even."""
    _, e = torch.frexp(a)
    step = torch.exp2((e - 1).clamp(min=lowest).double() - digits)
    return (torch.round(a / step) * step).clamp(max=most)


def _exact_codes8(y):
    b = y.float().to(torch.bfloat16).double().view(y.shape[0], -1, 32)
    s = _exact_scale(b.abs().amax(-1), 8, None)
    v = b / s.unsqueeze(-1)
    return (torch.sign(v) * _exact_grid(v.abs(), -6, 3, 448.0)).view(y.shape), s


def _exact_values4(q, s):
    n = torch.stack((q % 16, q // 16), -1).long().view(q.shape[0], -1)
    e, m = (n % 8) // 2, (n % 2).double()                        # E2M1: bias 1, one digit, e = 0 subnormal
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e.double() - 1), m / 2)
    return torch.where(n >= 8, -v, v) * torch.exp2(s.double() - 127).repeat_interleave(32, 1)


def _exact_values8(q, s):
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    c, op = case, case["op"]
    if op == "norm" and c["dir"] == "fwd":
        h = st["x"].double() if st["r"] is None else (st["x"].double() + st["r"].double()).to(st["x"].dtype).double()
        rstd = (h.pow(2).sum(-1) / c["K"] + EPS) ** -0.5
        y = h * rstd[:, None] * st["w"].double()
        q, s = _exact_codes8(y)
        return {"h": h, "y": y, "rstd": rstd, "q": q, "s": s}
    if op == "norm":
        h, g, r = st["h"].double(), st["dy"].double(), st["rstd"].double()[:, None]
        n = h * r
        gw = g * st["w"].double()
        dx = r * (gw - n * ((gw * n).sum(-1, keepdim=True) / c["K"]))
        return {"dx": dx if st["dh"] is None else dx + st["dh"].double(), "dw": (g * n).sum(0)}
    if op == "route":
        l = st["logits"].double()
        if c["dir"] == "bwd":
            return {"dlogits": _exact_route_grad(l, st["ids"], st["dw"].double(), c)}
        s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, -1))
        ids = _route(st["logits"], st["bias"], c)[0].long()      # the selection is whole numbers: those of 32 bits
        z = torch.cat((s, torch.zeros_like(s[:, :1])), 1).gather(1, torch.where(ids < 0, torch.full_like(ids, c["E"]), ids))
        return {"ids": None, "weights": c["scale"] * (z / (z.sum(-1, keepdim=True) + TINY) if c["renorm"] else z)}
    if op == "mxfp4":
        b = st["x"].double().view(c["M"], -1, 32)
        s = _exact_scale(b.abs().amax(-1), 2, 6.0 if c["rule"] == "rceil" else None)
        v = b / s.unsqueeze(-1)
        return {"y": (torch.sign(v) * _exact_grid(v.abs(), 0, 1, 6.0) * s.unsqueeze(-1)).view(c["M"], c["K"]), "s": s}
    x = (_exact_values8 if c["tokens"] == "mxfp8" else _exact_values4)(st["xq"], st["xs"])
    y = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    a = 0
    for g, b in enumerate(st["ends_host"]):
        if b > a:
            y[a:b] = x[a:b] @ _exact_values4(st["wq"][g], st["ws"][g]).t().contiguous()
        a = b
    return {"y": y}


def _exact_route_grad(l, ids, dw, c):
    """Through the Jacobians of the scores and of the division by their selected sum."""
    hot = torch.zeros(ids.shape + (l.shape[1] + 1,), dtype=torch.bool, device=l.device)
    hot = hot.scatter_(2, torch.where(ids < 0, torch.full_like(ids, l.shape[1]), ids).long().unsqueeze(-1), True)[..., :-1]
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, -1))
    any_, up = hot.any(1), torch.zeros_like(l)
    for j in range(ids.shape[1]):
        up = up + hot[:, j] * dw[:, j:j + 1] * c["scale"]
    if c["renorm"]:
        total = (s * any_).sum(-1, keepdim=True) + TINY
        up = any_ * (up / total - (up * s).sum(-1, keepdim=True) / total ** 2)
    return up * s * (1 - s) if c["score"] == "sigmoid" else s * (up - (up * s).sum(-1, keepdim=True))
