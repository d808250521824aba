"""Residual addition + layer norm with MXFP8 codes, and its gradients, against the 64-bit
definitions.

Bounds, with u = 2^-24.  A sum over a row is a chain of at most 32 fp32 adds in a lane and 14
across lanes and waves: 46 u of the sum of its magnitudes.  The mean's error is repaired by the
mean of the differences from it, d, which is good to 46 u of mean |d| and a rounding or two of
each d; the variance is good to 50 u, rstd to half of that and one rounding.  y is a product of
three factors and a sum: below 2^-18 of (|d| + mean |d|) rstd |w| + |b|, where 2^-17 is allowed.
dx adds three terms, each good to 60 u of its size.  dweight and dbias add at most 16 rows in a
register, 3 waves, then up to 512 parts in 32 slices of 16 and the slices: below 80 u of the sum
of magnitudes with M <= 2000."""
import numpy as np
import pytest
import torch

import gpu_util as U
import oracle
import plain64 as P
import plain64_training as T
from float8_quantization_moe_amd import mxq, training

pytestmark = pytest.mark.gpu

EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SUM = 2.0 ** -17
ROUND = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def guarded(n, dtype):
    return U.Guarded(n, dtype, (n,))


def inputs(M, K, dtype, seed, shift=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    r = torch.randn((M, K), generator=g) * torch.exp(torch.randn((M, 1), generator=g)) + shift * torch.randn((M, 1), generator=g)
    w = 1 + 0.2 * torch.randn(K, generator=g)
    b = 0.3 * torch.randn(K, generator=g)
    return [t.to(DT[dtype]).cuda() for t in (x, r, w, b)]


def check_forward(hv, w, b, y, mean, rstd, dtype):
    H, W, B = f64(hv), f64(w), None if b is None else f64(b)
    want, wm, wr = T.layernorm_fwd(H, W, B, EPS)
    d = np.abs(H - wm[:, None])
    size = (d + d.mean(-1, keepdims=True)) * wr[:, None] * np.abs(W) + (0 if b is None else np.abs(B))
    if y is not None:
        assert np.all(np.abs(f64(y) - want) <= P.half_step(want, dtype) + SUM * size)
    assert np.all(np.abs(f64(mean) - wm) <= 2 * ROUND * np.abs(wm) + SUM * d.mean(-1))
    assert np.all(np.abs(f64(rstd) - wr) <= SUM * wr)


SHAPES = [(1, 32), (3, 64), (5, 512), (4, 544), (7, 1024), (9, 1056), (2, 2048), (3, 2080), (33, 4096), (2, 4128),
          (1, 5120), (300, 5120), (3, 6144), (3, 6176), (5, 8192), (2, 8224), (3, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False], ids=["add", "plain"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, dtype, residual):
    x, r, w, b = inputs(M, K, dtype, M * 7 + K)
    dt, z = DT[dtype], x.element_size()
    h, y = guarded(M * K * z, torch.uint8), guarded(M * K * z, torch.uint8)
    q, s = guarded(M * K, torch.uint8), guarded(M * K // 32, torch.uint8)
    mean, rstd = guarded(M, torch.float32), guarded(M, torch.float32)
    mxq.mxq_add_layernorm(x, r if residual else None, w, b, EPS, h.t.view(dt), y.t.view(dt), q.t, s.t, mean.t, rstd.t)
    torch.cuda.synchronize()
    for gd in (h, y, q, s, mean, rstd):
        assert gd.guard_intact()
    hv, yv = h.t.view(dt).view(M, K), y.t.view(dt).view(M, K)
    want_h = (x.double() + r.double()).to(dt) if residual else x
    assert torch.equal(hv.float(), want_h.float())
    check_forward(hv, w, b, yv, mean.t, rstd.t, dtype)
    oq, os_ = oracle.mx_quantize(U.host_u16(yv.to(torch.bfloat16)))
    assert np.array_equal(U.host_u8(q.t).reshape(M, K), oq)
    assert np.array_equal(U.host_u8(s.t).reshape(M, K // 32), os_)


@pytest.mark.parametrize("K", [8, 40, 72, 520, 5128])
def test_forward_without_codes_or_bias_any_multiple_of_8(K):
    M = 5
    x, r, w, _ = inputs(M, K, "bf16", K)
    y, mean, rstd = guarded(M * K * 2, torch.uint8), guarded(M, torch.float32), guarded(M, torch.float32)
    mxq.mxq_add_layernorm(x, r, w, None, EPS, None, y.t.view(torch.bfloat16), mean=mean.t, rstd=rstd.t)
    torch.cuda.synchronize()
    assert y.guard_intact() and mean.guard_intact() and rstd.guard_intact()
    check_forward((x.double() + r.double()).to(torch.bfloat16), w, None, y.t.view(torch.bfloat16).view(M, K), mean.t, rstd.t, "bf16")


@pytest.mark.parametrize("shift", [1e3, 1e5])
@pytest.mark.parametrize("K", [64, 2048, 5120])
def test_a_mean_far_larger_than_the_spread(K, shift):
    x, _, w, b = inputs(6, K, "f32", K)
    x = x + shift
    h, y, q, s, mean, rstd = training.add_layernorm(x, None, w, b, EPS)
    check_forward(x, w, b, y, mean, rstd, "f32")


def test_codes_only_and_in_place():
    M, K = 37, 1024
    x, r, w, b = inputs(M, K, "bf16", 3)
    h, y, q, s, mean, rstd = training.add_layernorm(x, r, w, b, EPS)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    mxq.mxq_add_layernorm(x, r, w, b, EPS, q=q2, s=s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    x2, r2 = x.clone(), r.clone()
    mxq.mxq_add_layernorm(x2, r2, w, b, EPS, h=r2, y=x2, q=q2, s=s2)   # the stream and the row updated in place
    assert torch.equal(r2, h) and torch.equal(x2, y) and torch.equal(q, q2) and torch.equal(s, s2)


def test_rows_of_zeros_infinities_and_nan():
    M, K = 7, 256
    x, _, w, b = inputs(M, K, "bf16", 4)
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 1e-30                                                       # equal values far below eps
    x[4] = 3e38                                                        # the sum passes fp32
    x[5] = 7.25                                                        # equal values: only the bias is left
    h, y, q, s, mean, rstd = training.add_layernorm(x, None, w, b, EPS)
    torch.cuda.synchronize()
    for row in (1, 2, 4):
        assert torch.all(torch.isnan(y[row])) and torch.all(s[row] == 255) and torch.all(q[row] == 0x7F)
    for row in (0, 5):
        assert torch.equal(y[row], b)
    rows = [0, 3, 5, 6]
    check_forward(x[rows], w, b, y[rows], mean[rows], rstd[rows], "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False], ids=["dh", "nodh"])
@pytest.mark.parametrize("M,K", SHAPES + [(1025, 256), (2000, 1024), (1500, 2080), (17, 512), (7, 8), (5, 520)])
def test_backward(M, K, dtype, with_dh):
    g = torch.Generator().manual_seed(M + 3 * K)
    dt = DT[dtype]
    h = (torch.randn((M, K), generator=g) * torch.exp(torch.randn((M, 1), generator=g)) + torch.randn((M, 1), generator=g)).to(dt).cuda()
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(dt).cuda()
    dy = torch.randn((M, K), generator=g).to(dt).cuda()
    dh = torch.randn((M, K), generator=g).to(dt).cuda() if with_dh else None
    mean = h.double().mean(-1).float()
    rstd = (1 / torch.sqrt((h.double() - h.double().mean(-1, keepdim=True)).square().mean(-1) + EPS)).float()
    dx, dw, db = guarded(M * K * h.element_size(), torch.uint8), guarded(K, torch.float32), guarded(K, torch.float32)
    ws = guarded(mxq.mxq_add_layernorm_bwd_workspace_bytes(M, K), torch.uint8)
    mxq.mxq_add_layernorm_bwd(h, w, mean, rstd, dy, dh, dx.t.view(dt), dw.t, db.t, ws.t)
    torch.cuda.synchronize()
    for gd in (dx, dw, db, ws):
        assert gd.guard_intact()
    H, W, MU, R, G = f64(h), f64(w), f64(mean), f64(rstd), f64(dy)
    want, want_dw, want_db = T.layernorm_bwd(H, W, MU, R, G, None if dh is None else f64(dh))
    n = np.abs(H - MU[:, None]) * R[:, None]
    a = np.abs(G * W)
    size = R[:, None] * (a + a.mean(-1, keepdims=True) + n * (a * n).mean(-1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    got = f64(dx.t.view(dt).view(M, K))
    assert np.all(np.abs(got - want) <= P.half_step(want, dtype) + SUM * size)
    assert np.all(np.abs(f64(dw.t) - want_dw) <= 80 * ROUND * (np.abs(G) * n).sum(0))
    assert np.all(np.abs(f64(db.t) - want_db) <= 80 * ROUND * np.abs(G).sum(0))
    # the same inputs give the same bits; without dbias the rest is the same; dx may overwrite dy
    dx2, dw2, db2 = training.add_layernorm_bwd(h, w, mean, rstd, dy, dh)
    assert torch.equal(dx2, dx.t.view(dt).view(M, K)) and torch.equal(dw2, dw.t) and torch.equal(db2, db.t)
    dw2.fill_(float("nan"))
    mxq.mxq_add_layernorm_bwd(h, w, mean, rstd, dy, dh, dy, dw2, None, ws.t)
    assert torch.equal(dx2, dy) and torch.equal(dw2, dw.t)


def test_backward_against_differences():
    """dx, dweight and dbias of sum(y * dy) + sum(h * dh), against central differences of the 64-bit forward.
    The difference quotient with step 1e-4 is good to about 1e-7 of the terms' sizes, fp32 to 2^-17."""
    M, K = 6, 160
    x, r, w, b = inputs(M, K, "f32", 9)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn((M, K), generator=g).cuda()
    dh = torch.randn((M, K), generator=g).cuda()
    h, y, q, s, mean, rstd = training.add_layernorm(x, r, w, b, EPS)
    dx, dw, db = training.add_layernorm_bwd(h, w, mean, rstd, dy, dh)
    H, W, B, G, D = f64(h), f64(w), f64(b), f64(dy), f64(dh)

    def loss(h_, w_, b_):
        return (T.layernorm_fwd(h_, w_, b_, EPS)[0] * G).sum() + (h_ * D).sum()

    rng = np.random.default_rng(1)
    for _ in range(8):
        v, u, c, t = rng.standard_normal((M, K)), rng.standard_normal(K), rng.standard_normal(K), 1e-4
        num = (loss(H + t * v, W + t * u, B + t * c) - loss(H - t * v, W - t * u, B - t * c)) / (2 * t)
        parts = (f64(dx) * v, f64(dw) * u, f64(db) * c)
        assert abs(num - sum(p.sum() for p in parts)) <= 1e-5 * sum(np.abs(p).sum() for p in parts)


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    h, y, q, s, mean, rstd = training.add_layernorm(x, None, w, w, EPS)
    dx, dw, db = training.add_layernorm_bwd(x, w, mean, rstd, x)
    assert torch.all(dw == 0) and torch.all(db == 0) and dx.shape == (0, 64)


def test_past_two_to_the_31_elements():
    M, K = 131200, 16384                                               # 2.15e9 values
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for a in range(0, M, 16400):
        x[a:a + 16400] = (torch.randn((16400, K), generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    b = torch.full((K,), 0.25, dtype=torch.bfloat16, device="cuda")
    h, y, q, s, mean, rstd = training.add_layernorm(x, None, w, b, EPS)
    rows = [0, 1, 65599, 131071, 131072, M - 1]
    check_forward(x[rows], w, b, y[rows], mean[rows], rstd[rows], "bf16")
    oq, os_ = oracle.mx_quantize(U.host_u16(y[rows]))
    assert np.array_equal(U.host_u8(q[rows]), oq) and np.array_equal(U.host_u8(s[rows]), os_)
    dx, dw, db = training.add_layernorm_bwd(x, w, mean, rstd, y)
    want, _, _ = T.layernorm_bwd(f64(x[rows]), f64(w), f64(mean[rows]), f64(rstd[rows]), f64(y[rows]), None)
    size = np.abs(f64(rstd[rows]))[:, None] * (2 * np.abs(f64(y[rows])) + 2)
    assert np.all(np.abs(f64(dx[rows]) - want) <= P.half_step(want, "bf16") + SUM * (size + 1))
