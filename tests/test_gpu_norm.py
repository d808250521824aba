"""Residual addition + root-mean-square norm with MXFP8 codes, and its gradients,
against the 64-bit definitions.

Bounds, with u = 2^-24.  A row's sum of squares is a chain of at most 64 fp32 adds in
a lane and 10 across lanes and waves, so the sum is good to 74 u, rstd to half of it
and its own two roundings, and a product of three factors to 2 u more: below 2^-18
relative for an fp32 output, and half a step of bf16 more for a bf16 output.  dx
subtracts two terms, so its bound is relative to the terms' sizes; a dot product of
K terms in the same tree is good to 80 u of the sum of magnitudes.  dweight adds a
few rows in a register, the waves of a workgroup, then up to 1024 parts in 32 slices
and the slices: with M <= 2000 no more than (8 + 64 + 3) u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import gpu_util as U
import oracle
import plain64 as P
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu


def guarded(n, dtype):
    return U.Guarded(n, dtype, (n,))


EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SUM = 2.0 ** -17


def f64(t):
    return t.double().cpu().numpy()


def inputs(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    r = torch.randn((M, K), generator=g) * torch.exp(torch.randn((M, 1), generator=g))
    w = 1 + 0.2 * torch.randn(K, generator=g)
    return [t.to(DT[dtype]).cuda() for t in (x, r, w)]


SHAPES = [(1, 32), (3, 64), (5, 512), (4, 544), (7, 1024), (9, 1056), (2, 2048), (3, 2080), (33, 4096), (2, 4128),
          (1, 5120), (300, 5120), (3, 6144), (3, 6176), (5, 8192), (2, 8224), (3, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False], ids=["add", "plain"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, dtype, residual):
    x, r, w = inputs(M, K, dtype, M * 7 + K)
    dt = DT[dtype]
    h, y = guarded(M * K * x.element_size(), torch.uint8), guarded(M * K * x.element_size(), torch.uint8)
    q, s, rstd = guarded(M * K, torch.uint8), guarded(M * K // 32, torch.uint8), guarded(M, torch.float32)
    mxq.mxq_add_rmsnorm(x, r if residual else None, w, EPS, h.t.view(dt), y.t.view(dt), q.t, s.t, rstd.t)
    torch.cuda.synchronize()
    for gd in (h, y, q, s, rstd):
        assert gd.guard_intact()
    hv = h.t.view(dt).view(M, K)
    want_h = (x.double() + r.double()).to(dt) if residual else x
    assert torch.equal(hv.float(), want_h.float())
    want, want_rstd = P.norm_fwd(f64(hv), f64(w), EPS)
    yv = y.t.view(dt).view(M, K)
    assert np.all(np.abs(f64(yv) - want) <= P.half_step(want, dtype) + SUM * np.abs(want))
    assert np.all(np.abs(f64(rstd.t) - want_rstd) <= SUM * want_rstd)
    oq, os_ = oracle.mx_quantize(U.host_u16(yv.to(torch.bfloat16)))
    assert np.array_equal(U.host_u8(q.t).reshape(M, K), oq)
    assert np.array_equal(U.host_u8(s.t).reshape(M, K // 32), os_)


@pytest.mark.parametrize("K", [8, 40, 72, 520, 5128])
def test_forward_without_codes_any_multiple_of_8(K):
    M = 5
    x, r, w = inputs(M, K, "bf16", K)
    y = guarded(M * K * 2, torch.uint8)
    mxq.mxq_add_rmsnorm(x, r, w, EPS, None, y.t.view(torch.bfloat16))
    torch.cuda.synchronize()
    assert y.guard_intact()
    want, _ = P.norm_fwd(f64((x.double() + r.double()).to(torch.bfloat16)), f64(w), EPS)
    got = f64(y.t.view(torch.bfloat16).view(M, K))
    assert np.all(np.abs(got - want) <= P.half_step(want, "bf16") + SUM * np.abs(want))


def test_codes_only_and_in_place():
    M, K = 37, 1024
    x, r, w = inputs(M, K, "bf16", 3)
    h, y, q, s, rstd = mxq.add_rmsnorm(x, r, w, EPS)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    mxq.mxq_add_rmsnorm(x, r, w, EPS, q=q2, s=s2)                      # codes alone
    assert torch.equal(q, q2) and torch.equal(s, s2)
    x2, r2 = x.clone(), r.clone()
    mxq.mxq_add_rmsnorm(x2, r2, w, EPS, h=r2, y=x2, q=q2, s=s2)        # the stream and the row updated in place
    assert torch.equal(r2, h) and torch.equal(x2, y) and torch.equal(q, q2) and torch.equal(s, s2)


def test_rows_of_zeros_infinities_and_nan():
    M, K = 6, 256
    x, _, w = inputs(M, K, "bf16", 4)
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 1e-30                                                       # far below eps
    x[4] = 3e38                                                        # squares pass fp32: zeros, as documented
    h, y, q, s, rstd = mxq.add_rmsnorm(x, None, w, EPS)
    torch.cuda.synchronize()
    assert torch.all(y[0] == 0) and torch.all(q[0] & 0x7F == 0) and torch.all(s[0] == 0)
    assert torch.all(torch.isnan(y[1])) and torch.all(s[1] == 255) and torch.all(q[1] == 0x7F)
    assert torch.isnan(y[2, 9]) and s[2, 0] == 255
    assert torch.all(y[4] == 0) and rstd[4] == 0
    want, _ = P.norm_fwd(f64(x[3:]), f64(w), EPS)
    for row in (3, 5):
        assert np.all(np.abs(f64(y[row]) - want[row - 3]) <= P.half_step(want[row - 3], "bf16") + SUM * np.abs(want[row - 3]))
    # eps = 0 on a row of zeros is 0 * inf, as the formula has it
    assert torch.all(torch.isnan(mxq.add_rmsnorm(x[:1].contiguous(), None, w, 0.0)[1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False], ids=["dh", "nodh"])
@pytest.mark.parametrize("M,K", SHAPES + [(1025, 256), (2000, 1024), (1500, 2080), (7, 8), (5, 520)])
def test_backward(M, K, dtype, with_dh):
    g = torch.Generator().manual_seed(M + 3 * K)
    h = (torch.randn((M, K), generator=g) * torch.exp(torch.randn((M, 1), generator=g))).to(DT[dtype]).cuda()
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(DT[dtype]).cuda()
    dy = torch.randn((M, K), generator=g).to(DT[dtype]).cuda()
    dh = torch.randn((M, K), generator=g).to(DT[dtype]).cuda() if with_dh else None
    rstd = (1 / torch.sqrt(h.double().square().mean(-1) + EPS)).float()
    dx, dw = guarded(M * K * h.element_size(), torch.uint8), guarded(K, torch.float32)
    ws = guarded(mxq.mxq_add_rmsnorm_bwd_workspace_bytes(M, K), torch.uint8)
    mxq.mxq_add_rmsnorm_bwd(h, w, rstd, dy, dh, dx.t.view(DT[dtype]), dw.t, ws.t)
    torch.cuda.synchronize()
    assert dx.guard_intact() and dw.guard_intact() and ws.guard_intact()
    H, W, G, R = f64(h), f64(w), f64(dy), f64(rstd)
    want, want_dw = P.norm_bwd(H, W, R, G, None if dh is None else f64(dh))
    n = np.abs(H) * R[:, None]
    a = np.abs(G * W)
    size = R[:, None] * (a + n * (a * n).mean(-1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    got = f64(dx.t.view(DT[dtype]).view(M, K))
    assert np.all(np.abs(got - want) <= P.half_step(want, dtype) + SUM * size)
    assert np.all(np.abs(f64(dw.t) - want_dw) <= 75 * 2.0 ** -24 * (np.abs(G) * n).sum(0))
    # the same inputs give the same bits, and dx may overwrite dy
    dx2, dw2 = mxq.add_rmsnorm_bwd(h, w, rstd, dy, dh)
    assert torch.equal(dx2, dx.t.view(DT[dtype]).view(M, K)) and torch.equal(dw2, dw.t)
    mxq.mxq_add_rmsnorm_bwd(h, w, rstd, dy, dh, dy, dw2, ws.t)
    assert torch.equal(dx2, dy)


def test_backward_against_differences():
    """dx and dweight of sum(y * dy) + sum(h * dh), against central differences of the 64-bit forward.
    The difference quotient with step 1e-4 is good to about 1e-7 of the terms' sizes, fp32 to 2^-17."""
    M, K = 6, 160
    x, r, w = inputs(M, K, "f32", 9)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn((M, K), generator=g).cuda()
    dh = torch.randn((M, K), generator=g).cuda()
    h, y, q, s, rstd = mxq.add_rmsnorm(x, r, w, EPS)
    dx, dw = mxq.add_rmsnorm_bwd(h, w, rstd, dy, dh)
    H, W, G, D = f64(h), f64(w), f64(dy), f64(dh)

    def loss(h_, w_):
        return (P.norm_fwd(h_, w_, EPS)[0] * G).sum() + (h_ * D).sum()

    rng = np.random.default_rng(1)
    for _ in range(8):
        v, u, t = rng.standard_normal((M, K)), rng.standard_normal(K), 1e-4
        num = (loss(H + t * v, W + t * u) - loss(H - t * v, W - t * u)) / (2 * t)
        ana = (f64(dx) * v).sum() + (f64(dw) * u).sum()
        size = np.abs(f64(dx) * v).sum() + np.abs(f64(dw) * u).sum()
        assert abs(num - ana) <= 1e-5 * size


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    h, y, q, s, rstd = mxq.add_rmsnorm(x, None, w, EPS)
    dw = torch.full((64,), 3.0, device="cuda")
    mxq.mxq_add_rmsnorm_bwd(x, w, rstd, x, None, x, dw, torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert torch.all(dw == 0)


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_backward_keeps_its_workspace_while_another_stream_runs(as_handle):
    M, K = 512, 1024
    torch.manual_seed(3)
    h, dy = (torch.randn(M, K, device="cuda").to(torch.bfloat16) for _ in range(2))
    w, rstd = torch.ones(K, dtype=torch.bfloat16, device="cuda"), torch.rand(M, device="cuda") + 0.5
    dx, dw = mxq.add_rmsnorm_bwd(h, w, rstd, dy)
    size = mxq.mxq_add_rmsnorm_bwd_workspace_bytes(M, K)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)                       # a bounded spin: the call's kernels come after it
    dx2, dw2 = mxq.add_rmsnorm_bwd(h, w, rstd, dy, stream=st.cuda_stream if as_handle else st)
    held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and len(held) == 4


def test_other_stream():
    x, r, w = inputs(257, 5120, "bf16", 8)
    want = mxq.add_rmsnorm(x, r, w, EPS)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = mxq.add_rmsnorm(x, r, w, EPS)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_past_two_to_the_31_elements():
    M, K = 131200, 16384                                               # 2.15e9 values
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for a in range(0, M, 16400):
        x[a:a + 16400] = torch.randn((16400, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    h, y, q, s, rstd = mxq.add_rmsnorm(x, None, w, EPS)
    rows = [0, 1, 65599, 131071, 131072, M - 1]
    want, _ = P.norm_fwd(f64(x[rows]), f64(w), EPS)
    assert np.all(np.abs(f64(y[rows]) - want) <= P.half_step(want, "bf16") + SUM * np.abs(want))
    oq, os_ = oracle.mx_quantize(U.host_u16(y[rows]))
    assert np.array_equal(U.host_u8(q[rows]), oq) and np.array_equal(U.host_u8(s[rows]), os_)
    dx, _ = mxq.add_rmsnorm_bwd(x, w, rstd, y)
    want, _ = P.norm_bwd(f64(x[rows]), f64(w), f64(rstd[rows]), f64(y[rows]), None)
    size = 2 * np.abs(f64(rstd[rows]))[:, None] * np.abs(f64(y[rows]))
    assert np.all(np.abs(f64(dx[rows]) - want) <= P.half_step(want, "bf16") + SUM * (size + 1))
