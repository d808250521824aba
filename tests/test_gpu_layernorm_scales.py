"""Gradients of the layer norm where the rows' spread, and so rstd, is far from one: rstd is in fp32's
range down to spreads of 1e-38 and up to 1e38, its square only between 1e-19 and 1e19 or so.

Bounds, with u = 2^-24: d = h - mean is rounded once, n = d * rstd twice, dy * w once.  A sum over a row
is a chain of at most 32 fp32 adds in a lane and 14 across lanes and waves, of terms good to 4 u; its
mean times rstd takes two more roundings, times n three more, and the three terms of dx two adds: below
64 u of the sum of the terms' sizes.  Adding dh takes one more, of the result.  dweight's terms, good
to 3 u, are added up over a handful of rows.  The values keep away from subnormal results."""
import numpy as np
import pytest
import torch

import plain64 as P
import plain64_training as T
from float8_quantization_moe_amd import training

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U24 = 2.0 ** -24
SPREADS = [1e34, 1e23, 1e21, 3e19, 1e19, 1.0, 1e-10, 1e-19, 1e-20, 1e-25, 1e-33]


def f64(t):
    return t.double().cpu().numpy()


def inputs(K, dtype, spread, seed):
    """Rows of the given spread and means of its size; w and dy ordinary."""
    g = torch.Generator().manual_seed(seed)
    M = 6
    h = ((torch.randn((M, K), generator=g, dtype=torch.float64) + torch.randn((M, 1), generator=g, dtype=torch.float64)) * spread)
    w = 1 + 0.2 * torch.randn(K, generator=g)
    b = 0.3 * torch.randn(K, generator=g)
    dy = torch.randn((M, K), generator=g)
    return [t.to(DT[dtype]).cuda() for t in (h, w, b, dy)]


def check_backward(h, w, mean, rstd, dy, dh, dtype):
    dx, dw, db = training.add_layernorm_bwd(h, w, mean, rstd, dy, dh)
    H, W, MU, R, G = f64(h), f64(w), f64(mean), f64(rstd), f64(dy)
    D = 0 if dh is None else f64(dh)
    want, want_dw, want_db = T.layernorm_bwd(H, W, MU, R, G, None if dh is None else D)
    n = np.abs(H - MU[:, None]) * R[:, None]
    a = np.abs(G * W)
    size = R[:, None] * (a + a.mean(-1, keepdims=True) + n * (a * n).mean(-1, keepdims=True))
    got = f64(dx)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= P.half_step(want, dtype) + 64 * U24 * size + 2 * U24 * (np.abs(want) + np.abs(D)))
    rows = h.shape[0]
    assert np.all(np.abs(f64(dw) - want_dw) <= (4 + rows) * U24 * (np.abs(G) * n).sum(0))
    assert np.all(np.abs(f64(db) - want_db) <= rows * U24 * np.abs(G).sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 1024, 2048, 4096, 5120, 8192, 16384])       # each of the kernel's shapes
@pytest.mark.parametrize("spread", SPREADS)
def test_backward(spread, K, dtype):
    h, w, b, dy = inputs(K, dtype, spread, K)
    mean = h.double().mean(-1)
    rstd = (1 / torch.sqrt((h.double() - mean[:, None]).square().mean(-1))).float()
    dh = (torch.randn(h.shape, generator=torch.Generator().manual_seed(1)).cuda() / spread).to(DT[dtype])
    for d in (None, dh):
        check_backward(h, w, mean.float(), rstd, dy, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread,eps", [(1e34, 1e-5), (1e23, 1e-5), (1e21, 0.0), (1e-20, 0.0), (1e-25, 0.0), (1e-30, 1e-5)])
def test_forward_then_backward(spread, eps, dtype):
    """What the forward pass leaves is what the gradients take."""
    K = 1056
    h, w, b, dy = inputs(K, dtype, spread, 3)
    _, y, _, _, mean, rstd = training.add_layernorm(h, None, w, b, eps)
    want, wm, wr = T.layernorm_fwd(f64(h), f64(w), f64(b), float(np.float32(eps)))
    d = np.abs(f64(h) - wm[:, None])
    size = (d + d.mean(-1, keepdims=True)) * wr[:, None] * np.abs(f64(w)) + np.abs(f64(b))
    assert np.all(np.abs(f64(y) - want) <= P.half_step(want, dtype) + 2.0 ** -17 * size)
    check_backward(h, w, mean, rstd, dy, None, dtype)
