"""rstd of the norm to the last units.

With u = 2^-24: a lane adds up C chunks in eight chains (C roundings, of fused products), joins
them in 3 adds, 64 lanes in 6 and four waves in 3 more; every term is positive, so the sum of
squares is good to (C + 12) u, and 1 / sqrt, taken in doubles and rounded once, to half of
that and one u."""
import numpy as np
import pytest
import torch

from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-5, 0.3])
@pytest.mark.parametrize("M,K", [(2000, 32), (500, 512), (500, 1024), (500, 2048), (500, 4096), (700, 5120), (300, 8192), (300, 16384)])
def test_rstd(M, K, eps, dtype):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn((M, K), generator=g) * torch.exp(2 * torch.randn((M, 1), generator=g))).to(dtype).cuda()
    h, _, _, _, rstd = mxq.add_rmsnorm(x, None, torch.ones(K, dtype=dtype, device="cuda"), eps)
    sq = x.double().cpu().numpy() ** 2
    want = 1 / np.sqrt(sq.mean(-1) + np.float64(np.float32(eps)))
    C = -(-K // 8 // (64 if K <= 2048 else 256))
    bound = ((C + 12) / 2 + 1) * 2.0 ** -24
    assert np.all(np.abs(rstd.double().cpu().numpy() - want) <= bound * want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 2048, 5120])
def test_nan_and_infinity_as_the_formula_has_them(K, dtype):
    """rstd is NaN, or 0: a row with NaN is NaN; one with an infinity is 0, and inf * 0 where it stands."""
    x = torch.randn((4, K), generator=torch.Generator().manual_seed(K)).to(dtype).cuda()
    r = torch.zeros_like(x)
    x[0, K - 1] = float("nan")
    x[1, 33], x[3, 0], r[3, 0] = -float("inf"), float("inf"), -float("inf")          # (the last sum is NaN)
    h, y, q, s, rstd = mxq.add_rmsnorm(x, r, torch.ones(K, dtype=dtype, device="cuda"), 1e-5)
    for row in (0, 3):
        assert torch.isnan(y[row]).all() and (s[row] == 255).all() and (q[row] == 0x7F).all() and torch.isnan(rstd[row])
    at = torch.arange(K, device="cuda") == 33
    assert torch.equal(torch.isnan(y[1]), at) and (y[1][~at] == 0).all() and rstd[1] == 0
    assert torch.equal(s[1] == 255, torch.arange(K // 32, device="cuda") == 1)
    assert torch.isfinite(y[2]).all()
