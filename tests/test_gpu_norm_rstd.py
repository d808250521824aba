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
