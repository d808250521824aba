"""The routed-experts example end to end against plain 64-bit arithmetic on the same
MXFP4 weights, step by step from each step's actual inputs."""
import os
import sys

import numpy as np
import pytest
import torch

import plain64 as P
from float8_quantization_moe_amd import mxq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("M", [1, 3, 200, 1000])
def test_block(M):
    import routed_experts as R
    K, F, E, topk = 512, 384, 6, 2
    b = R.Block.random(K, F, E, topk, seed=M)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    h, out, saved = R.forward(b, x, res)
    _, rstd, y, logits, ids, per_pair = saved
    assert torch.equal(h, (x.double() + res.double()).to(torch.bfloat16))
    I = ids.cpu().numpy()
    assert ((I >= 0) & (I < E)).all()
    # the experts on the tokens as the pack encodes them, in 64 bits; the silu's rows are encoded in 4 bits, so
    # a value near a rounding boundary there may fall to either side (steps of up to a quarter of it): the bound
    # is on the norm, 0.02 for the few that do and the bf16 roundings of the two products
    q8, s8 = mxq.quantize_mx(y)
    xt = P.mxfp8_decode(q8.cpu().numpy(), s8.cpu().numpy())
    up = np.stack([P.mxfp4_decode(b.up[0][e].cpu().numpy(), b.up[1][e].cpu().numpy()) for e in range(E)])
    down = np.stack([P.mxfp4_decode(b.down[0][e].cpu().numpy(), b.down[1][e].cpu().numpy()) for e in range(E)])
    want = np.zeros((M, topk, K))
    for m in range(M):
        for j in range(topk):
            u = P.bf16_round(up[I[m, j]] @ xt[m])
            a = P.bf16_round(u / (1 + np.exp(-u)))
            q, s = P.mxfp4_encode(a[None], 0)
            want[m, j] = down[I[m, j]] @ P.mxfp4_decode(q, s)[0]
    got = f64(per_pair)
    assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want)
    w = P.route(f64(logits), f64(b.bias), True, 1, 1, topk, True, False, 1.0)[1]
    o = (w[..., None] * got).sum(1)
    assert np.all(np.abs(f64(out) - o) <= P.half_step(o, "bf16") + 2.0 ** -17 * np.abs(w[..., None] * got).sum(1))
    # gradients: the router's path, in 64 bits from the same saved values
    dh, dout = torch.ones_like(h), out
    dx, dnorm, drouter = R.backward(b, saved, dh, dout)
    dw = (f64(dout)[:, None, :] * got).sum(-1)
    dl = P.route_bwd(f64(logits), I.astype(np.int64), dw, True, True, 1.0)
    dy = dl @ f64(b.router)
    want_dx, want_dn = P.norm_bwd(f64(h), f64(b.norm), f64(rstd), dy, f64(dh))
    # dlogits, dy and dx are rounded to bf16 in turn: 3 half steps of 2^-8
    assert np.linalg.norm(f64(dx) - want_dx) <= 3 * 2.0 ** -8 * np.linalg.norm(want_dx)
    assert np.linalg.norm(f64(dnorm) - want_dn) <= 3 * 2.0 ** -8 * np.linalg.norm(want_dn)
    want_dr = dl.T @ f64(y)
    assert np.linalg.norm(f64(drouter) - want_dr) <= 3 * 2.0 ** -8 * np.linalg.norm(want_dr)
