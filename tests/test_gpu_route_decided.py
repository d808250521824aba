"""Biased selection on keys that no rounding can reorder: neighbours lie 0.6 / E apart, an
fp32 score is good to 1e-6, so that every row's ids and weights are compared."""
import numpy as np
import pytest
import torch

import plain64 as P
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu


def spaced(M, E, seed):
    """Keys (M, E): in each row the same E values from 0.2 to 0.8, in another order."""
    rng = np.random.default_rng(seed)
    return np.stack([rng.permutation(E) for _ in range(M)]) * (0.6 / E) + 0.2, rng


def check(l, bias, sigmoid, ng, kg, k, top2, least):
    ids, w = mxq.route_topk(l, k, bias=bias, score="sigmoid" if sigmoid else "softmax", n_groups=ng, topk_groups=kg,
                            renormalize=True, group_top2=top2, scale=2.5)
    want, ww, sure = P.route(l.double().cpu().numpy(), bias.double().cpu().numpy(), sigmoid, ng, kg, k, True, top2, 2.5)
    assert sure.mean() >= least
    assert np.array_equal(ids.cpu().numpy()[sure], want[sure])
    assert np.all(np.abs(w.double().cpu().numpy() - ww)[sure] <= 2.0 ** -18 * ww[sure])


# sums of two keys can tie exactly: those rows are not compared, of five or more rows never all
GROUPS = [(1, 1, False, 1.0), (2, 1, False, 1.0), (8, 4, False, 1.0), (8, 3, True, 0.2)]


@pytest.mark.parametrize("ng,kg,top2,least", GROUPS)
@pytest.mark.parametrize("M,E,k", [(1, 8, 1), (2, 16, 2), (3, 64, 16), (8, 128, 8), (40, 256, 8), (5, 512, 64), (6, 1024, 64), (7, 800, 9)])
def test_sigmoid(M, E, k, ng, kg, top2, least):
    if k > kg * E // ng:
        k = kg * E // ng
    key, rng = spaced(M, E, E + k)
    bias = torch.from_numpy(rng.uniform(-0.1, 0.1, E).astype(np.float32)).cuda()
    s = key - bias.double().cpu().numpy()
    l = torch.from_numpy(np.log(s / (1 - s)).astype(np.float32)).cuda()
    check(l, bias, True, ng, kg, k, top2, least if M > 4 or least == 1.0 else 0.0)


@pytest.mark.parametrize("ng,kg,top2,least", GROUPS[:3])
@pytest.mark.parametrize("E,k", [(8, 1), (16, 2), (64, 16), (128, 8), (256, 8), (512, 64), (1024, 64), (800, 9)])
def test_softmax(E, k, ng, kg, top2, least):
    """One row: its bias makes the keys."""
    k = min(k, kg * E // ng)
    key, rng = spaced(1, E, E)
    l = (2 * rng.standard_normal((1, E))).astype(np.float32)
    bias = (key[0] - P.scores(l.astype(np.float64), False)[0]).astype(np.float32)
    check(torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda(), False, ng, kg, k, top2, least)
