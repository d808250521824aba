"""The routing's gradient where the selected scores are small against the row's others:
a bias or groups keep the row's largest logits out of the selection.

Bounds.  A softmax score is good to what the rounding of the difference l - max l does to
its exponential (2^-18 while that is below 128) and a few units of 2^-24 of the exponential,
the sum and the divide.  The gradient is products of such scores and their sums, so each of
its terms is good to four such factors: 2^-16 of the terms' sizes, and half a step of a
bf16 output."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import plain64 as P
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def sizes(L, I, D, scale):
    """Sums of the magnitudes of the renormalised softmax's gradient terms."""
    s = P.scores(L, False)
    some = I >= 0
    sel = np.where(some, np.take_along_axis(s, np.maximum(I, 0), 1), 0.0)
    S = sel.sum(-1, keepdims=True)
    kept, tiny = S / (S + P.TINY), P.TINY / (S + P.TINY)
    q = sel / np.where(S > 0, S, 1.0)
    u = np.where(some, np.abs(D), 0.0) * scale
    m = (u * q).sum(-1, keepdims=True)
    size = s * m * kept * tiny
    for r in range(len(L)):
        size[r, I[r][some[r]]] += (q * kept * (u + m))[r][some[r]]
    return size


def gradient(L, I, D, scale):
    """The renormalised softmax's gradient from 64-bit scores, its differences in 60 digits: in doubles they would
    cancel to 1e-17 of the weights, where gradients of 1e-20 of them are looked at."""
    s = P.scores(L, False)
    out = np.zeros_like(s)
    with localcontext() as c:
        c.prec = 60
        for r in range(len(L)):
            row = [Decimal(float(v)) for v in s[r]]
            g = {int(e): Decimal(float(u)) * Decimal(scale) for e, u in zip(I[r], D[r]) if e >= 0}
            total = sum((row[e] for e in g), Decimal(0)) + Decimal("1e-20")
            mean = sum((u * row[e] for e, u in g.items()), Decimal(0)) / total
            up = {e: (u - mean) / total for e, u in g.items()}
            through = sum((u * row[e] for e, u in up.items()), Decimal(0))
            out[r] = [float(row[e] * (up.get(e, Decimal(0)) - through)) for e in range(len(row))]
    return out


def check(l, ids, dw, scale, dtype):
    got = f64(mxq.route_topk_bwd(l, ids, dw, renormalize=True, scale=scale))
    L, I, D = f64(l), ids.cpu().numpy().astype(np.int64), f64(dw)
    want = gradient(L, I, D, scale)
    assert np.all(np.abs(want - P.route_bwd(L, I, D, False, True, scale)) <= 1e-14 * (1 + np.abs(D).max()) * scale)
    assert np.all(np.abs(got - want) <= P.half_step(want, dtype) + 2.0 ** -16 * sizes(L, I, D, scale) + 1e-30)
    return L, I, D, got


@pytest.mark.parametrize("gap", [0.0, 20.0, 40.0, 46.0, 50.0, 60.0, 80.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,k", [(6, 1), (6, 2), (64, 6), (100, 8), (256, 8), (600, 10), (1024, 64)])
def test_a_bias_takes_the_largest_logit_out(E, k, dtype, gap):
    """Softmax, renormalised; the selected logits lie `gap` below one that its bias masks."""
    M = 9
    g = torch.Generator().manual_seed(E + k)
    l = 0.5 * torch.randn((M, E), generator=g)
    at = torch.randint(0, E, (), generator=g).item()
    l[:, at] = gap
    l = l.to(DT[dtype]).cuda()
    bias = torch.zeros(E, device="cuda")
    bias[at] = -float("inf")
    # (the keys are scores of about exp(-gap): any expert but the masked one may be selected)
    ids, w = mxq.route_topk(l, k, bias=bias, renormalize=True)
    I = ids.cpu().numpy()
    assert not (I == at).any()
    dw = torch.randn((M, k), generator=g).cuda()
    check(l, ids, dw, 1.5, dtype)


def test_weights_and_gradient_are_of_one_function():
    """Central differences (step 1e-4: good to 1e-7 of the second derivatives' size) of the 64-bit weights."""
    E, k = 12, 3
    for gap in (30.0, 44.0, 46.0, 48.0):
        l = torch.randn((4, E), generator=torch.Generator().manual_seed(3)).cuda()
        l[:, 0] = gap
        bias = torch.zeros(E, device="cuda")
        bias[0] = -float("inf")
        ids, w = mxq.route_topk(l, k, bias=bias, renormalize=True, scale=2.0)
        dw = torch.randn((4, k), generator=torch.Generator().manual_seed(4)).cuda()
        d = f64(mxq.route_topk_bwd(l, ids, dw, renormalize=True, scale=2.0))
        L, I, D = f64(l), ids.cpu().numpy().astype(np.int64), f64(dw)

        def weights(L_):
            s = np.take_along_axis(P.scores(L_, False), I, 1)
            return 2.0 * s / (s.sum(-1, keepdims=True) + P.TINY)

        assert np.all(np.abs(f64(w) - weights(L)) <= 2.0 ** -16 * weights(L))
        size = sizes(L, I, D, 2.0)
        rng = np.random.default_rng(5)
        for _ in range(6):
            v, t = rng.standard_normal(L.shape), 1e-4
            num = (weights(L + t * v) * D - weights(L - t * v) * D).sum() / (2 * t)
            assert abs(num - (d * v).sum()) <= 2.0 ** -16 * (size * np.abs(v)).sum() + 1e-6 * size.sum()


@pytest.mark.parametrize("n_groups,topk_groups", [(8, 2), (4, 1)])
def test_groups_keep_the_largest_logit_out(n_groups, topk_groups):
    """The value of a group is the sum of its two largest keys: a masked-off group may hold the row's largest logit."""
    M, E, k = 33, 64, 4
    g = torch.Generator().manual_seed(9)
    l = torch.randn((M, E), generator=g).cuda()
    size = E // n_groups
    l[:, -size:] += 52.0                                     # the last group's experts dominate the softmax ...
    bias = torch.zeros(E, device="cuda")
    bias[-size:] = -4.0                                      # ... and their bias takes that group out
    ids, _ = mxq.route_topk(l, k, bias=bias, n_groups=n_groups, topk_groups=topk_groups, renormalize=True, group_top2=True)
    assert (ids < E - size).all() and (ids >= 0).all()
    dw = torch.randn((M, k), generator=g).cuda()
    check(l, ids, dw, 1.0, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_with_nothing_selected(dtype):
    l = torch.randn((5, 40), generator=torch.Generator().manual_seed(2)).to(DT[dtype]).cuda()
    l[1] = -float("inf")
    l[2, 7:] = -float("inf")
    ids = torch.tensor([[-1, -1], [-1, -1], [3, -1], [5, 39], [-1, 0]], dtype=torch.int32, device="cuda")
    dw = torch.randn((5, 2), generator=torch.Generator().manual_seed(3)).cuda()
    _, _, _, got = check(l, ids, dw, 1.0, dtype)
    assert (got[:2] == 0).all() and (got[2, 7:] == 0).all()


@pytest.mark.parametrize("renorm", [False, True], ids=["raw", "renorm"])
@pytest.mark.parametrize("top", [5.0, 12.0, 17.0, 25.0, 60.0])
def test_sigmoid_of_large_logits(top, renorm):
    """The slope s (1 - s) of a sigmoid near 1 is exp(-l), not the rounding of 1 - s.

    Its exponential is good to 2^-24 (2 + l / 2) (the exponent's rounding and a few units), the rest to six units: 2^-19 of
    the slope up to l = 60.  With renormalisation the slope is multiplied by a difference, good to 2^-19 of its terms."""
    M, E, k = 12, 64, 5
    g = torch.Generator().manual_seed(int(top))
    l = (top * (2 * torch.rand((M, E), generator=g) - 1)).cuda()
    ids, _ = mxq.route_topk(l, k, score="sigmoid")
    ids[1::2] = E - 1 - ids[1::2] if (ids >= 0).all() else ids[1::2]       # other experts than the largest too
    dw = torch.randn((M, k), generator=g).cuda()
    got = f64(mxq.route_topk_bwd(l, ids, dw, score="sigmoid", renormalize=renorm, scale=2.0))
    L, I, D = f64(l), ids.cpu().numpy().astype(np.int64), 2.0 * f64(dw)
    x = np.take_along_axis(L, I, 1)
    e = np.exp(-np.abs(x))
    slope = e / (1 + e) ** 2
    u, size = D, np.abs(D)
    if renorm:
        s = np.where(x > 0, 1, e) / (1 + e)
        t = s.sum(-1, keepdims=True) + P.TINY
        u = (D - (D * s).sum(-1, keepdims=True) / t) / t
        size = (np.abs(D) + (np.abs(D) * s).sum(-1, keepdims=True) / t) / t
    tol = slope * (2.0 ** -19 * np.abs(u) + (2.0 ** -19 * size if renorm else 0))
    assert np.all(np.abs(np.take_along_axis(got, I, 1) - slope * u) <= tol + 1e-36)
    other = np.ones((M, E), bool)
    np.put_along_axis(other, I, False, 1)
    assert (got[other] == 0).all()


@pytest.mark.parametrize("renorm", [False, True], ids=["raw", "renorm"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E", [5, 40, 128, 250, 300, 1000])
def test_a_row_with_nan_or_infinity_has_a_gradient_of_nan(E, dtype, renorm):
    """As its weights are; the rows beside it, which share its wave, are as without it."""
    M, k = 21, 3
    l = torch.randn((M, E), generator=torch.Generator().manual_seed(E)).to(DT[dtype]).cuda()
    ids, _ = mxq.route_topk(l, k)
    dw = torch.randn((M, k), generator=torch.Generator().manual_seed(1)).cuda()
    want = mxq.route_topk_bwd(l, ids, dw, renormalize=renorm)
    bad = l.clone()
    bad[3, E - 1] = float("nan")                         # (of an expert that need not be selected)
    bad[8, 0] = float("inf")
    bad[13] = float("nan")
    bad[14, 1:] = -float("inf")                          # no fault: a row with one expert left
    got = mxq.route_topk_bwd(bad, ids, dw, renormalize=renorm)
    for r in (3, 8, 13):
        assert torch.isnan(got[r]).all()
        assert torch.isnan(mxq.route_topk(bad, k, renormalize=renorm)[1][r]).all()
    assert torch.isfinite(got[14]).all()
    rest = [r for r in range(M) if r not in (3, 8, 13, 14)]
    assert torch.equal(got[rest], want[rest])
