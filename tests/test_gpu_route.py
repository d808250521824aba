"""Expert routing and its gradient against the 64-bit definitions.

Bounds: a score is an exponential and a divide in fp32 (a few units in the last
place), over a sum of at most 1024 terms in a tree of at most 16 + 6 adds; weights
divide by a second sum: 2^-18 relative covers both.  The gradient is a difference
of such products: 2^-17 of the terms' sizes, and half a step of a bf16 output.
Rows whose 64-bit keys lie within 1e-5 of each other at a deciding place are left
out of the comparison of ids (only with a bias or groups; without, the logits
decide and every row counts)."""
import numpy as np
import pytest
import torch

import gpu_util as U
import plain64 as P
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu


def guarded(n, dtype):
    return U.Guarded(n, dtype, (n,))


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def logits_of(M, E, dtype, seed, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    l = 2 * torch.randn((M, E), generator=g)
    if masked:
        l[torch.rand((M, E), generator=g) < masked] = -float("inf")
    if M > 2:
        l[M // 2] = -float("inf")
    return l.to(DT[dtype]).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()


def run(l, bias, sigmoid, ng, kg, k, renorm, top2, scale):
    M = l.shape[0]
    ids, w = guarded(M * k, torch.int32), guarded(M * k, torch.float32)
    flags = (mxq.MXQ_ROUTE_RENORM if renorm else 0) | (mxq.MXQ_ROUTE_GROUP_TOP2 if top2 else 0)
    mxq.mxq_route_topk(l, bias, mxq.MXQ_SCORE_SIGMOID if sigmoid else mxq.MXQ_SCORE_SOFTMAX, ng, kg, flags, scale,
                       ids.t.view(M, k), w.t)
    torch.cuda.synchronize()
    assert ids.guard_intact() and w.guard_intact()
    return ids.t.view(M, k).cpu().numpy().astype(np.int64), f64(w.t).reshape(M, k)


def check(l, bias, sigmoid, ng, kg, k, renorm, top2, scale, least=0.8):
    ids, w = run(l, bias, sigmoid, ng, kg, k, renorm, top2, scale)
    want, ww, sure = P.route(f64(l), None if bias is None else f64(bias), sigmoid, ng, kg, k, renorm, top2, scale)
    assert sure.mean() >= least
    assert np.array_equal(ids[sure], want[sure])
    assert np.all(np.abs(w - ww)[sure] <= 2.0 ** -18 * np.abs(ww)[sure] + 1e-30)
    for row in ids:                                     # valid and distinct, whatever the rounding
        r = row[row >= 0]
        assert len(set(r)) == len(r) and (r < l.shape[1]).all()


SHAPES = [(1, 1, 1), (3, 2, 2), (17, 3, 2), (65, 8, 1), (100, 60, 4), (33, 64, 64), (40, 65, 6), (31, 127, 8), (70, 128, 8),
          (16, 160, 6), (19, 255, 3), (48, 256, 8), (5, 257, 8), (9, 384, 9), (6, 511, 64), (13, 512, 10), (7, 777, 5), (4, 1024, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k", SHAPES)
def test_plain(M, E, k, dtype, sigmoid):
    l, bias = logits_of(M, E, dtype, M + E)
    check(l, None, sigmoid, 1, 1, k, False, False, 1.0, least=1.0)
    check(l, None, sigmoid, 1, 1, k, True, False, 2.5, least=1.0)
    check(l, bias, sigmoid, 1, 1, k, True, False, 1.0, least=0.0 if k > 8 or M < 9 else 0.5)


@pytest.mark.parametrize("top2", [False, True], ids=["max", "top2"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,ng,kg,k", [(8, 8, 3, 2), (8, 4, 1, 2), (60, 5, 2, 7), (64, 64, 9, 9), (128, 8, 4, 8), (126, 7, 6, 5),
                                        (256, 8, 4, 8), (256, 2, 1, 12), (320, 10, 3, 6), (512, 16, 1, 4), (1024, 32, 5, 10)])
def test_groups(E, ng, kg, k, sigmoid, top2):
    M = 41
    for dtype, masked in (("f32", 0.0), ("bf16", 0.3)):
        l, bias = logits_of(M, E, dtype, E + ng, masked)
        check(l, None, sigmoid, ng, kg, k, True, top2, 1.0, least=0.5 if dtype == "f32" else 0.1)
        check(l, bias, sigmoid, ng, kg, k, False, top2, 2.5, least=0.3)


@pytest.mark.parametrize("E", [6, 64, 100, 256, 600])
def test_ties_go_to_the_lowest_index(E):
    l = torch.zeros((5, E), device="cuda")
    l[1, 1::2] = 1.0
    l[2, 0] = -0.0
    l[3] = torch.finfo(torch.float32).min                # the type's lowest value is a value
    l[4, E - 1] = 2.0
    k = min(4, E)
    ids, w = run(l, None, False, 1, 1, k, True, False, 1.0)
    assert ids[0].tolist() == list(range(k))
    odd = [i for i in range(1, E, 2)] + [i for i in range(0, E, 2)]
    assert ids[1].tolist() == odd[:k]
    assert ids[2].tolist() == list(range(k))             # -0 equals +0
    assert ids[3].tolist() == list(range(k)) and np.allclose(w[3], 1.0 / k)
    assert ids[4].tolist() == [E - 1] + list(range(k - 1))
    if E % 2 == 0:
        ids, _ = run(l[:1].contiguous(), torch.zeros(E, device="cuda"), True, 2, 1, min(3, E // 2), False, True, 1.0)
        assert ids[0].tolist() == list(range(min(3, E // 2)))


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True], ids=["nobias", "bias"])
def test_masked_infinite_and_nan(sigmoid, with_bias):
    inf, nan = float("inf"), float("nan")
    E, k = 12, 4
    l = torch.randn((7, E), generator=torch.Generator().manual_seed(1)).cuda()
    l[0] = -inf                                          # an empty row
    l[1, 2:] = -inf                                      # fewer experts than slots
    l[2, 5] = nan
    l[3, 4] = inf
    l[4, :11] = torch.finfo(torch.float32).min
    bias = torch.zeros(E, device="cuda") if with_bias else None
    if with_bias:
        bias[0] = -inf                                   # an expert taken out by its bias
    ids, w = run(l, bias, sigmoid, 1, 1, k, True, False, 1.0)
    assert ids[0].tolist() == [-1] * k and (w[0] == 0).all()
    left = [e for e in (0, 1) if not (with_bias and e == 0)]
    assert sorted(ids[1][:len(left)].tolist()) == left and (ids[1][len(left):] == -1).all()
    assert abs(w[1].sum() - 1) < 1e-6 and (w[1][len(left):] == 0).all()
    assert 5 not in ids[2] and np.isnan(w[2]).all()
    assert (ids[3] < E).all()
    if sigmoid:
        assert ids[3][0] == 4 and np.isfinite(w[3]).all()
    else:
        assert np.isnan(w[3]).all()
    assert ids[4][0] == 11 and np.isfinite(w[4]).all()
    if with_bias:
        assert not (ids == 0).any()
    # groups in which nothing is left
    ids, w = run(l, bias, sigmoid, 4, 2, k, True, True, 1.0)
    assert ids[0].tolist() == [-1] * k and (w[0] == 0).all()
    assert sorted(ids[1][:len(left)].tolist()) == left and (ids[1][len(left):] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [False, True], ids=["raw", "renorm"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k", SHAPES)
def test_backward(M, E, k, sigmoid, renorm, dtype):
    l, _ = logits_of(M, E, dtype, 3 * M + E, 0.1)
    ids, _ = mxq.route_topk(l, k, score="sigmoid" if sigmoid else "softmax")
    dw = torch.randn((M, k), generator=torch.Generator().manual_seed(E)).cuda()
    d = guarded(M * E * l.element_size(), torch.uint8)
    mxq.mxq_route_topk_bwd(l, mxq.MXQ_SCORE_SIGMOID if sigmoid else mxq.MXQ_SCORE_SOFTMAX, ids,
                           mxq.MXQ_ROUTE_RENORM if renorm else 0, 1.5, dw, d.t.view(DT[dtype]))
    torch.cuda.synchronize()
    assert d.guard_intact()
    L, I, D = f64(l), ids.cpu().numpy().astype(np.int64), f64(dw)
    want = P.route_bwd(L, I, D, sigmoid, renorm, 1.5)
    size = P.scores(L, sigmoid) * 1.5 * np.abs(D).max(-1, keepdims=True)
    if renorm:
        s = P.scores(L, sigmoid)
        size = size * 2 / (np.where(I >= 0, np.take_along_axis(s, np.maximum(I, 0), 1), 0).sum(-1, keepdims=True) + 1e-20)
    got = f64(d.t.view(DT[dtype]).view(M, E))
    assert np.all(np.abs(got - want) <= P.half_step(want, dtype) + 2.0 ** -17 * (2 * size + np.abs(want)) + 1e-37)


@pytest.mark.parametrize("renorm", [False, True], ids=["raw", "renorm"])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_backward_against_differences(sigmoid, renorm):
    """Central differences (step 1e-5, good to 1e-9) of the 64-bit weights of the fixed selection."""
    M, E, k = 5, 24, 4
    l, _ = logits_of(M, E, "f32", 11)
    ids, _ = mxq.route_topk(l, k)
    dw = torch.randn((M, k), generator=torch.Generator().manual_seed(2)).cuda()
    d = f64(mxq.route_topk_bwd(l, ids, dw, score="sigmoid" if sigmoid else "softmax", renormalize=renorm, scale=2.0))
    L, I, D = f64(l), ids.cpu().numpy().astype(np.int64), f64(dw)

    def loss(L_):
        s = np.where(I >= 0, np.take_along_axis(P.scores(L_, sigmoid), np.maximum(I, 0), 1), 0.0)
        return (2.0 * (s / (s.sum(-1, keepdims=True) + 1e-20) if renorm else s) * D).sum()

    rng = np.random.default_rng(3)
    for _ in range(8):
        v, t = rng.standard_normal((M, E)), 1e-5
        num = (loss(L + t * v) - loss(L - t * v)) / (2 * t)
        assert abs(num - (d * v).sum()) <= 1e-5 * (np.abs(d * v).sum() + 1e-3)


def test_backward_ignores_ids_out_of_range():
    l, _ = logits_of(1, 40, "f32", 5)
    ids = torch.tensor([[3, -1, 40, 1 << 30]], dtype=torch.int32, device="cuda")
    dw = torch.ones((1, 4), device="cuda")
    d = mxq.route_topk_bwd(l, ids, dw)
    only = mxq.route_topk_bwd(l, ids[:, :1].contiguous(), dw[:, :1].contiguous())
    assert torch.equal(d, only)


def test_ids_feed_the_dispatch_pack():
    """Padding rows route nowhere: the pack drops their slots and keeps every other pair, by expert."""
    M, E, k, K = 200, 16, 2, 256
    l, bias = logits_of(M, E, "f32", 6)
    ids, w = mxq.route_topk(l, k, bias=bias, score="sigmoid", renormalize=True)
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    packed = torch.empty((M * k, K + K // 32), dtype=torch.uint8, device="cuda")
    ends, src = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(M * k, dtype=torch.int32, device="cuda")
    ws = torch.empty(mxq.mxq_dispatch_pack_workspace_bytes(M, K, k, E), dtype=torch.uint8, device="cuda")
    mxq.mxq_dispatch_pack_mx(x, ids, E, packed, ends, src, ws)
    torch.cuda.synchronize()
    flat = ids.cpu().numpy().reshape(-1)
    keep = np.nonzero(flat >= 0)[0]
    assert int(ends[-1]) == len(keep) == (M - 1) * k
    assert np.array_equal(src.cpu().numpy()[:len(keep)], keep[np.argsort(flat[keep], kind="stable")])


def test_past_two_to_the_31_values():
    M, E, k = 2100000, 1024, 2                           # 2.15e9 logits
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.empty((M, E), dtype=torch.bfloat16, device="cuda")
    for a in range(0, M, 262500):
        l[a:a + 262500] = torch.randn((262500, E), generator=g, device="cuda").to(torch.bfloat16)
    ids, w = mxq.route_topk(l, k)
    rows = [0, 1, 1048576, 2097151, 2097152, M - 1]
    want, ww, _ = P.route(f64(l[rows]), None, False, 1, 1, k, False, False, 1.0)
    assert np.array_equal(ids[rows].cpu().numpy(), want)
    assert np.all(np.abs(f64(w[rows]) - ww) <= 2.0 ** -18 * ww)
    d = mxq.route_topk_bwd(l, ids, w)
    want = P.route_bwd(f64(l[rows]), want, f64(w[rows]), False, False, 1.0)
    assert np.all(np.abs(f64(d[rows]) - want) <= P.half_step(want, "bf16") + 2.0 ** -17 * np.abs(f64(w[rows])).max())


def test_no_rows_and_other_stream():
    ids, w = mxq.route_topk(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2)
    l, bias = logits_of(3000, 128, "f32", 7)
    want = mxq.route_topk(l, 8, bias=bias, score="sigmoid", n_groups=8, topk_groups=4, group_top2=True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = mxq.route_topk(l, 8, bias=bias, score="sigmoid", n_groups=8, topk_groups=4, group_top2=True)
    st.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
