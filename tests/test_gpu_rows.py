"""Rows to their experts and back: the gather (exact), the weighted sum of a token's rows and
its gradients against the 64-bit definitions.

Bounds, with u = 2^-24.  out adds topk products in fp32: topk u of the sum of magnitudes and a
rounding to the type.  drows is one product rounded to fp32, then to the type.  dweights is a
chain of at most 8 ceil(K / 2048) adds in a lane, 6 across the wave and 4 over the waves."""
import numpy as np
import pytest
import torch

import gpu_util as U
import plain64 as P
import plain64_training as T
from float8_quantization_moe_amd import mxq, training

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def step(x, dtype):
    """Rounding to the type: half a step of bf16; of fp32 u of the value."""
    return P.half_step(x, dtype) if dtype == "bf16" else ROUND * np.abs(x)


def ids_of(M, topk, E, dropped, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(max(E, topk))[:topk] for _ in range(M)]).astype(np.int32) if M else np.zeros((0, topk), np.int32)
    ids[rng.random(ids.shape) < dropped] = -1
    ids[rng.random(ids.shape) < dropped / 4] = E
    return np.where(ids >= E, E, ids).astype(np.int32)


CASES = [(1, 8, 1, 1, 0.0), (3, 512, 2, 4, 0.0), (33, 5120, 8, 128, 0.0), (257, 264, 3, 7, 0.2), (5, 16392, 2, 3, 0.5),
         (700, 1032, 1, 300, 0.1), (40, 24, 10, 64, 0.1), (9, 2048, 17, 1024, 0.3), (6, 520, 64, 64, 0.0), (4, 64, 4, 8, 1.0),
         (5000, 40, 6, 16, 0.02)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,topk,E,dropped", CASES)
def test_there_and_back(M, K, topk, E, dropped, dtype):
    dt = DT[dtype]
    ids = ids_of(M, topk, E, dropped, M + K)
    g = torch.Generator().manual_seed(K)
    x = torch.randn((M, K), generator=g).to(dt).cuda()
    n = M * topk
    z = x.element_size()
    rows, ends = U.Guarded(n * K * z, torch.uint8, (n * K * z,)), U.Guarded(E, torch.int32, (E,))
    src, place = U.Guarded(n, torch.int32, (n,)), U.Guarded(n, torch.int32, (M, topk))
    ws = U.Guarded(mxq.mxq_dispatch_rows_workspace_bytes(M, topk, E), torch.uint8, (mxq.mxq_dispatch_rows_workspace_bytes(M, topk, E),))
    rv = rows.t.view(dt).view(n, K)
    mxq.mxq_dispatch_rows(x, torch.from_numpy(ids).cuda(), E, rv, ends.t, src.t, place.t, ws.t)
    torch.cuda.synchronize()
    for gd in (rows, ends, src, place, ws):
        assert gd.guard_intact()
    we, wsrc, wrow = T.dispatch_order(ids, E)
    assert np.array_equal(ends.t.cpu().numpy(), we) and np.array_equal(src.t.cpu().numpy(), wsrc)
    assert np.array_equal(place.t.cpu().numpy(), wrow)
    last = int(we[-1])
    assert torch.equal(rv[:last], x[torch.from_numpy(wsrc[:last].astype(np.int64) // topk).cuda()])
    assert torch.all(rows.t.view(n, K * z)[last:] == U.CANARY)         # rows past the last end: as they were
    # the inverse from src_pair alone
    again = U.Guarded(n, torch.int32, (M, topk))
    mxq.mxq_pair_rows(src.t, again.t)
    assert again.guard_intact() and torch.equal(again.t, place.t)
    # back, from other rows (as the experts leave them), weighted and not
    y = torch.randn((n, K), generator=g).to(dt).cuda()
    y[last:] = float("nan")                                            # rows of no pair reach nothing
    weights = torch.rand((M, topk), generator=g).cuda() + 0.1
    for w in (weights, None):
        out = U.Guarded(M * K * z, torch.uint8, (M * K * z,))
        mxq.mxq_combine_rows(y, place.t, w, out.t.view(dt))
        torch.cuda.synchronize()
        assert out.guard_intact()
        want, size = T.combine(f64(y), wrow, None if w is None else f64(w))
        assert np.all(np.abs(f64(out.t.view(dt).view(M, K)) - want) <= step(want, dtype) + (topk + 1) * ROUND * size)
        dout = torch.randn((M, K), generator=g).to(dt).cuda()
        drows, dw = U.Guarded(n * K * z, torch.uint8, (n * K * z,)), U.Guarded(n, torch.float32, (M, topk))
        mxq.mxq_combine_rows_bwd(dout, y, place.t, w, drows.t.view(dt).view(n, K), dw.t)
        torch.cuda.synchronize()
        assert drows.guard_intact() and dw.guard_intact()
        want_r, want_w, size = T.combine_bwd(f64(dout), f64(y), wrow, None if w is None else f64(w))
        got = f64(drows.t.view(dt).view(n, K))
        assert np.all(np.abs(got[:last] - want_r[:last]) <= step(want_r[:last], dtype) + 2 * ROUND * np.abs(want_r[:last]))
        assert torch.all(drows.t.view(n, K * z)[last:] == U.CANARY)
        assert np.all(np.abs(f64(dw.t) - want_w) <= (8 * -(-K // 2048) + 12) * ROUND * size)
        # drows alone, and in place
        d2 = torch.zeros((n, K), dtype=dt, device="cuda")
        mxq.mxq_combine_rows_bwd(dout, None, place.t, w, d2)
        y2, dw2 = y.clone(), torch.empty_like(dw.t)
        mxq.mxq_combine_rows_bwd(dout, y2, place.t, w, y2, dw2)
        assert torch.equal(d2[:last], drows.t.view(dt).view(n, K)[:last]) and torch.equal(y2[:last], d2[:last])
        assert torch.equal(dw2, dw.t)


def test_combine_is_the_gradient_of_dispatch():
    """<dispatch(x), v> = <x, combine(v)>: exact in small integers."""
    M, K, topk, E = 300, 136, 4, 9
    g = torch.Generator().manual_seed(1)
    ids = torch.from_numpy(ids_of(M, topk, E, 0.2, 3)).cuda()
    x = torch.randint(-4, 5, (M, K), generator=g).float().cuda()
    rows, ends, src, place = training.dispatch_rows(x, ids, E)
    n = int(ends[-1])
    v = torch.randint(-4, 5, rows.shape, generator=g).float().cuda()
    back = training.combine_rows(v, place)
    assert torch.equal((rows[:n] * v[:n]).double().sum(), (x * back).double().sum())


def test_pair_rows_of_a_packed_dispatch():
    M, K, topk, E = 500, 512, 2, 6
    ids = torch.from_numpy(ids_of(M, topk, E, 0.1, 8)).cuda()
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    packed = torch.empty((M * topk, K + K // 32), dtype=torch.uint8, device="cuda")
    ends, src = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(M * topk, dtype=torch.int32, device="cuda")
    ws = torch.empty(mxq.mxq_dispatch_pack_workspace_bytes(M, K, topk, E), dtype=torch.uint8, device="cuda")
    mxq.mxq_dispatch_pack_mx(x, ids, E, packed, ends, src, ws)
    rows, ends2, src2, place = training.dispatch_rows(x, ids, E)
    assert torch.equal(ends, ends2) and torch.equal(src, src2)
    assert torch.equal(training.pair_rows(src, topk), place)
    bad = src.clone()
    bad[3], bad[7] = M * topk, -5                                      # entries that name no pair
    got = training.pair_rows(bad, topk).view(-1).cpu()
    want = place.view(-1).clone().cpu()
    want[src[3].item()] = want[src[7].item()] = -1
    assert torch.equal(got, want)


def test_rows_out_of_range_are_empty_slots():
    K = 72
    rows = torch.randn((5, K), device="cuda")
    place = torch.tensor([[0, 5, -1], [4, 2147483647, -2147483648], [9, -7, 5]], dtype=torch.int32, device="cuda")
    w = torch.rand((3, 3), device="cuda")
    out = training.combine_rows(rows, place, w)
    assert torch.equal(out[0], rows[0] * w[0, 0]) and torch.equal(out[1], rows[4] * w[1, 0]) and torch.all(out[2] == 0)
    drows = torch.full((5, K), 7.0, device="cuda")
    dw = torch.empty((3, 3), device="cuda")
    dout = torch.randn((3, K), device="cuda")
    mxq.mxq_combine_rows_bwd(dout, rows, place, w, drows, dw)
    assert torch.equal(drows[0], dout[0] * w[0, 0]) and torch.equal(drows[4], dout[1] * w[1, 0])
    assert torch.all(drows[1:4] == 7.0) and torch.all(dw.view(-1)[[1, 2, 4, 5, 6, 7, 8]] == 0)
    # no rows at all
    empty = torch.empty((0, K), device="cuda")
    assert torch.all(training.combine_rows(empty, place, w) == 0)
    _, dw = training.combine_rows_bwd(dout, empty, place, w)
    assert torch.all(dw == 0)


def test_a_row_named_by_several_tokens():
    """Forward only: a row may be read by any number of pairs."""
    rows = torch.randn((3, 40), device="cuda").to(torch.bfloat16)
    place = torch.tensor([[0, 0], [0, 2], [2, 2]], dtype=torch.int32, device="cuda")
    out = training.combine_rows(rows, place)
    want = torch.stack([rows[0].float() * 2, rows[0].float() + rows[2].float(), rows[2].float() * 2]).to(torch.bfloat16)
    assert torch.equal(out, want)


def test_nan_and_infinities_stay_with_their_tokens():
    M, K, topk, E = 20, 96, 2, 4
    ids = torch.from_numpy(ids_of(M, topk, E, 0.0, 2)).cuda()
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    x[3, 5] = float("nan")
    rows, ends, src, place = training.dispatch_rows(x, ids, E)
    out = training.combine_rows(rows, place, torch.full((M, topk), 0.5, device="cuda"))
    bad = torch.isnan(out)
    assert bad[3, 5] and bad.sum() == 1
    dout = torch.zeros((M, K), device="cuda").to(torch.bfloat16)
    _, dw = training.combine_rows_bwd(dout, rows, place, None)
    assert torch.all(torch.isnan(dw[3])) and torch.isnan(dw).sum() == topk


def test_no_tokens_and_no_width():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    rows, ends, src, place = training.dispatch_rows(x, torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    assert rows.shape == (0, 64) and torch.all(ends == 0)
    assert training.combine_rows(rows, place).shape == (0, 64)
    dw = torch.full((4, 2), 5.0, device="cuda")
    none = torch.empty((4, 0), device="cuda")
    mxq.mxq_combine_rows_bwd(none, torch.empty((8, 0), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda"), None,
                             torch.empty((8, 0), device="cuda"), dw)
    assert torch.all(dw == 0)


def test_past_two_to_the_31_elements():
    M, K, topk, E = 70000, 16384, 2, 8                                 # rows: 2.3e9 values
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for a in range(0, M, 17500):
        x[a:a + 17500] = torch.randn((17500, K), device="cuda").to(torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.rand((M, E), generator=g, device="cuda").sort(dim=-1).indices[:, :topk].to(torch.int32).contiguous()
    rows, ends, src, place = training.dispatch_rows(x, ids, E)
    at = torch.tensor([0, 1, 65536, 131072, 131073, 139999], device="cuda")
    assert torch.equal(rows[at], x[(src[at] // topk).long()])
    out = training.combine_rows(rows, place)                           # topk copies of a row: doubled exactly
    for t in (0, 34999, M - 1):
        assert torch.equal(out[t].float(), 2 * x[t].float())
    drows, dw = training.combine_rows_bwd(x, rows, place)
    assert torch.equal(drows[at], rows[at])
    want = x[M - 1].double().square().sum()
    assert torch.all((dw[M - 1].double() - want).abs() <= (8 * 8 + 12) * ROUND * want)
