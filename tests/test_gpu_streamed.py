"""Inputs past the size of the last-level cache (256 MB), which the layer norm's and the rows' kernels read, and some
write, as streams: the same rows in pieces below that size have to give the same bits, since a row's results depend on
that row alone.  (The pieces' kernels are compared with 64-bit forms in their own tests.)  The sums over the rows are
compared with sums in doubles: the rows of a workgroup one after the other, its waves, then up to 512 parts in 32 slices
of 16 and the slices, of terms good to 4 u, u = 2^-24."""
import pytest
import torch

from float8_quantization_moe_amd import mxq, training

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CACHE = 256 << 20
U24 = 2.0 ** -24
EPS = 1e-5
WIDTHS = [512, 1024, 2048, 4096, 5120, 8192, 16384]        # each of the layer norm's shapes


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


def pieces(M, parts=5):
    at = [M * i // parts for i in range(parts + 1)]
    return [slice(a, b) for a, b in zip(at, at[1:])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False], ids=["add", "plain"])
@pytest.mark.parametrize("K", WIDTHS)
def test_layer_norm(K, residual, dtype):
    z = 2 if dtype == "bf16" else 4
    M = CACHE // (z * K * (2 if residual else 1)) + 37
    x = rand((M, K), dtype, K) + 0.5
    r = rand((M, K), dtype, K + 1) if residual else None
    w, b = (1 + 0.2 * rand((K,), "f32", 2)).to(DT[dtype]), (0.3 * rand((K,), "f32", 3)).to(DT[dtype])
    whole = training.add_layernorm(x, r, w, b, EPS)
    for p in pieces(M):
        part = training.add_layernorm(x[p], None if r is None else r[p], w, b, EPS)
        for name, a, c in zip("h y q s mean rstd".split(), whole, part):
            assert torch.equal(a[p], c), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False], ids=["dh", "nodh"])
@pytest.mark.parametrize("K", WIDTHS)
def test_layer_norm_gradients(K, with_dh, dtype):
    z = 2 if dtype == "bf16" else 4
    M = CACHE // (z * K * (3 if with_dh else 2)) + 37
    h, dy = rand((M, K), dtype, K) + 0.5, rand((M, K), dtype, K + 1)
    dh = rand((M, K), dtype, K + 2) if with_dh else None
    w = (1 + 0.2 * rand((K,), "f32", 2)).to(DT[dtype])
    mean = h.double().mean(-1).float()
    rstd = (1 / torch.sqrt(h.double().var(-1, unbiased=False) + EPS)).float()
    dx, dw, db = training.add_layernorm_bwd(h, w, mean, rstd, dy, dh)
    sums = torch.zeros((4, K), dtype=torch.float64, device="cuda")              # dw, db and their sums of magnitudes
    for p in pieces(M):
        part, _, _ = training.add_layernorm_bwd(h[p], w, mean[p], rstd[p], dy[p], None if dh is None else dh[p])
        assert torch.equal(dx[p], part)
        n, g = (h[p].double() - mean[p].double()[:, None]) * rstd[p].double()[:, None], dy[p].double()
        sums += torch.stack([(g * n).sum(0), g.sum(0), (g * n).abs().sum(0), g.abs().sum(0)])
    adds = -(-M // (512 * (4 if K <= 2048 else 1))) + 3 + 16 + 32
    assert torch.all((dw.double() - sums[0]).abs() <= (adds + 4) * U24 * sums[2])
    assert torch.all((db.double() - sums[1]).abs() <= adds * U24 * sums[3])


def routed(M, topk, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand((M, E), generator=g, device="cuda").sort(dim=-1).indices[:, :topk].to(torch.int32)
    ids[torch.rand((M, topk), generator=g, device="cuda") < 0.05] = -1
    return ids.contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,topk", [(5120, 8), (1032, 2), (264, 10)])
def test_rows(K, topk, dtype):
    z, E = 2 if dtype == "bf16" else 4, 16
    M = CACHE // (z * K * topk) + 37
    ids = routed(M, topk, E, K)
    x = rand((M, K), dtype, K)
    rows, ends, src, place = training.dispatch_rows(x, ids, E)
    n = int(ends[-1])
    assert torch.equal(rows[:n], x[(src[:n] // topk).long()]) and torch.all(src[n:] == -1)
    assert torch.equal(place.view(-1)[src[:n].long()], torch.arange(n, dtype=torch.int32, device="cuda"))
    y, weights = rand((M * topk, K), dtype, 5), rand((M, topk), "f32", 6).abs()
    out, bare = training.combine_rows(y, place, weights), training.combine_rows(y, place)
    dout = rand((M, K), dtype, 7)
    drows, dweights = torch.zeros_like(y), torch.empty_like(weights)
    mxq.mxq_combine_rows_bwd(dout, y, place, weights, drows, dweights)
    again = torch.zeros_like(y)
    for p in pieces(M):
        at, wp = place[p].contiguous(), weights[p].contiguous()
        assert torch.equal(out[p], training.combine_rows(y, at, wp)) and torch.equal(bare[p], training.combine_rows(y, at))
        dw = torch.empty_like(wp)
        mxq.mxq_combine_rows_bwd(dout[p], y, at, wp, again, dw)
        assert torch.equal(dweights[p], dw)
    assert torch.equal(drows, again) and torch.all(again[n:] == 0)
