"""Inf and NaN do not end at the product with MXFP4 weights: the codes and scales that the
quantizers write for them give NaN in exactly the results that they reach."""
import pytest
import torch

import gpu_util as U
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu

FMTS = [mxq.MXQ_FMT_E4M3, mxq.MXQ_FMT_E2M1]
# few rows; tiles of 128 and of 256 rows; K of one scale word, with half a slot at its end, of whole slots
SHAPES = [(5, 136, 128), (9, 72, 640), (5, 136, 2560), (300, 136, 128), (333, 264, 384), (700, 520, 1024), (4400, 4104, 640)]


def tokens(x, fmt):
    return mxq.quantize_mx(x) if fmt == mxq.MXQ_FMT_E4M3 else mxq.quantize_mxfp4(x)


def case(M, N, K, fmt):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((2 * N, K), generator=g, device="cuda").to(torch.bfloat16)
    ends = torch.tensor([M // 3, M - 1], dtype=torch.int32, device="cuda")        # a row of its own past the last end
    return x, w, ends


def product(xq, xs, w, ends, fmt, dtype):
    wq, ws = mxq.quantize_mxfp4(w, mxq.MXQ_SCALE_RCEIL)
    return mxq.mxfp4_grouped_mm(xq, xs, wq.view(2, w.shape[0] // 2, -1), ws.view(2, w.shape[0] // 2, -1), ends, x_format=fmt,
                                out_dtype=dtype)


def check(got, clean, where):
    assert torch.equal(torch.isnan(got), where)
    assert torch.equal(torch.where(where, torch.zeros_like(got), got), torch.where(where, torch.zeros_like(clean), clean))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", FMTS, ids=["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_token_rows(M, N, K, fmt, dtype):
    """A row for as many places along K as there are rows to spare, Inf and NaN in turn."""
    x, w, ends = case(M, N, K, fmt)
    clean = product(*tokens(x, fmt), w, ends, fmt, dtype)
    bad, where = x.clone(), torch.zeros((M, N), dtype=torch.bool, device="cuda")
    n = min(M // 2, 40)
    for i in range(n):
        r = (2 * i * (M - 2)) // (2 * n)
        bad[r, (K - 1) * i // max(n - 1, 1)] = [float("nan"), float("inf"), -float("inf")][i % 3]
        where[r] = True
    bad[M - 1, 0] = float("nan")                          # past the last end: zeros all the same
    check(product(*tokens(bad, fmt), w, ends, fmt, dtype), clean, where)


@pytest.mark.parametrize("fmt", FMTS, ids=["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weight_rows(M, N, K, fmt):
    x, w, ends = case(M, N, K, fmt)
    q = tokens(x, fmt)
    clean = product(*q, w, ends, fmt, torch.float32)
    bad, where = w.clone(), torch.zeros((M, N), dtype=torch.bool, device="cuda")
    for g, n, k in ((0, 3, 0), (0, N - 1, K - 1), (1, 0, K // 2), (1, N - 1, 33)):
        bad[g * N + n, k] = float("nan")
        where[M // 3 if g else 0:M - 1 if g else M // 3, n] = True
    check(product(*q, bad, ends, fmt, torch.float32), clean, where)


@pytest.mark.parametrize("M", [4, 500])
def test_a_nan_code_under_an_ordinary_scale(M):
    N, K = 64, 512
    x, w, ends = case(M, N, K, mxq.MXQ_FMT_E4M3)
    q, s = mxq.quantize_mx(x)
    clean = product(q, s, w, ends, mxq.MXQ_FMT_E4M3, torch.float32)
    q = q.clone()
    q[0, 77], q[M - 2, K - 1] = 0x7F, 0xFF
    where = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    where[0], where[M - 2] = True, True
    check(product(q, s, w, ends, mxq.MXQ_FMT_E4M3, torch.float32), clean, where)


def test_from_the_pack_and_the_norm():
    """A token row with NaN through the norm, the pack and the product on packed rows."""
    M, K, N, E, k = 96, 512, 128, 4, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    x[17, 300] = float("nan")
    y = mxq.add_rmsnorm(x, None, torch.ones(K, dtype=torch.bfloat16, device="cuda"), 1e-5)[1]
    ids, _ = mxq.route_topk(torch.randn((M, E), generator=g, device="cuda"), k)
    packed = torch.empty((M * k, K + K // 32), dtype=torch.uint8, device="cuda")
    ends, src = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(M * k, dtype=torch.int32, device="cuda")
    mxq.mxq_dispatch_pack_mx(y, ids, E, packed, ends, src, torch.empty(
        mxq.mxq_dispatch_pack_workspace_bytes(M, K, k, E), dtype=torch.uint8, device="cuda"))
    w = torch.randn((E * N, K), generator=g, device="cuda").to(torch.bfloat16)
    wq, ws = mxq.quantize_mxfp4(w)
    out = torch.empty((M * k, N), dtype=torch.bfloat16, device="cuda")
    mxq.mxq_mxfp4_grouped_mm_packed(packed, wq.view(E, N, -1), ws.view(E, N, -1), ends, out)
    assert torch.equal(torch.isnan(out), (src // k == 17).unsqueeze(1).expand(M * k, N))
    assert U.host_u8(packed[(src // k == 17)][:, K:]).max() == 255
