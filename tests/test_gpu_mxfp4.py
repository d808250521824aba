"""MXFP4 codec (bit for bit) and the grouped product with MXFP4 weights against the
64-bit definitions.

Bounds of the product, relative to A = sum |x w|: with E2M1 tokens a block of 32
products is exact (multiples of 1/4 below 36 * 32), so only the adds of at most
K / 32 blocks and two per step round: (K / 16) 2^-24 A.  With E4M3 tokens the matrix
core cuts products off 14 bits below a block's largest: 2^-10 A, as for the MXFP8
product.  A bf16 result adds half a step of bf16 (and the
step grows with what the sum is off: 2^-7 of the bound)."""
import numpy as np
import pytest
import torch

import gpu_util as U
import plain64 as P
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu


def guarded(n, dtype):
    return U.Guarded(n, dtype, (n,))


RULES = [mxq.MXQ_SCALE_FLOOR, mxq.MXQ_SCALE_RCEIL]


def quantize(bits, rule):
    M, K = bits.shape
    q, s = guarded(M * K // 2, torch.uint8), guarded(M * K // 32, torch.uint8)
    mxq.mxq_quantize_mxfp4(U.dev_bf16(bits), rule, q.t, s.t)
    torch.cuda.synchronize()
    assert q.guard_intact() and s.guard_intact()
    return U.host_u8(q.t).reshape(M, K // 2), U.host_u8(s.t).reshape(M, K // 32)


@pytest.mark.parametrize("rule", RULES, ids=["floor", "rceil"])
def test_every_significand_under_every_scale(rule):
    """For each exponent of a block's maximum and three of its significands: every bf16 of the six binades below,
    both signs (smaller values round to zero like the smallest of these)."""
    rows = []
    for E in range(255):
        mags = np.arange(max(0, E - 5) << 7, (E + 1) << 7, dtype=np.int64)
        for top in (0x7F, 0x41, 0x40, 0x00):
            m = np.minimum(mags, (E << 7) | top)
            both = np.concatenate([m, m | 0x8000])
            both = np.concatenate([both, np.zeros(-len(both) % 31, np.int64)])
            blocks = both.reshape(-1, 31)
            lead = np.full((len(blocks), 1), (E << 7) | top)
            rows.append(np.concatenate([lead, blocks], 1))
    bits = np.concatenate(rows).astype(np.uint16)
    q, s = quantize(bits, rule)
    oq, os_ = P.mxfp4_encode(P.bf16_value(bits), rule)
    assert np.array_equal(s, os_)
    bad = np.nonzero(q != oq)
    assert np.array_equal(q, oq), (bits[bad[0][0]], q[bad[0][0]], oq[bad[0][0]])


@pytest.mark.parametrize("rule", RULES, ids=["floor", "rceil"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 64), (3, 96), (7, 1024), (129, 2080), (33, 5120), (1, 16384)])
def test_quantize_shapes_and_round_trip(M, K, rule):
    rng = np.random.default_rng(M + K)
    bits = rng.integers(0, 1 << 16, (M, K)).astype(np.uint16)          # every pattern: infinities and NaN too
    near = (rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))).astype(np.float32)
    for b in (bits, (near.view(np.uint32) >> 16).astype(np.uint16)):
        q, s = quantize(b, rule)
        v = P.bf16_value(b)
        oq, os_ = P.mxfp4_encode(v, rule)
        assert np.array_equal(q, oq) and np.array_equal(s, os_)
        y = guarded(M * K * 2, torch.uint8)
        mxq.mxq_dequantize_mxfp4(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), y.t.view(torch.bfloat16).view(M, K))
        torch.cuda.synchronize()
        assert y.guard_intact()
        want = P.past_bf16_is_inf(P.mxfp4_decode(q, s))
        got = y.t.view(torch.bfloat16).view(M, K).double().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(np.signbit(got[~np.isnan(got)]), np.signbit(want[~np.isnan(want)]))


def test_every_code_under_every_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))            # row s: every byte, scale s in all 16 blocks
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    y = mxq.dequantize_mxfp4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    got = y.double().cpu().numpy()
    want = P.past_bf16_is_inf(P.mxfp4_decode(codes, scales))
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(U.host_u16(y[255]), np.full(512, 0x7FC0, np.uint16))


def test_codec_past_two_to_the_31_elements():
    M, K = 131200, 16384
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for a in range(0, M, 16400):
        x[a:a + 16400] = torch.randn((16400, K), generator=g, device="cuda").to(torch.bfloat16)
    q, s = mxq.quantize_mxfp4(x)
    y = mxq.dequantize_mxfp4(q, s)
    rows = [0, 65599, 131071, 131072, M - 1]
    oq, os_ = P.mxfp4_encode(x[rows].double().cpu().numpy(), 0)
    assert np.array_equal(U.host_u8(q[rows]), oq) and np.array_equal(U.host_u8(s[rows]), os_)
    assert np.array_equal(y[rows].double().cpu().numpy(), P.mxfp4_decode(oq, os_))


# ------------------------------------------------------------------ product --
def operands(M, N, K, G, fmt, seed, wide=True):
    """Random codes (no NaN) with a scale of its own for every block."""
    rng = np.random.default_rng(seed)
    lo, hi = (118, 136) if wide else (127, 128)
    wq = rng.integers(0, 256, (G, N, K // 2)).astype(np.uint8)
    ws = rng.integers(lo, hi, (G, N, K // 32)).astype(np.uint8)
    xs = rng.integers(lo, hi, (M, K // 32)).astype(np.uint8)
    if fmt == mxq.MXQ_FMT_E2M1:
        xq = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
    else:
        xq = rng.integers(0, 256, (M, K)).astype(np.uint8)
        xq = np.where(xq & 0x7F == 0x7F, 0x40, xq).astype(np.uint8)
    return xq, xs, wq, ws


def multiply(xq, xs, wq, ws, ends, fmt, dtype):
    M, (G, N, half) = xq.shape[0], wq.shape
    size = 2 if dtype == torch.bfloat16 else 4
    y = guarded(M * N * size, torch.uint8)
    dev = [torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in (xq, xs, wq, ws)]
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")
    mxq.mxq_mxfp4_grouped_mm(dev[0], dev[1], fmt, dev[2], dev[3], offs, y.t.view(dtype).view(M, N))
    torch.cuda.synchronize()
    assert y.guard_intact()
    return y.t.view(dtype).view(M, N)


def check(xq, xs, wq, ws, ends, fmt, dtype):
    G, N, half = wq.shape
    K = 2 * half
    y = multiply(xq, xs, wq, ws, ends, fmt, dtype).double().cpu().numpy()
    x = P.mxfp4_decode(xq, xs) if fmt == mxq.MXQ_FMT_E2M1 else P.mxfp8_decode(xq, xs)
    w = P.mxfp4_decode(wq.reshape(G * N, half), ws.reshape(G * N, -1)).reshape(G, N, K)
    want, size = P.product(x, w, ends)
    tol = (K / 16 * 2.0 ** -24 if fmt == mxq.MXQ_FMT_E2M1 else 2.0 ** -10) * size
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -7) + P.half_step(want, "bf16")
    bad = np.abs(y - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(y - want).max(), bad.mean())
    return y


FMTS = [mxq.MXQ_FMT_E4M3, mxq.MXQ_FMT_E2M1]
# (M, N, K, ends): one row to many, odd column counts, empty groups, rows past the last end, offsets out of order
CASES = [
    (1, 8, 128, [1]),
    (1, 64, 256, [0, 1, 1]),
    (1, 1736, 5120, [0, 0, 1, 1]),
    (5, 24, 384, [2, 2, 5]),
    (16, 72, 128, [16]),
    (17, 136, 640, [1, 17]),
    (33, 200, 512, [10, 30]),                       # rows past the last end: zeros
    (31, 64, 1152, [40, 12, 31]),                   # clamped offsets
    (40, 128, 256, [-3, 7, 7, 90]),
    (64, 264, 768, [64]),
    (65, 256, 896, [65]),
    (129, 520, 640, [0, 128, 129]),
    (200, 264, 1408, [3, 3, 68, 69, 197]),
    (300, 248, 128, [257, 300]),
    (513, 1032, 384, [100, 356, 513]),
    (700, 512, 2048, [130, 131, 387, 700]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", FMTS, ids=["mxfp8", "mxfp4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%dx%d" % c[:3])
def test_product(case, fmt, dtype):
    M, N, K, ends = case
    check(*operands(M, N, K, len(ends), fmt, M + N + K), ends, fmt, dtype)


# enough tiles for 256 rows each, the groups' last ones of every height; K of one slot and less, odd halves
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", FMTS, ids=["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,N,K,ends", [
    (4200, 4096, 128, [4200]),
    (4200, 4096, 256, [1030, 1300, 4190]),
    (4300, 4104, 384, [300, 300, 1000, 4300]),
    (4170, 4360, 640, [60, 130, 4100, 4170]),
    (4400, 4096, 1024, [2000, 4400]),
], ids=lambda v: str(v) if isinstance(v, int) else "")
def test_product_many_rows(M, N, K, ends, fmt, dtype):
    check(*operands(M, N, K, len(ends), fmt, M + N + K), ends, fmt, dtype)


@pytest.mark.parametrize("seed", range(24))
def test_product_random_shapes(seed):
    r = np.random.default_rng(seed)
    G = int(r.choice([1, 2, 3, 7, 16, 40]))
    M, N, K = int(np.exp(r.uniform(0, np.log(900)))), 8 * int(r.integers(1, 90)), 128 * int(r.integers(1, 13))
    ends = np.sort(r.integers(0, M + 4, G)).tolist()
    fmt, dtype = int(r.choice(FMTS)), [torch.bfloat16, torch.float32][int(r.integers(0, 2))]
    print(M, N, K, ends, fmt, dtype, flush=True)
    check(*operands(M, N, K, G, fmt, seed), ends, fmt, dtype)


@pytest.mark.parametrize("fmt", FMTS, ids=["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M", [3, 300])
def test_every_k_position_and_scale_block(M, fmt):
    """One-hot tokens: row m holds a single 1 at k = 7 m (mod K) and picks column k of the weights exactly."""
    K, N = 512, 72
    _, _, wq, ws = operands(1, N, K, 1, fmt, 5)
    xs = np.random.default_rng(1).integers(120, 134, (M, K // 32)).astype(np.uint8)
    k = (7 * np.arange(M)) % K
    if fmt == mxq.MXQ_FMT_E2M1:
        xq = np.zeros((M, K // 2), np.uint8)
        xq[np.arange(M), k // 2] = np.where(k % 2, 0x20, 0x02)           # E2M1 code 2 is 1.0
    else:
        xq = np.zeros((M, K), np.uint8)
        xq[np.arange(M), k] = 0x38                                       # E4M3 code 0x38 is 1.0
    y = multiply(xq, xs, wq, ws, [M], fmt, torch.float32).double().cpu().numpy()
    w = P.mxfp4_decode(wq[0], ws[0])
    f = np.ldexp(1.0, xs[np.arange(M), k // 32].astype(np.int64) - 127)
    assert np.array_equal(y, w.T[k] * f[:, None])


@pytest.mark.parametrize("M", [6, 400])
def test_packed_rows_are_the_unpacked_product(M):
    K, N, G, k = 512, 136, 5, 2
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    ids = torch.from_numpy(rng.integers(-1, G, (M, k)).astype(np.int32)).cuda()
    packed = torch.zeros((M * k, K + K // 32), dtype=torch.uint8, device="cuda")
    ends, src = torch.empty(G, dtype=torch.int32, device="cuda"), torch.empty(M * k, dtype=torch.int32, device="cuda")
    mxq.mxq_dispatch_pack_mx(x, ids, G, packed, ends, src, torch.empty(
        mxq.mxq_dispatch_pack_workspace_bytes(M, K, k, G), dtype=torch.uint8, device="cuda"))
    w = torch.from_numpy((0.05 * rng.standard_normal((G * N, K))).astype(np.float32)).to(torch.bfloat16).cuda()
    wq, ws = mxq.quantize_mxfp4(w, mxq.MXQ_SCALE_RCEIL)
    wq, ws = wq.view(G, N, -1), ws.view(G, N, -1)
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.empty((M * k, N), dtype=dtype, device="cuda")
        mxq.mxq_mxfp4_grouped_mm_packed(packed, wq, ws, ends, y)
        z = mxq.mxfp4_grouped_mm(packed[:, :K].contiguous(), packed[:, K:].contiguous(), wq, ws, ends, out_dtype=dtype)
        assert torch.equal(y, z)
        assert torch.all(y[int(ends[-1]):] == 0) and torch.any(y[:int(ends[-1])] != 0)


def test_product_many_groups():
    G, N, K = 1500, 8, 128
    rng = np.random.default_rng(4)
    sizes = rng.integers(0, 3, G)
    ends = np.cumsum(sizes).tolist()
    M = ends[-1] + 5
    check(*operands(M, N, K, G, mxq.MXQ_FMT_E2M1, 9), ends, mxq.MXQ_FMT_E2M1, torch.float32)


def test_product_more_tiles_than_one_launch_of_workgroups_lists():
    """Over 16384 output tiles of 256 x 256, sampled rows against the plain product."""
    M, N, K = 131072 + 77, 8192, 128
    ends = [70001, 70300, M - 3]
    wq = torch.randint(0, 256, (3, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.randint(122, 130, (3, N, K // 32), dtype=torch.uint8, device="cuda")
    xq = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda")
    xs = torch.randint(122, 130, (M, K // 32), dtype=torch.uint8, device="cuda")
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")
    y = mxq.mxfp4_grouped_mm(xq, xs, wq, ws, offs, mxq.MXQ_FMT_E2M1, out_dtype=torch.float32)
    assert torch.all(y[M - 3:] == 0)
    starts = [0] + ends[:-1]
    for g, (a, b) in enumerate(zip(starts, ends)):
        rows = sorted({a, a + 1, (a + b) // 2, b - 2, b - 1} | {a + (b - a) * i // 57 for i in range(57)})
        x = P.mxfp4_decode(xq[rows].cpu().numpy(), xs[rows].cpu().numpy())
        w = P.mxfp4_decode(wq[g].cpu().numpy(), ws[g].cpu().numpy())
        size = np.abs(x) @ np.abs(w).T
        assert np.all(np.abs(y[rows].double().cpu().numpy() - x @ w.T) <= K / 16 * 2.0 ** -24 * size)


def test_product_weights_past_two_to_the_31_bytes():
    """Weights of 2.7 GB: the last experts' rows, sampled columns, against the plain product."""
    G, N, K, M = 128, 8192, 5120, 24
    wq = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.randint(122, 130, (G, N, K // 32), dtype=torch.uint8, device="cuda")
    xq, xs, _, _ = operands(M, 8, K, 1, mxq.MXQ_FMT_E4M3, 3)
    ends = [0] * 100 + [8] * 26 + [16, 24]
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")
    y = mxq.mxfp4_grouped_mm(torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), wq, ws, offs,
                             out_dtype=torch.float32).double().cpu().numpy()
    x = P.mxfp8_decode(xq, xs)
    cols = [0, 1, 4095, 8191]
    for g, (a, b) in ((100, (0, 8)), (126, (8, 16)), (127, (16, 24))):
        w = P.mxfp4_decode(wq[g, cols].cpu().numpy(), ws[g, cols].cpu().numpy())
        size = np.abs(x[a:b]) @ np.abs(w).T
        assert np.all(np.abs(y[a:b][:, cols] - x[a:b] @ w.T) <= 2.0 ** -10 * size)


def test_product_repeats_and_other_stream():
    xq, xs, wq, ws = operands(300, 520, 640, 3, mxq.MXQ_FMT_E4M3, 2)
    a = multiply(xq, xs, wq, ws, [100, 101, 300], mxq.MXQ_FMT_E4M3, torch.float32)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = multiply(xq, xs, wq, ws, [100, 101, 300], mxq.MXQ_FMT_E4M3, torch.float32)
    assert torch.equal(a, b)


def test_empty_product():
    wq = torch.zeros((2, 16, 64), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((2, 16, 4), dtype=torch.uint8, device="cuda")
    x = torch.zeros((0, 128), dtype=torch.uint8, device="cuda")
    y = mxq.mxfp4_grouped_mm(x, torch.zeros((0, 4), dtype=torch.uint8, device="cuda"), wq, ws,
                             torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 16)
