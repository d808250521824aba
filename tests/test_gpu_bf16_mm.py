"""Grouped products in bf16 (the rows' product and the gradients of rows and weights) against the
64-bit products.

Small integers are exact: with values of at most 4 in size and up to 2^15 terms every partial sum
is a whole number below 2^19, so an fp32 result has to be equal and a bf16 one the nearest to it,
whatever the order.  For other values the products of two bf16 are exact in fp32, and the matrix
cores add 16 of them at a time to an fp32 sum: a chain of depth / 16 adds, and 18 terms aligned in
each, good to 2^-23 of the sum of magnitudes each (2^-23 and not 2^-24: they may cut off)."""
import numpy as np
import pytest
import torch

import gpu_util as U
import plain64 as P
import plain64_training as T
from float8_quantization_moe_amd import mxq, training

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PRODUCTS = {"y": mxq.MXQ_PRODUCT_Y, "dx": mxq.MXQ_PRODUCT_DX, "dw": mxq.MXQ_PRODUCT_DW}


def f64(t):
    return t.double().cpu().numpy()


def ints(shape, g):
    return torch.randint(-4, 5, shape, generator=g, device="cuda").to(torch.bfloat16)


def operands(M, N, K, G, seed, make=ints):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"x": make((M, K), g), "dy": make((M, N), g), "w": make((G, N, K), g)}


def shape_of(product, M, N, K, G):
    return {"y": (M, N), "dx": (M, K), "dw": (G, N, K)}[product]


def call(product, t, ends, out, ws, accumulate=False):
    if product == "y":
        mxq.mxq_bf16_grouped_mm(t["x"], t["w"], ends, out, ws)
    elif product == "dx":
        mxq.mxq_bf16_grouped_mm_dx(t["dy"], t["w"], ends, out, ws)
    else:
        mxq.mxq_bf16_grouped_mm_dw(t["dy"], t["x"], ends, out, accumulate, ws)


def want_of(product, t, ends, M):
    """(exact product, sum of magnitudes) in doubles on the device."""
    spans = P.group_spans(ends, M)
    d = {k: v.double() for k, v in t.items()}
    G, N, K = t["w"].shape
    out = torch.zeros(shape_of(product, M, N, K, G), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    for g, (a, b) in enumerate(spans):
        if a == b:
            continue
        for o, f in ((out, lambda v: v), (size, torch.abs)):
            if product == "y":
                o[a:b] = f(d["x"][a:b]) @ f(d["w"][g]).t().contiguous()
            elif product == "dx":
                o[a:b] = f(d["dy"][a:b]) @ f(d["w"][g])
            else:
                o[g] = f(d["dy"][a:b]).t().contiguous() @ f(d["x"][a:b])
    return out, size


def run(product, t, ends, out_dtype, M):
    """The product into a guarded buffer, with exactly the workspace it asks for."""
    G, N, K = t["w"].shape
    shape = shape_of(product, M, N, K, G)
    n = int(np.prod(shape))
    dt = DT[out_dtype]
    z = 2 if out_dtype == "bf16" else 4
    out = U.Guarded(n * z, torch.uint8, (n * z,))
    need = mxq.mxq_bf16_grouped_mm_workspace_bytes(PRODUCTS[product], M, N, K, G)
    ws = U.Guarded(need, torch.uint8, (need,)) if need else None
    call(product, t, torch.tensor(ends, dtype=torch.int32, device="cuda"), out.t.view(dt).view(shape), None if ws is None else ws.t)
    torch.cuda.synchronize()
    assert out.guard_intact() and (ws is None or ws.guard_intact())
    return out.t.view(dt).view(shape)


# M, N, K, ends
CASES = [
    (1, 8, 8, [1]),
    (1, 264, 72, [0, 1, 1]),
    (3, 40, 136, [3]),
    (8, 512, 1024, [1, 1, 2, 3, 3, 7, 8]),
    (16, 8, 2056, [16]),
    (33, 1032, 8, [5, 33]),
    (65, 256, 64, [65]),
    (200, 264, 200, [64, 130, 130, 199]),                  # a row past the last end
    (256, 256, 256, [256]),
    (257, 520, 328, [257]),
    (300, 328, 520, [-3, 40, 20, 260, 900]),               # ends out of order and past M
    (500, 72, 448, [0, 0, 0, 0]),                          # no group has rows
    (777, 1736, 1408, [100, 164, 228, 293, 293, 400, 401, 420, 500, 510, 600, 650, 700, 750, 776, 777]),
    (1000, 136, 264, list(range(3, 1000, 7))),             # 143 small groups
    (2000, 264, 520, [1500, 2000]),
    (4100, 32, 48, [4100]),                                # few tiles, a long sum for dw
    (700, 2048, 8, [699]),
    (130, 8200, 24, [65, 130]),
    (64, 24, 8200, [10, 64]),
    (40, 136, 8200, [9, 33]),                              # few workgroups, long sums: in parts
    (70, 8200, 72, [70]),
    (7000, 72, 200, [700 * i for i in range(1, 8)] + [5000, 7000]),   # dW: few results
    (1500, 200, 328, [0, 1400, 1400, 1490]),
    # rows enough for tiles (the smaller ones above go to the kernel for few rows)
    (600, 264, 16392, [120, 250]),                         # few tiles, a long sum: in parts
    (600, 16392, 264, [3, 290, 290]),
    (1100, 1032, 1288, [300, 300, 301, 560, 577, 1099]),
    (1100, 1288, 1032, [64, 129, 1000]),
    (5000, 520, 456, [1300, 1300, 2600, 2601, 4990]),
    (20000, 264, 264, [300 * i for i in range(1, 66)]),    # 65 groups, their last tiles of 44 rows
    (300, 2696, 2696, [0, 300]),
    (1100, 1032, 1288, [0, 0, -5]),                        # no group has rows, nor is the matrix small
    (20000, 264, 264, [5 * i for i in range(4094)] + [19999]),        # 4095 groups of 5 rows, -1 empty
    (66000, 8192, 72, [1000 * i for i in range(1, 65)] + [66000]),    # two workgroups' lists a CU
]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("product", ["y", "dx", "dw"])
@pytest.mark.parametrize("M,N,K,ends", CASES, ids=[f"{c[0]}x{c[1]}x{c[2]}g{len(c[3])}" for c in CASES])
def test_integers_are_exact(M, N, K, ends, product, out):
    t = operands(M, N, K, len(ends), M + N + K)
    want, _ = want_of(product, t, ends, M)
    got = run(product, t, ends, out, M)
    assert torch.equal(got.double(), want.to(DT[out]).double())


@pytest.mark.parametrize("product", ["y", "dx", "dw"])
@pytest.mark.parametrize("M,N,K,ends", [c for c in CASES if c[0] in (8, 200, 257, 600, 777, 1100, 2000, 4100)],
                         ids=lambda v: str(v) if isinstance(v, int) else f"g{len(v)}")
def test_real_values(M, N, K, ends, product):
    def make(shape, g):
        return (torch.randn(shape, generator=g, device="cuda") * torch.exp(torch.randn((shape[0],) + (1,) * (len(shape) - 1), generator=g, device="cuda"))).to(torch.bfloat16)
    t = operands(M, N, K, len(ends), 5, make)
    want, size = want_of(product, t, ends, M)
    depth = {"y": K, "dx": N, "dw": M}[product]
    bound = (depth / 16 + 18) * 2.0 ** -23 * size
    for out in ("f32", "bf16"):
        got = run(product, t, ends, out, M)
        half = torch.from_numpy(P.half_step(f64(want), out) * np.ones(want.shape)).cuda()
        assert torch.all((got.double() - want).abs() <= half + bound)
        assert torch.equal(got, run(product, t, ends, out, M))         # the same bits again


@pytest.mark.parametrize("M,N,K,ends", [(300, 264, 200, [100, 100, 250]), (4100, 32, 48, [4000]), (5, 512, 520, [5]), (900, 1032, 1160, [300, 300, 890]),
                                         (20000, 264, 264, [20000])])
def test_gradient_added_to_what_is_there(M, N, K, ends):
    t = operands(M, N, K, len(ends), 3)
    want, _ = want_of("dw", t, ends, M)
    dw = torch.randint(-100, 100, want.shape, device="cuda").float()
    before = dw.clone()
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    got = training.bf16_grouped_mm_dw(t["dy"], t["x"], e, dw=dw)
    assert got is dw and torch.equal(dw.double(), before.double() + want)
    none = torch.zeros_like(e)                             # no group has rows: nothing changes
    before = dw.clone()
    training.bf16_grouped_mm_dw(t["dy"], t["x"], none, dw=dw)
    assert torch.equal(dw, before)


@pytest.mark.parametrize("M,N,K,ends", [(200, 264, 200, [64, 130, 130, 190]), (40, 72, 136, [17, 39]), (1100, 1032, 1288, [300, 600, 1090])])
def test_nan_and_infinity_reach_their_own_sums_only(M, N, K, ends):
    base = operands(M, N, K, len(ends), 1)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    last, second = ends[-1], ends[0]
    for bad in (float("nan"), float("inf")):
        t = {k: v.clone() for k, v in base.items()}
        t["x"][3, K - 1] = bad
        t["x"][last:] = bad                                # rows of no group
        t["dy"][last:] = bad
        t["w"][1, N - 1, 0] = bad
        clean = {k: torch.nan_to_num(v, nan=0.0, posinf=0.0) for k, v in t.items()}
        y = run("y", t, ends, "f32", M)
        wy, _ = want_of("y", clean, ends, M)
        dirty = torch.zeros_like(y, dtype=torch.bool)
        dirty[3] = True                                    # 3 < ends[0]: the row's every sum
        dirty[second:ends[1], N - 1] = True                # group 1's rows, the last column
        assert torch.equal(y[~dirty].double(), wy[~dirty])
        assert not torch.isfinite(y[3]).any() or bad == float("inf")
        assert torch.all(y[last:] == 0)
        dx = run("dx", t, ends, "f32", M)
        wd, _ = want_of("dx", clean, ends, M)
        dirty = torch.zeros_like(dx, dtype=torch.bool)
        dirty[second:ends[1], 0] = True
        assert torch.equal(dx[~dirty].double(), wd[~dirty]) and torch.all(dx[last:] == 0)
        dw = run("dw", t, ends, "f32", M)
        ww, _ = want_of("dw", clean, ends, M)
        dirty = torch.zeros_like(dw, dtype=torch.bool)
        dirty[0, :, K - 1] = True
        assert torch.equal(dw[~dirty].double(), ww[~dirty])
        if bad != bad:
            assert torch.isnan(dw[0, :, K - 1]).all() and torch.isnan(y[second:ends[1], N - 1]).all()


@pytest.mark.parametrize("product", ["y", "dx", "dw"])
def test_a_layer_of_a_rank(product):
    """The (16640, 5120) tokens of a rank against 16 experts of 8192: every value in integers."""
    M, N, K, G = 16640, 8192, 5120, 16
    sizes = [4000, 1, 0, 2500, 1250, 900, 700, 3000, 64, 600, 500, 425, 800, 300, 700, 892]
    ends = np.cumsum(sizes).tolist()
    t = operands(M, N, K, G, 11)
    want, _ = want_of(product, t, ends, M)
    got = run(product, t, ends, "f32" if product == "dw" else "bf16", M)
    assert torch.equal(got.double(), want.to(got.dtype).double())


def test_no_rows():
    w = torch.ones((3, 16, 24), dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, dy = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    assert training.bf16_grouped_mm(x, w, e).shape == (0, 16)
    assert training.bf16_grouped_mm_dx(dy, w, e).shape == (0, 24)
    assert torch.all(training.bf16_grouped_mm_dw(dy, x, e) == 0)
    dw = torch.full((3, 16, 24), 2.0, device="cuda")
    assert torch.all(training.bf16_grouped_mm_dw(dy, x, e, dw=dw) == 2.0)


@pytest.mark.parametrize("product", ["y", "dx", "dw"])
def test_results_past_two_to_the_31_elements(product):
    """Ones times a pattern: the result's rows repeat, so the far ones are known."""
    if product == "dw":
        M, N, K, G = 64, 8192, 8192, 33                    # 2.2e9 results
    else:
        M, N, K, G = 262400, 8192 if product == "y" else 64, 64 if product == "y" else 8192, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    ends = [M // G * (i + 1) for i in range(G)]
    ends[-1] = M
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    one = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    if product == "dw":
        row = ints((1, K), g)
        dw = training.bf16_grouped_mm_dw(one(M, N), row.expand(M, K).contiguous(), e, out_dtype=torch.bfloat16)
        for grp, n in ((0, 0), (31, 8191), (32, 0), (32, 8191)):
            rows = ends[grp] - (ends[grp - 1] if grp else 0)
            assert torch.equal(dw[grp, n].float(), (rows * row[0].float()).to(torch.bfloat16).float())
        return
    w = ints((G, N, K), g)
    if product == "y":
        out, want = training.bf16_grouped_mm(one(M, K), w, e), w.float().sum(2)
    else:
        out, want = training.bf16_grouped_mm_dx(one(M, N), w, e), w.float().sum(1)
    for m in (0, ends[0] - 1, ends[0], 262143, 262144, M - 1):
        assert torch.equal(out[m].float(), want[0 if m < ends[0] else 1].to(torch.bfloat16).float())
