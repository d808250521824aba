"""NaN and infinities in the grouped products in bf16: which sums they reach, and as what.

The operands are small whole numbers, zeros among them, with a NaN or an infinity here and there, so each
result that meets one is NaN or an infinity whatever the order of its sum: an infinity times 0 is NaN, times
another number an infinity of the product's sign, and infinities of both signs sum to NaN.  What a result has
to be is taken from its terms in doubles.  All other results are exact (partial sums are whole numbers below
2^19)."""
import numpy as np
import pytest
import torch

import plain64 as P
from float8_quantization_moe_amd import training

pytestmark = pytest.mark.gpu

BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": -float("inf")}
# few rows; few columns and rows; many rows (tiles of 128 and 256)
SHAPES = [(40, 72, 136, [17, 39]), (200, 264, 200, [64, 130, 130, 190]), (1100, 1032, 1288, [300, 600, 1090]),
          (5000, 520, 456, [1300, 1300, 2600, 4990])]


def sums(terms):
    """Sums over the last axis, NaN and infinities as IEEE has them (plain additions, no library product)."""
    with np.errstate(invalid="ignore"):
        return np.add.reduce(terms, axis=-1)


def products(a, b):
    with np.errstate(invalid="ignore"):
        return a * b


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("M,N,K,ends", SHAPES, ids=[f"{c[0]}x{c[1]}x{c[2]}" for c in SHAPES])
def test_nan_and_infinities(M, N, K, ends, bad):
    rng = np.random.default_rng(M)
    G, v = len(ends), BAD[bad]
    x, dy, w = (rng.integers(-4, 5, s).astype(np.float64) for s in ((M, K), (M, N), (G, N, K)))
    last, second = ends[-1], ends[1] if ends[1] > ends[0] else ends[2]
    g2 = 1 if ends[1] > ends[0] else 2                     # the second group with rows
    clean = x.copy(), dy.copy(), w.copy()
    x[3, K - 1] = v                                        # a row of group 0
    dy[5, 2] = v
    w[g2, N - 1, 0] = v
    x[last:], dy[last:] = v, v                             # rows of no group: they reach nothing
    clean[0][last:], clean[1][last:] = 0, 0
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    tx, tdy, tw = (torch.from_numpy(t).to(torch.bfloat16).cuda() for t in (x, dy, w))
    rows0, rows2 = slice(0, ends[0]), slice(ends[g2 - 1], second)
    spans = P.group_spans(ends, M)

    want = np.zeros((M, N))
    for g, (a, b) in enumerate(spans):
        want[a:b] = clean[0][a:b] @ clean[2][g].T
    want[3] = sums(products(w[0], x[3]))
    want[rows2, N - 1] = sums(products(x[rows2], w[g2, N - 1]))
    assert not np.isfinite(want[3]).any() and not np.isfinite(want[rows2, N - 1]).any()
    for dt in (torch.float32, torch.bfloat16):
        assert same(training.bf16_grouped_mm(tx, tw, e, out_dtype=dt).double().cpu().numpy(),
                    torch.from_numpy(want).to(dt).double().numpy())

    want = np.zeros((M, K))
    for g, (a, b) in enumerate(spans):
        want[a:b] = clean[1][a:b] @ clean[2][g]
    want[5] = sums(products(w[0].T, dy[5]))
    want[rows2, 0] = sums(products(dy[rows2], w[g2, :, 0]))
    assert not np.isfinite(want[5]).any() and not np.isfinite(want[rows2, 0]).any()
    for dt in (torch.float32, torch.bfloat16):
        assert same(training.bf16_grouped_mm_dx(tdy, tw, e, out_dtype=dt).double().cpu().numpy(),
                    torch.from_numpy(want).to(dt).double().numpy())

    want = np.zeros((G, N, K))
    for g, (a, b) in enumerate(spans):
        want[g] = clean[1][a:b].T @ clean[0][a:b]
    want[0, :, K - 1] = sums(products(dy[rows0].T, x[rows0, K - 1]))
    want[0, 2, :] = sums(products(x[rows0].T, dy[rows0, 2]))
    assert not np.isfinite(want[0, :, K - 1]).any() and not np.isfinite(want[0, 2]).any()
    for dt in (torch.float32, torch.bfloat16):
        assert same(training.bf16_grouped_mm_dw(tdy, tx, e, out_dtype=dt).double().cpu().numpy(),
                    torch.from_numpy(want).to(dt).double().numpy())
    # added to a gradient that is there
    dw = torch.from_numpy(rng.integers(-50, 50, want.shape).astype(np.float32))
    with np.errstate(invalid="ignore"):
        total = want + dw.double().numpy()
    assert same(training.bf16_grouped_mm_dw(tdy, tx, e, dw=dw.cuda()).double().cpu().numpy(), total)
