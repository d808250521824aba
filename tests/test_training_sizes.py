"""Workspace sizes of the bf16 products (no GPU is needed)."""
import pytest

from float8_quantization_moe_amd import mxq

Y, DX, DW = mxq.MXQ_PRODUCT_Y, mxq.MXQ_PRODUCT_DX, mxq.MXQ_PRODUCT_DW


def size(*a):
    return mxq.mxq_bf16_grouped_mm_workspace_bytes(*a)


@pytest.mark.parametrize("M,N,K,G", [(1, 64, 64, 1), (2048, 64, 64, 1), (4096, 64, 128, 2), (8192, 8, 8, 4), (8192, 64, 128, 64), (777, 240, 600, 1),
                                     (4000, 512, 512, 8)])
def test_small_weight_gradients_need_none(M, N, K, G):
    """Their sums are at most 2048 rows a group on average, which four waves of a workgroup share."""
    assert size(DW, M, N, K, G) == 0


def test_split_sums_ask_for_their_parts():
    # 3 x 9 workgroups, 101 steps of the sum: parts of three steps a wave, 101 // 12
    assert size(DX, 142, 6416, 552, 1) == 8 * 142 * 552 * 4
    n = size(DW, 16000, 64, 64, 1)                                              # one tile: its sum in parts
    assert n > 0 and n % (64 * 64 * 4) == 0


@pytest.mark.parametrize("product", [-1, 3, 1 << 30])
def test_an_unknown_product_has_no_size(product):
    assert size(product, 142, 6416, 552, 1) == 0
