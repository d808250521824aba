"""The helpers given a stream: their outputs and workspaces are that stream's memory, so
neither a block that the current stream still uses nor one that it takes meanwhile is theirs."""
import pytest
import torch

import gpu_util as U  # noqa: F401
from float8_quantization_moe_amd import mxq

pytestmark = pytest.mark.gpu

M, K, N, E = 640, 512, 256, 8


def inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    t = {}
    t["x"], t["r"], t["dy"] = (torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    t["w"] = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    t["ends"] = torch.tensor([100, 101, 101, 230, 400, 410, 600, M], dtype=torch.int32, device="cuda")
    t["q"], t["s"] = mxq.quantize_mx(t["x"])
    t["q4"], t["s4"] = mxq.quantize_mxfp4(t["x"])
    big = torch.randn((E * N, K), generator=g, device="cuda").to(torch.bfloat16)
    t["w8"], t["ws8"] = (v.view(E, N, -1) for v in mxq.quantize_mx(big))
    t["w4"], t["ws4"] = (v.view(E, N, -1) for v in mxq.quantize_mxfp4(big))
    t["h"], _, _, _, t["rstd"] = mxq.add_rmsnorm(t["x"], t["r"], t["w"], 1e-5)
    t["l"] = torch.randn((M, 64), generator=g, device="cuda")
    t["ids"], t["dw"] = mxq.route_topk(t["l"], 4)
    torch.cuda.synchronize()
    return t


HELPERS = {
    "quantize_mx": lambda t, **kw: mxq.quantize_mx(t["x"], **kw),
    "dequantize_mx": lambda t, **kw: mxq.dequantize_mx(t["q"], t["s"], **kw),
    "group_scale_fp8": lambda t, **kw: mxq.group_scale_fp8(t["x"], t["ends"], **kw),
    "transpose_u8": lambda t, **kw: mxq.transpose_u8(t["q"], **kw),
    "scaled_grouped_mm": lambda t, **kw: mxq.scaled_grouped_mm(t["q"], t["s"], t["w8"], t["ws8"], t["ends"], **kw),
    "add_rmsnorm": lambda t, **kw: mxq.add_rmsnorm(t["x"], t["r"], t["w"], 1e-5, **kw),
    "add_rmsnorm_bwd": lambda t, **kw: mxq.add_rmsnorm_bwd(t["h"], t["w"], t["rstd"], t["dy"], t["x"], **kw),
    "route_topk": lambda t, **kw: mxq.route_topk(t["l"], 4, **kw),
    "route_topk_bwd": lambda t, **kw: mxq.route_topk_bwd(t["l"], t["ids"], t["dw"], **kw),
    "quantize_mxfp4": lambda t, **kw: mxq.quantize_mxfp4(t["x"], **kw),
    "dequantize_mxfp4": lambda t, **kw: mxq.dequantize_mxfp4(t["q4"], t["s4"], **kw),
    "mxfp4_grouped_mm": lambda t, **kw: mxq.mxfp4_grouped_mm(t["q4"], t["s4"], t["w4"], t["ws4"], t["ends"],
                                                            x_format=mxq.MXQ_FMT_E2M1, **kw),
}


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", HELPERS)
def test_outputs_on_another_stream(name, as_handle):
    t, f = inputs(), HELPERS[name]
    st = torch.cuda.Stream()
    given = st.cuda_stream if as_handle else st
    want = tensors(f(t))
    torch.cuda.synchronize()
    got = tensors(f(t, stream=given))
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.cuda.current_stream() != st
    # blocks that the current stream has freed are not taken for the other stream
    shapes = [(v.shape, v.dtype) for v in want]
    mine = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
    torch.cuda.synchronize()
    freed = {v.data_ptr() for v in mine} | {v.data_ptr() for v in want}
    del mine, want, got
    outs = tensors(f(t, stream=given))
    assert not freed & {v.data_ptr() for v in outs}
    torch.cuda.synchronize()


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", HELPERS)
def test_dropped_outputs_and_workspaces_are_not_handed_out_early(name, as_handle):
    t, f = inputs(), HELPERS[name]
    st = torch.cuda.Stream()
    sizes = [v.numel() * v.element_size() for v in tensors(f(t))]
    sizes += [mxq.mxq_add_rmsnorm_bwd_workspace_bytes(M, K), mxq.mxq_grouped_mm_workspace_bytes(M, N, K, E),
              mxq.mxq_group_scale_workspace_bytes(M, K, E)]
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)                       # a bounded spin: the helper's kernels come after it
    f(t, stream=st.cuda_stream if as_handle else st)        # (outputs dropped at once)
    held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((v == 255).all()) for v in held)


def test_the_null_handle_is_the_default_stream():
    t = inputs()
    want = mxq.quantize_mx(t["x"])
    got = mxq.quantize_mx(t["x"], stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
