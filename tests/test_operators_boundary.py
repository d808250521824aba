"""Argument checks of the norm, the routing and the MXFP4 entry points, on the host:
every call below fails validation or is a no-op, so nothing reaches a device."""
import pytest

from float8_quantization_moe_amd import mxq

NULL, SHAPE, ALIGN, WORKSPACE, DTYPE, RULE = 1, 2, 3, 5, 8, 9
A = 1 << 20


@pytest.fixture(scope="module")
def L():
    return mxq.lib()


def caller(f, names, **base):
    def call(**kw):
        args = dict(base, **kw)
        return f(*[args[n] for n in names.split()])
    return call


def test_add_rmsnorm(L):
    f = caller(L.mxq_add_rmsnorm, "x r w dt M K eps h y q s rstd st", x=A, r=A, w=A, dt=0, M=4, K=64, eps=1e-5, h=A, y=A,
               q=A, s=A, rstd=A, st=0)
    assert f(M=-1) == SHAPE and f(K=48) == SHAPE and f(K=16416) == SHAPE and f(M=1 << 36, K=64) == SHAPE
    assert f(K=20, q=0, s=0) == SHAPE and f(K=40) == SHAPE
    assert f(dt=2) == DTYPE and f(dt=-1) == DTYPE
    assert f(eps=-1e-6) == RULE and f(eps=float("nan")) == RULE
    assert f(x=0) == NULL and f(w=0) == NULL and f(y=0, q=0, s=0) == NULL
    assert f(q=0) == NULL and f(s=0) == NULL
    for p in ("x", "r", "w", "h", "y", "q", "s"):
        assert f(**{p: A + 8}) == ALIGN
    assert f(rstd=A + 2) == ALIGN
    assert f(M=0, x=0, w=0, y=0, q=0, s=0) == 0 and f(K=0) == 0


def test_add_rmsnorm_bwd(L):
    wb = L.mxq_add_rmsnorm_bwd_workspace_bytes
    need = wb(4, 64)
    assert need == 64 * 4 and wb(100000, 5120) == 512 * 5120 * 4
    assert wb(-1, 64) == 0 and wb(4, 60) == 0 and wb(4, 16392) == 0 and wb(0, 64) == 0
    f = caller(L.mxq_add_rmsnorm_bwd, "h w rstd dy dh dt M K dx dw ws wb st", h=A, w=A, rstd=A, dy=A, dh=A, dt=0, M=4,
               K=64, dx=A, dw=A, ws=A, wb=need, st=0)
    assert f(K=60) == SHAPE and f(M=-1) == SHAPE and f(dt=3) == DTYPE
    for p in ("h", "w", "rstd", "dy", "dx", "dw"):
        assert f(**{p: 0}) == NULL
    for p in ("h", "w", "dy", "dh", "dx", "dw", "ws"):
        assert f(**{p: A + 4}) == ALIGN
    assert f(rstd=A + 1) == ALIGN
    assert f(ws=0) == WORKSPACE and f(wb=need - 1) == WORKSPACE
    assert f(K=0) == 0


def test_route_topk(L):
    f = caller(L.mxq_route_topk, "l dt M E b sc ng kg k fl scale ids w st", l=A, dt=1, M=4, E=64, b=A, sc=1, ng=8, kg=4, k=8,
               fl=3, scale=1.0, ids=A, w=A, st=0)
    assert f(M=-1) == SHAPE and f(E=0) == SHAPE and f(E=1025) == SHAPE and f(E=1032, ng=8) == SHAPE
    assert f(k=0) == SHAPE and f(k=65) == SHAPE and f(E=4, ng=1, kg=1, k=5) == SHAPE
    assert f(ng=0) == SHAPE and f(ng=7) == SHAPE and f(kg=0) == SHAPE and f(kg=9) == SHAPE
    assert f(kg=1, k=9) == SHAPE                                  # one group of 8 cannot fill 9 slots
    assert f(dt=2) == DTYPE and f(sc=2) == RULE and f(fl=4) == RULE and f(fl=-1) == RULE
    assert f(l=0) == NULL and f(ids=0) == NULL and f(w=0) == NULL
    assert f(l=A + 8) == ALIGN and f(b=A + 2) == ALIGN and f(ids=A + 1) == ALIGN and f(w=A + 2) == ALIGN
    assert f(M=0, l=0, ids=0, w=0) == 0


def test_route_topk_bwd(L):
    f = caller(L.mxq_route_topk_bwd, "l dt M E sc ids k fl scale dw dl st", l=A, dt=0, M=4, E=64, sc=0, ids=A, k=8, fl=1,
               scale=1.0, dw=A, dl=A, st=0)
    assert f(E=2000) == SHAPE and f(k=65) == SHAPE and f(M=-5) == SHAPE
    assert f(dt=5) == DTYPE and f(sc=-1) == RULE and f(fl=2) == RULE
    for p in ("l", "ids", "dw", "dl"):
        assert f(**{p: 0}) == NULL
        assert f(**{p: A + 2}) == ALIGN
    assert f(M=0, l=0, ids=0, dw=0, dl=0) == 0


def test_mxfp4_codec(L):
    q = caller(L.mxq_quantize_mxfp4, "x M K rule q s st", x=A, M=4, K=64, rule=0, q=A, s=A, st=0)
    assert q(K=48) == SHAPE and q(M=-1) == SHAPE and q(rule=2) == RULE and q(rule=-1) == RULE
    for p in ("x", "q", "s"):
        assert q(**{p: 0}) == NULL and q(**{p: A + 8}) == ALIGN
    assert q(M=0, x=0, q=0, s=0) == 0 and q(K=0) == 0 and q(M=0, rule=5) == RULE
    d = caller(L.mxq_dequantize_mxfp4, "q s M K y st", q=A, s=A, M=4, K=64, y=A, st=0)
    assert d(K=33) == SHAPE and d(M=1 << 36, K=64) == SHAPE
    for p in ("q", "s", "y"):
        assert d(**{p: 0}) == NULL and d(**{p: A + 4}) == ALIGN
    assert d(M=0, q=0, s=0, y=0) == 0


def test_mxfp4_grouped_mm(L):
    f = caller(L.mxq_mxfp4_grouped_mm, "xq xs fmt wq ws offs M N K G dt y st", xq=A, xs=A, fmt=0, wq=A, ws=A, offs=A,
               M=700, N=264, K=1024, G=5, dt=0, y=A, st=0)
    assert f(K=64) == SHAPE and f(N=4) == SHAPE and f(M=-1) == SHAPE and f(G=0) == SHAPE and f(K=1 << 24) == SHAPE
    assert f(K=1000) == SHAPE and f(N=260) == SHAPE and f(G=4096) == SHAPE and f(M=1 << 31) == SHAPE and f(K=0) == SHAPE
    assert f(fmt=2) == DTYPE and f(dt=2) == DTYPE
    for p in ("xq", "xs", "wq", "ws", "offs", "y"):
        assert f(**{p: 0}) == NULL
        assert f(**{p: A + 2}) == ALIGN
    assert f(M=0, xq=0, y=0) == 0 and f(N=0, wq=0, y=0) == 0
    g = caller(L.mxq_mxfp4_grouped_mm_packed, "p wq ws offs M N K G dt y st", p=A, wq=A, ws=A, offs=A, M=700, N=264,
               K=1024, G=5, dt=0, y=A, st=0)
    assert g(K=1152) == SHAPE and g(dt=7) == DTYPE and g(p=0) == NULL and g(p=A + 8) == ALIGN
    assert g(offs=A + 1) == ALIGN and g(M=0, p=0, y=0) == 0


def test_binding_refuses_what_is_not_a_dense_device_tensor():
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mxq.add_rmsnorm(x, None, w, 1e-5)
    with pytest.raises(TypeError):
        mxq.mxq_add_rmsnorm(x.to(torch.float16), None, w, 1e-5)
    with pytest.raises(ValueError):
        mxq.route_topk(torch.zeros((4, 8)), 2)
    with pytest.raises(TypeError):
        mxq.route_topk(torch.zeros((4, 8), dtype=torch.float64), 2)
    with pytest.raises(KeyError):
        mxq.route_topk(torch.zeros((4, 8)), 2, score="relu")
    with pytest.raises(ValueError):
        mxq.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        mxq.mxfp4_grouped_mm(torch.zeros((4, 100), dtype=torch.uint8), x, torch.zeros((1, 8, 64), dtype=torch.uint8), x, x)
