"""Argument checks of the training step's entry points, and the helpers' streams, on the host:
every library call below fails validation, is a no-op, or is recorded and not made."""
import pytest
import torch

from float8_quantization_moe_amd import mxq, training
from test_helper_streams import Recorder, bf, i32

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


def test_add_layernorm(L):
    f = caller(L.mxq_add_layernorm, "x r w b dt M K eps h y q s mean rstd st", x=A, r=A, w=A, b=A, dt=0, M=4, K=64, eps=1e-5,
               h=A, y=A, q=A, s=A, mean=A, rstd=A, st=0)
    assert f(M=-1) == SHAPE and f(K=48) == SHAPE and f(K=16416) == SHAPE and f(M=1 << 36, K=64) == SHAPE
    assert f(K=20, q=0, s=0) == SHAPE and f(dt=2) == DTYPE and f(dt=-1) == DTYPE
    assert f(eps=-1e-6) == RULE and f(eps=float("nan")) == RULE
    assert f(x=0) == NULL and f(w=0) == NULL and f(y=0, q=0, s=0) == NULL and f(q=0) == NULL and f(s=0) == NULL
    for p in ("x", "r", "w", "b", "h", "y", "q", "s"):
        assert f(**{p: A + 8}) == ALIGN
    assert f(rstd=A + 2) == ALIGN and f(mean=A + 1) == ALIGN
    assert f(M=0, x=0, w=0, y=0, q=0, s=0) == 0 and f(K=0) == 0


def test_add_layernorm_bwd(L):
    wb = L.mxq_add_layernorm_bwd_workspace_bytes
    need = wb(4, 64)
    assert need == 64 * 8 and wb(100000, 5120) == 512 * 5120 * 8
    assert wb(-1, 64) == 0 and wb(4, 60) == 0 and wb(4, 16392) == 0 and wb(0, 64) == 0
    f = caller(L.mxq_add_layernorm_bwd, "h w mean rstd dy dh dt M K dx dw db ws wb st", h=A, w=A, mean=A, rstd=A, dy=A, dh=A,
               dt=0, M=4, K=64, dx=A, dw=A, db=A, ws=A, wb=need, st=0)
    assert f(K=60) == SHAPE and f(M=-1) == SHAPE and f(dt=3) == DTYPE
    for p in ("h", "w", "mean", "rstd", "dy", "dx", "dw"):
        assert f(**{p: 0}) == NULL
    for p in ("h", "w", "dy", "dh", "dx", "dw", "db", "ws"):
        assert f(**{p: A + 4}) == ALIGN
    assert f(rstd=A + 1) == ALIGN and f(mean=A + 2) == ALIGN
    assert f(ws=0) == WORKSPACE and f(wb=need - 1) == WORKSPACE and f(K=0) == 0


def test_dispatch_rows(L):
    wb = L.mxq_dispatch_rows_workspace_bytes
    need = wb(700, 2, 16)
    assert need == 6 * 16 * 4 and wb(0, 2, 16) == 64 and wb(4, 65, 16) == 0 and wb(4, 2, 0) == 0 and wb(-1, 2, 16) == 0
    f = caller(L.mxq_dispatch_rows, "x dt M K ids k E rows ends src place ws wb st", x=A, dt=0, M=700, K=264, ids=A, k=2, E=16,
               rows=A, ends=A, src=A, place=A, ws=A, wb=need, st=0)
    assert f(K=4) == SHAPE and f(K=0) == SHAPE and f(K=(1 << 23) + 8) == SHAPE and f(M=-1) == SHAPE
    assert f(k=0) == SHAPE and f(k=65) == SHAPE and f(E=0) == SHAPE and f(E=1025) == SHAPE and f(M=1 << 30) == SHAPE
    assert f(M=1 << 31, k=1) == SHAPE and f(M=1 << 24, K=1 << 16, k=2) == SHAPE
    assert f(dt=2) == DTYPE
    for p in ("x", "ids", "rows", "ends", "src", "place"):
        assert f(**{p: 0}) == NULL and f(**{p: A + 2}) == ALIGN
    assert f(x=A + 8) == ALIGN and f(rows=A + 8) == ALIGN and f(ws=A + 4) == ALIGN
    assert f(ws=0) == WORKSPACE and f(wb=need - 1) == WORKSPACE


def test_pair_rows(L):
    f = caller(L.mxq_pair_rows, "src n place st", src=A, n=10, place=A, st=0)
    assert f(n=-1) == SHAPE and f(n=1 << 31) == SHAPE and f(src=0) == NULL and f(place=0) == NULL
    assert f(src=A + 2) == ALIGN and f(place=A + 1) == ALIGN and f(n=0, src=0, place=0) == 0


def test_combine_rows(L):
    f = caller(L.mxq_combine_rows, "rows dt R K place M k w out st", rows=A, dt=1, R=9, K=40, place=A, M=4, k=2, w=A, out=A, st=0)
    assert f(K=20) == SHAPE and f(K=(1 << 23) + 8) == SHAPE and f(R=-1) == SHAPE and f(R=1 << 31) == SHAPE and f(M=-1) == SHAPE
    assert f(k=0) == SHAPE and f(k=65) == SHAPE and f(M=1 << 31) == SHAPE and f(R=1 << 30, K=1 << 20) == SHAPE
    assert f(dt=-1) == DTYPE
    for p in ("rows", "place", "out"):
        assert f(**{p: 0}) == NULL and f(**{p: A + 2}) == ALIGN
    assert f(w=A + 2) == ALIGN and f(M=0, rows=0, place=0, out=0) == 0 and f(K=0, rows=0, out=0) == 0


def test_combine_rows_bwd(L):
    f = caller(L.mxq_combine_rows_bwd, "dout rows dt R K place M k w drows dw st", dout=A, rows=A, dt=0, R=9, K=40, place=A, M=4,
               k=2, w=A, drows=A, dw=A, st=0)
    assert f(K=20) == SHAPE and f(R=-1) == SHAPE and f(k=0) == SHAPE and f(dt=2) == DTYPE
    for p in ("dout", "rows", "place", "drows"):
        assert f(**{p: 0}) == NULL and f(**{p: A + 2}) == ALIGN
    assert f(w=A + 2) == ALIGN and f(dw=A + 1) == ALIGN
    assert f(M=0, dout=0, rows=0, place=0, drows=0, dw=0) == 0 and f(K=0, dw=0, dout=0, rows=0, drows=0) == 0


def test_bf16_grouped_mm(L):
    wb = L.mxq_bf16_grouped_mm_workspace_bytes
    assert wb(3, 64, 64, 64, 2) == 0 and wb(-1, 64, 64, 64, 2) == 0 and wb(0, 64, 60, 64, 2) == 0 and wb(2, 64, 64, 64, 0) == 0
    big = 1 << 40
    f = caller(L.mxq_bf16_grouped_mm, "x w offs M N K G dt y ws wb st", x=A, w=A, offs=A, M=70, N=264, K=1024, G=5, dt=0, y=A,
               ws=A, wb=big, st=0)
    g = caller(L.mxq_bf16_grouped_mm_dx, "x w offs M N K G dt y ws wb st", x=A, w=A, offs=A, M=70, N=264, K=1024, G=5, dt=0, y=A,
               ws=A, wb=big, st=0)
    h = caller(L.mxq_bf16_grouped_mm_dw, "x w offs M N K G dt acc y ws wb st", x=A, w=A, offs=A, M=70, N=264, K=1024, G=5, dt=1,
               acc=0, y=A, ws=A, wb=big, st=0)
    for c in (f, g, h):
        assert c(K=0) == SHAPE and c(N=0) == SHAPE and c(K=1028) == SHAPE and c(N=260) == SHAPE and c(M=-1) == SHAPE
        assert c(G=0) == SHAPE and c(G=4096) == SHAPE and c(K=(1 << 20) + 8) == SHAPE and c(N=(1 << 20) + 8) == SHAPE
        assert c(M=1 << 31) == SHAPE and c(N=1 << 20, K=1 << 20, G=2) == SHAPE
        assert c(dt=2) == DTYPE and c(dt=-1) == DTYPE
        for p in ("x", "w", "offs", "y"):
            assert c(**{p: 0}) == NULL and c(**{p: A + 2}) == ALIGN
        assert c(x=A + 8) == ALIGN and c(ws=A + 4) == ALIGN
    assert f(M=0, x=0, y=0) == 0 and g(M=0, x=0, y=0) == 0
    assert h(acc=2) == RULE and h(acc=-1) == RULE and h(acc=1, dt=0) == DTYPE and h(acc=1, M=0, x=0, w=0, y=0) == 0
    assert h(M=0, x=0, w=0, y=0) == NULL                   # dw is written as zeros


def test_workspace_is_asked_for(L):
    """Every product at some size: one byte less than it says, or none, is refused."""
    wb = L.mxq_bf16_grouped_mm_workspace_bytes
    for product, f in enumerate((L.mxq_bf16_grouped_mm, L.mxq_bf16_grouped_mm_dx, L.mxq_bf16_grouped_mm_dw)):
        for M, N, K, G in ((1, 512, 4096, 2), (4, 64, 8192, 1), (8, 8192, 64, 1), (16640, 64, 64, 1), (20000, 512, 256, 2)):
            need = wb(product, M, N, K, G)
            if need == 0:
                continue
            head = (A, A, A, M, N, K, G, 1) + ((0,) if product == 2 else ())
            assert f(*head, A, A, need - 1, 0) == WORKSPACE and f(*head, A, 0, need, 0) == WORKSPACE


def test_bindings_refuse_what_does_not_fit():
    x, w, e = bf(4, 64), bf(2, 16, 64), i32(2)
    with pytest.raises(ValueError):
        training.bf16_grouped_mm(x, w, e)                  # not on a device
    with pytest.raises(ValueError):
        mxq.mxq_bf16_grouped_mm(x, bf(2, 16, 32), e, bf(4, 16))
    with pytest.raises(ValueError):
        mxq.mxq_bf16_grouped_mm_dx(bf(4, 8), w, e, bf(4, 64))
    with pytest.raises(ValueError):
        mxq.mxq_bf16_grouped_mm_dw(bf(4, 16), x, e, bf(2, 16, 32))
    with pytest.raises(ValueError):
        training.bf16_grouped_mm_dw(bf(4, 16), x, e, dw=torch.zeros(1, 16, 64))
    with pytest.raises(TypeError):
        mxq.mxq_add_layernorm(x.to(torch.float16), None, bf(64), None, 1e-5)
    with pytest.raises(ValueError):
        training.add_layernorm(bf(64), None, bf(64), None, 1e-5)
    with pytest.raises(ValueError):
        mxq.mxq_dispatch_rows(x, i32(3, 2), 4, bf(8, 64), i32(4), i32(8), i32(4, 2), i32(4))
    with pytest.raises(ValueError):
        mxq.mxq_combine_rows(bf(64), i32(3, 2), None, bf(3, 64))
    with pytest.raises(ValueError):
        training.combine_rows_bwd(bf(4, 64), bf(64), i32(4, 2))


# helper, arguments, options, tensors it allocates (workspace included; the recorder's library asks for 64 bytes)
CALLS = [
    ("bf16_grouped_mm", lambda: (bf(4, 64), bf(2, 16, 64), i32(2)), {"out_dtype": torch.float32}, 2),
    ("bf16_grouped_mm_dx", lambda: (bf(4, 16), bf(2, 16, 64), i32(2)), {"out_dtype": torch.float32}, 2),
    ("bf16_grouped_mm_dw", lambda: (bf(4, 16), bf(4, 64), i32(2)), {"dw": torch.zeros(2, 16, 64)}, 1),
    ("add_layernorm", lambda: (bf(4, 64), bf(4, 64), bf(64), bf(64), 1e-5), {}, 6),
    ("add_layernorm_bwd", lambda: (bf(4, 64), bf(64), torch.zeros(4), torch.zeros(4), bf(4, 64)), {"dh": bf(4, 64)}, 4),
    ("dispatch_rows", lambda: (bf(4, 64), i32(4, 2), 8), {}, 5),
    ("pair_rows", lambda: (i32(8), 2), {}, 1),
    ("combine_rows", lambda: (bf(8, 64), i32(4, 2)), {"weights": torch.zeros(4, 2)}, 1),
    ("combine_rows_bwd", lambda: (bf(4, 64), bf(8, 64), i32(4, 2)), {"weights": torch.zeros(4, 2)}, 2),
]


@pytest.mark.parametrize("name,args,options,allocations", CALLS, ids=[c[0] for c in CALLS])
def test_a_given_stream_is_current_for_the_whole_helper(name, args, options, allocations, monkeypatch):
    inputs = args()
    r = Recorder(monkeypatch)
    getattr(training, name)(*inputs, **options)
    (entry, on, sizes), = r.launched
    assert on is None and r.allocated == [None] * allocations
    for handle, stream in ((4096, ("external", 4096)), (0, ("default",))):
        r.allocated.clear(), r.launched.clear()
        getattr(training, name)(*inputs, **options, stream=handle)
        assert r.launched == [(entry, stream, sizes)]             # the same call, options and all
        assert r.allocated == [stream] * allocations
        assert r.current is None


def test_every_helper_that_takes_a_stream_is_listed():
    import inspect
    takes = {n for n, f in vars(training).items() if inspect.isfunction(f) and not n.startswith("_")
             and "stream" in inspect.signature(f).parameters}
    assert takes == {c[0] for c in CALLS}
