"""Host-side checks of the C entries that move rows (experts' routing, embedding): every
call here fails argument validation, has nothing to do or is a pure host helper."""
import ctypes
import os

import pytest

qll = pytest.importorskip("quantized_linear_layer_amd")
torch = pytest.importorskip("torch")
from quantized_linear_layer_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libfp4lin.so not built (run __graft_entry__.build())", allow_module_level=True)

L = _lib.load()
P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced (validation fails first)
ODD, HALF = P(0x10001), P(0x10002)
BIG = 1 << 40


def dispatch(X=FAKE, dt=0, expert=FAKE, T=4, k=2, E=3, H=8, ldx=8, Xs=FAKE, ldxs=8, row_end=FAKE, slot_row=FAKE):
    return L.fp4lin_experts_dispatch(X, dt, expert, T, k, E, H, ldx, Xs, ldxs, row_end, slot_row, None)


def combine(Y=FAKE, ydt=0, slot_row=FAKE, row_end=FAKE, weight=FAKE, residual=FAKE, T=4, k=2, E=3, H=8, ldy=8, ldr=8,
            out=FAKE, odt=0, ldo=8):
    return L.fp4lin_experts_combine(Y, ydt, slot_row, row_end, weight, residual, T, k, E, H, ldy, ldr, out, odt, ldo,
                                    None)


def back(dout=FAKE, odt=0, Y=FAKE, ydt=0, slot_row=FAKE, row_end=FAKE, weight=FAKE, T=4, k=2, E=3, H=8, lddo=8, ldy=8,
         dY=FAKE, dydt=0, lddy=8, dweight=FAKE):
    return L.fp4lin_experts_combine_backward(dout, odt, Y, ydt, slot_row, row_end, weight, T, k, E, H, lddo, ldy, dY,
                                             dydt, lddy, dweight, None)


SIZES = (dict(T=-1), dict(k=0), dict(E=0), dict(E=65535), dict(H=0), dict(H=1 << 31), dict(T=1 << 31),
         dict(T=1 << 20, k=1 << 11), dict(k=1 << 62), dict(T=1 << 29, k=1, H=100))


@pytest.mark.parametrize("call,pointers,types,strides,halves", [
    (dispatch, ("X", "expert", "Xs", "row_end", "slot_row"), ("dt",), ("ldx", "ldxs"), ()),
    (combine, ("Y", "slot_row", "row_end", "out"), ("ydt", "odt"), ("ldy", "ldr", "ldo"), ("weight", "residual")),
    (back, ("dout", "Y", "slot_row", "row_end", "dY"), ("odt", "ydt", "dydt"), ("lddo", "ldy", "lddy"),
     ("weight", "dweight"))])
def test_route_refusals(call, pointers, types, strides, halves):
    for name in pointers:
        assert call(**{name: None}) == _lib.ERR_NULL, name
        assert call(**{name: HALF}) == _lib.ERR_ALIGN, name  # float32 and int32
    for name in halves:
        assert call(**{name: HALF}) == _lib.ERR_ALIGN, name
    for name in types:
        assert call(**{name: 2}) == _lib.ERR_DTYPE, name
    for name in strides:
        assert call(**{name: 7}) == _lib.ERR_SHAPE, name
    for bad in SIZES:
        big = {s: bad.get("H", 8) for s in strides}
        assert call(**{**big, **bad}) == _lib.ERR_SHAPE, bad


def test_bfloat16_alignment():
    assert dispatch(X=ODD, dt=1) == _lib.ERR_ALIGN
    assert combine(Y=ODD, ydt=1) == _lib.ERR_ALIGN
    assert back(dY=ODD, dydt=1) == _lib.ERR_ALIGN


def test_no_tokens_enqueue_nothing():
    none = dict(T=0, slot_row=None)
    assert combine(Y=None, out=None, weight=None, residual=None, **none) == _lib.OK
    assert back(dout=None, Y=None, dY=None, weight=None, dweight=None, **none) == _lib.OK
    assert dispatch(T=0, X=None, expert=None, Xs=None, slot_row=None, row_end=None) == _lib.ERR_NULL


def embed(table=FAKE, dt=0, token=FAKE, T=4, V=10, H=8, ldt=8, scale=1.0, out=FAKE, odt=0, ldo=8):
    return L.fp4lin_embed(table, dt, token, T, V, H, ldt, scale, out, odt, ldo, None)


def embed_back(dX=FAKE, dt=0, token=FAKE, T=4, V=10, H=8, lddx=8, scale=1.0, add=0, dE=FAKE, edt=0, ldde=8, ws=FAKE,
               n=BIG):
    return L.fp4lin_embed_backward(dX, dt, token, T, V, H, lddx, scale, add, dE, edt, ldde, ws, n, None)


@pytest.mark.parametrize("call,pointers,types,strides", [
    (embed, ("table", "token", "out"), ("dt", "odt"), ("ldt", "ldo")),
    (embed_back, ("dX", "token", "dE", "ws"), ("dt", "edt"), ("lddx", "ldde"))])
def test_embed_refusals(call, pointers, types, strides):
    for name in pointers:
        assert call(**{name: None}) == _lib.ERR_NULL, name
        assert call(**{name: HALF}) == _lib.ERR_ALIGN, name
    for name in types:
        assert call(**{name: -1}) == _lib.ERR_DTYPE, name
    for name in strides:
        assert call(**{name: 7}) == _lib.ERR_SHAPE, name
    for bad in (dict(T=-1), dict(V=0), dict(H=0), dict(V=1 << 31), dict(T=1 << 31), dict(T=1 << 29, H=100)):
        assert call(**{**{s: bad.get("H", 8) for s in strides}, **bad}) == _lib.ERR_SHAPE, bad
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert call(scale=scale) == _lib.ERR_VALUE


def test_embed_workspace():
    w = L.fp4lin_embed_backward_workspace_bytes
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 0), (1 << 31, 5, 5), (5, 1 << 31, 5), (5, 1 << 29, 100)):
        assert w(*bad) == 0, bad
    assert w(0, 5, 5) >= 256
    # positions, ends, and two fp32 rows of each piece of a list that can be long
    assert w(8192, 32000, 4096) >= 4 * 8192 + 4 * 32000 + 8192 // 64 * 2 * 4 * 4096
    assert w(1, 1 << 20, 64) < (4 << 20) + 1024
    assert embed_back(n=w(4, 10, 8) - 1) == _lib.ERR_WORKSPACE
    assert embed(T=0, table=None, token=None, out=None) == _lib.OK


# ---- the binding -----------------------------------------------------------------------
@pytest.fixture
def library(monkeypatch):
    """Notes the calls of the C entries and the GPU they were made on; GPU 0 is current."""
    class Library:
        calls, gpus, current = [], [], 0

        def __getattr__(self, name):
            def call(*args):
                self.calls.append(name)
                self.gpus.append(self.current)
                return 0
            return call

    lib = Library()
    lib.calls, lib.gpus = [], []

    class Device:
        def __init__(self, number):
            self.number = number

        def __enter__(self):
            self.before, lib.current = lib.current, self.number

        def __exit__(self, *_):
            lib.current = self.before

    monkeypatch.setattr(qll, "lib", lambda: lib)
    monkeypatch.setattr(qll, "_queue", lambda stream, device: 0)
    monkeypatch.setattr(qll, "_current", lambda: lib.current)
    monkeypatch.setattr(qll, "_gpu", lambda *tensors: 1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    return lib


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_calls_on_the_tensors_gpu(library):
    X, Y, w = torch.zeros((4, 8)), torch.zeros((8, 8)), torch.zeros((4, 2))
    qll.fp4lin_experts_dispatch(X, ints(4, 2), Y, ints(3), ints(4, 2))
    qll.fp4lin_experts_combine(Y, ints(4, 2), ints(3), X, w, X)
    qll.fp4lin_experts_combine_backward(X, Y, ints(4, 2), ints(3), Y, w, w)
    qll.fp4lin_embed(Y, ints(4), X)
    qll.fp4lin_embed_backward(X, ints(4), Y, torch.zeros(64, dtype=torch.uint8))
    assert len(library.calls) == 5 and library.gpus == [1] * 5 and library.current == 0


def test_binding_refusals(library):
    X, Y, w = torch.zeros((4, 8)), torch.zeros((8, 8)), torch.zeros((4, 2))
    bad = [
        lambda: qll.fp4lin_experts_dispatch(X, ints(3, 2), Y, ints(3), ints(3, 2)),
        lambda: qll.fp4lin_experts_dispatch(X, ints(4, 3), Y, ints(3), ints(4, 3)),
        lambda: qll.fp4lin_experts_dispatch(X, ints(4, 2).long(), Y, ints(3), ints(4, 2)),
        lambda: qll.fp4lin_experts_dispatch(X, ints(2, 4).t(), Y, ints(3), ints(4, 2)),
        lambda: qll.fp4lin_experts_dispatch(X, ints(4, 2), Y.bfloat16(), ints(3), ints(4, 2)),
        lambda: qll.fp4lin_experts_dispatch(X, ints(4, 2), Y, ints(3).long(), ints(4, 2)),
        lambda: qll.fp4lin_experts_dispatch(X, ints(4, 2), Y, ints(3), ints(7)),
        lambda: qll.fp4lin_experts_dispatch(X.double(), ints(4, 2), Y.double(), ints(3), ints(4, 2)),
        lambda: qll.fp4lin_experts_combine(Y, ints(4, 2), ints(3), X, w.double()),
        lambda: qll.fp4lin_experts_combine(Y, ints(4, 2), ints(3), X, torch.zeros((4, 3))),
        lambda: qll.fp4lin_experts_combine(Y, ints(4, 2), ints(3), X, w, X.bfloat16()),
        lambda: qll.fp4lin_experts_combine(Y, ints(4, 2), ints(3), X, w, Y),
        lambda: qll.fp4lin_experts_combine(X, ints(4, 2), ints(3), X, w),
        lambda: qll.fp4lin_experts_combine(Y, ints(5, 2), ints(3), X, w),
        lambda: qll.fp4lin_experts_combine(Y.t()[:, ::2].t(), ints(4, 2), ints(3), X, w),
        lambda: qll.fp4lin_experts_combine_backward(X, None, ints(4, 2), ints(3), Y, w, w),
        lambda: qll.fp4lin_experts_combine_backward(X, X, ints(4, 2), ints(3), Y, w, w),
        lambda: qll.fp4lin_experts_combine_backward(X, Y, ints(4, 2), ints(3), X, w, w),
        lambda: qll.fp4lin_experts_combine_backward(X, Y, ints(4, 2), ints(3), Y, w, w[:3]),
        lambda: qll.fp4lin_embed(Y, ints(3), X),
        lambda: qll.fp4lin_embed(Y, ints(4).long(), X),
        lambda: qll.fp4lin_embed(Y[:, :4], ints(4), X),
        lambda: qll.fp4lin_embed_backward(X, ints(4), Y[:, :4], torch.zeros(64)),
        lambda: qll.fp4lin_embed_backward(X, ints(5), Y, torch.zeros(64)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert library.calls == [], i


# ---- the head loss against a teacher's top logits --------------------------------------
HID, VOC = _lib.HEAD_HIDDEN_MAJOR, _lib.HEAD_VOCAB_MAJOR


def distill_ws(dt=1, layout=HID, T=64, H=64, V=512, k=8, ldx=64, ldw=512, backward=False):
    f = L.fp4lin_head_distill_backward_workspace_bytes if backward else L.fp4lin_head_distill_workspace_bytes
    return f(dt, layout, T, H, V, k, ldx, ldw)


def distill(X=FAKE, W=FAKE, dt=1, layout=HID, index=FAKE, teacher=FAKE, tdt=0, k=8, temperature=1.0, T=4, H=64, V=512,
            ldx=64, ldw=512, loss=FAKE, lse=FAKE, ws=FAKE, n=BIG):
    return L.fp4lin_head_distill(X, W, dt, layout, index, teacher, tdt, k, temperature, T, H, V, ldx, ldw, loss, lse,
                                 ws, n, None)


def distill_back(X=FAKE, W=FAKE, dt=1, layout=HID, index=FAKE, teacher=FAKE, tdt=0, k=8, temperature=1.0, T=4, H=64,
                 V=512, ldx=64, ldw=512, lse=FAKE, dloss=FAKE, dX=FAKE, lddx=64, dW=FAKE, lddw=512, ws=FAKE, n=BIG):
    return L.fp4lin_head_distill_backward(X, W, dt, layout, index, teacher, tdt, k, temperature, lse, dloss, T, H, V,
                                          ldx, ldw, dX, lddx, dW, lddw, ws, n, None)


@pytest.mark.parametrize("call,pointers", [
    (distill, ("X", "W", "index", "teacher", "loss", "lse", "ws")),
    (distill_back, ("X", "W", "index", "teacher", "lse", "dloss", "dX", "dW", "ws"))])
def test_distill_refusals(call, pointers):
    for name in pointers:
        assert call(**{name: None}) == _lib.ERR_NULL, name
    assert call(dt=2) == _lib.ERR_DTYPE and call(tdt=2) == _lib.ERR_DTYPE
    for bad in (dict(layout=5), dict(T=-1), dict(H=0), dict(V=0), dict(ldx=63), dict(ldw=511), dict(k=0), dict(k=1025)):
        assert call(**bad) == _lib.ERR_SHAPE, bad
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-40, 1e46):
        assert call(temperature=bad) == _lib.ERR_VALUE, bad
    for name in ("X", "W", "ws", "index", "teacher"):
        assert call(**{name: HALF}) == _lib.ERR_ALIGN, name
    assert call(teacher=ODD, tdt=1) == _lib.ERR_ALIGN
    assert call(n=distill_ws(T=4, backward=call is distill_back) - 1) == _lib.ERR_WORKSPACE
    if call is distill_back:
        assert call(lddx=63) == _lib.ERR_SHAPE and call(lddw=511) == _lib.ERR_SHAPE
    else:
        assert call(T=0, X=None, index=None, teacher=None, loss=None, lse=None) == _lib.OK


@pytest.mark.parametrize("backward", [False, True])
def test_distill_workspace(backward):
    plain = L.fp4lin_head_loss_backward_workspace_bytes if backward else L.fp4lin_head_loss_workspace_bytes
    # a teacher's pairs and where every 32 columns begin among them
    assert distill_ws(backward=backward) >= plain(1, HID, 64, 64, 512, 64, 512) + 64 * (8 * 8 + 17 * 2)
    assert distill_ws(T=0, backward=backward) >= 256
    for bad in (dict(k=0), dict(k=1025), dict(T=-1), dict(V=0), dict(layout=2), dict(dt=3), dict(ldw=511)):
        assert distill_ws(**bad, backward=backward) == 0, bad


def test_distill_binding_refusals(library):
    X, W, f, ws = torch.zeros((4, 8)), torch.zeros((8, 6)), torch.zeros(4), torch.zeros(64, dtype=torch.uint8)
    i, u = ints(4, 3), torch.zeros((4, 3))
    bad = [
        lambda: qll.fp4lin_head_distill(X, W, i.long(), u, f, f, ws),
        lambda: qll.fp4lin_head_distill(X, W, ints(3, 4).t(), u, f, f, ws),
        lambda: qll.fp4lin_head_distill(X, W, ints(3, 3), torch.zeros((3, 3)), f, f, ws),
        lambda: qll.fp4lin_head_distill(X, W, ints(4), torch.zeros(4), f, f, ws),
        lambda: qll.fp4lin_head_distill(X, W, i, torch.zeros((4, 2)), f, f, ws),
        lambda: qll.fp4lin_head_distill(X, W, i, u.double(), f, f, ws),
        lambda: qll.fp4lin_head_distill(X, W, i, u, f[:3], f, ws),
        lambda: qll.fp4lin_head_distill(X, W, i, u, f, f, ws, by_vocab=True),
        lambda: qll.fp4lin_head_distill_backward(X, W, i, u, f, f.double(), X, W, ws),
        lambda: qll.fp4lin_head_distill_backward(X, W, i, u, f, f, X[:3], W, ws),
        lambda: qll.fp4lin_head_distill_backward(X, W, i, u, f, f, X, W.t(), ws),
        lambda: qll.fp4lin_head_distill_backward(X, W, i, u, f, f, X.bfloat16(), W, ws),
    ]
    for n, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert library.calls == [], n
    qll.fp4lin_head_distill(X, W, i, u, f, f, ws)
    qll.fp4lin_head_distill_backward(X, W, i, u, f, f, X, W, ws)
    assert library.gpus == [1, 1]
