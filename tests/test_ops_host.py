"""Host-side checks of the C entries of the experts' products, the head loss and
the gradient clipping (no GPU work): every call here fails argument validation or is a pure host helper."""
import ctypes
import os

import pytest

qll = pytest.importorskip("quantized_linear_layer_amd")
from quantized_linear_layer_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libfp4lin.so not built (run __graft_entry__.build())", allow_module_level=True)

L = _lib.load()
P = ctypes.c_void_p
FAKE = P(0x10000)        # 16-byte aligned, never dereferenced (validation fails first)
MISALIGNED = P(0x10004)
PASSES = (_lib.EXPERTS_FORWARD, _lib.EXPERTS_DGRAD, _lib.EXPERTS_WGRAD, _lib.EXPERTS_APPLY)
BIG = 1 << 40


def ws_bytes(which, E, M, K, N):
    return L.fp4lin_experts_workspace_bytes(which, E, M, K, N)


def pad(n, a=256):
    return (n + a - 1) // a * a


@pytest.mark.parametrize("E,M,K,N", [(1, 1, 1, 1), (8, 8192, 4096, 11008), (5, 777, 515, 1003),
                                     (64, 3, 100, 7)])
def test_experts_workspace_bytes(E, M, K, N):
    """Codes and scales of both operands of each pass, 256-byte aligned."""
    def packed(rows, length):
        ldq = L.fp4lin_packed_ld(length)
        return pad(rows * ldq) + pad(rows * ldq // 16)
    steps = (M + min(E, M) * 127) // 128
    # any split of M rows over E experts fits the steps
    assert steps >= max(-(-M // 128), (M - min(E, M) + 1 + 127) // 128 + min(E, M) - 1)
    assert ws_bytes(_lib.EXPERTS_FORWARD, E, M, K, N) == packed(M, K) + packed(E * N, K)
    assert ws_bytes(_lib.EXPERTS_DGRAD, E, M, K, N) == packed(M, N) + packed(E * K, N)
    assert ws_bytes(_lib.EXPERTS_APPLY, E, M, K, N) == packed(M, K)
    assert ws_bytes(_lib.EXPERTS_WGRAD, E, M, K, N) == sum(
        pad(r * steps * 64) + pad(r * steps * 4) for r in (K, N))


def test_experts_workspace_bytes_invalid():
    for which in PASSES:
        assert ws_bytes(which, 0, 4, 4, 4) == 0
        assert ws_bytes(which, 65535, 4, 4, 4) == 0
        assert ws_bytes(which, 2, -1, 4, 4) == 0
        assert ws_bytes(which, 2, 4, 0, 4) == 0
        assert ws_bytes(which, 2, 4, 4, 0) == 0
        assert ws_bytes(which, 2, 1 << 31, 4, 4) == 0
        # operands beyond 32-bit offsets
        assert ws_bytes(which, 2, 1 << 20, 1 << 20, 1 << 20) == 0
        # no rows is a valid batch
        assert ws_bytes(which, 2, 0, 4, 4) >= 256
    assert ws_bytes(7, 2, 4, 4, 4) == 0
    # scales of all experts beyond 32-bit offsets
    assert ws_bytes(_lib.EXPERTS_APPLY, 65534, 4, 32768, 4096) == 0


def forward(A=FAKE, W=FAKE, dt=0, end=FAKE, E=2, M=4, K=8, N=8, lda=8, ldw=8, Y=FAKE, ydt=0, ldy=8,
            ws=FAKE, n=BIG):
    return L.fp4lin_experts_forward_mx(A, W, dt, end, E, M, K, N, lda, ldw, Y, ydt, ldy, ws, n, None)


def dgrad(A=FAKE, W=FAKE, dt=0, end=FAKE, E=2, M=4, K=8, N=8, lda=8, ldw=8, Y=FAKE, ydt=0, ldy=8,
          ws=FAKE, n=BIG):
    return L.fp4lin_experts_dgrad_mx(A, W, dt, end, E, M, K, N, lda, ldw, Y, ydt, ldy, ws, n, None)


def wgrad(A=FAKE, W=FAKE, dt=0, end=FAKE, E=2, M=4, K=8, N=8, lda=8, ldw=8, Y=FAKE, ydt=0, ldy=8,
          ws=FAKE, n=BIG):
    return L.fp4lin_experts_wgrad_mx(A, W, dt, end, E, M, K, N, lda, ldw, Y, ydt, ldy, ws, n, None)


def apply(A=FAKE, W=FAKE, dt=0, end=FAKE, E=2, M=4, K=8, N=8, lda=8, ldw=8, Y=FAKE, ydt=0, ldy=8,
          ws=FAKE, n=BIG, Ws=FAKE):
    return L.fp4lin_experts_apply_mx(A, dt, W, Ws, end, E, M, K, N, lda, Y, ydt, ldy, ws, n, None)


@pytest.mark.parametrize("call", [forward, dgrad, wgrad, apply])
def test_experts_refusals(call):
    for name in ("A", "W", "end", "Y", "ws"):
        assert call(**{name: None}) == _lib.ERR_NULL, name
    assert call(dt=2) == _lib.ERR_DTYPE
    assert call(ydt=-1) == _lib.ERR_DTYPE
    for bad in (dict(E=0), dict(E=65535), dict(M=-1), dict(K=0), dict(N=0), dict(M=1 << 31),
                dict(lda=7), dict(ldy=7)):
        assert call(**bad) == _lib.ERR_SHAPE, bad
    assert call(ws=MISALIGNED) == _lib.ERR_ALIGN
    assert call(n=255) == _lib.ERR_WORKSPACE
    if call is not apply:
        assert call(ldw=7) == _lib.ERR_SHAPE
    else:
        assert call(Ws=None) == _lib.ERR_NULL
        assert call(W=MISALIGNED) == _lib.ERR_ALIGN


@pytest.mark.parametrize("call", [forward, dgrad, apply])
def test_experts_no_rows_enqueue_nothing(call):
    """M = 0: done, with or without the M-row arrays."""
    assert call(M=0) == _lib.OK
    assert call(M=0, A=None, Y=None) == _lib.OK


def test_experts_quantize_weight_refusals():
    def q(W=FAKE, dt=0, E=2, K=8, N=8, ldw=8, Wq=FAKE, Ws=FAKE):
        return L.fp4lin_experts_quantize_weight_mx(W, dt, E, K, N, ldw, Wq, Ws, None)
    for name in ("W", "Wq", "Ws"):
        assert q(**{name: None}) == _lib.ERR_NULL
    assert q(dt=5) == _lib.ERR_DTYPE
    for bad in (dict(E=0), dict(K=0), dict(N=0), dict(ldw=7), dict(K=65535 * 128 + 1)):
        assert q(**bad) == _lib.ERR_SHAPE, bad
    assert q(Wq=MISALIGNED) == _lib.ERR_ALIGN
    assert q(Ws=MISALIGNED) == _lib.ERR_ALIGN


# ---- head loss -------------------------------------------------------------------
HID, VOC = _lib.HEAD_HIDDEN_MAJOR, _lib.HEAD_VOCAB_MAJOR


def head_ws(dt=1, layout=HID, T=64, H=64, V=512, ldx=64, ldw=512, backward=False):
    f = L.fp4lin_head_loss_backward_workspace_bytes if backward else L.fp4lin_head_loss_workspace_bytes
    return f(dt, layout, T, H, V, ldx, ldw)


@pytest.mark.parametrize("backward", [False, True])
def test_head_workspace_bytes(backward):
    ok = dict(backward=backward)
    assert head_ws(**ok) >= 256
    assert head_ws(T=0, **ok) >= 256
    # a padded copy of an operand whose rows are not whole 16-byte pieces
    assert head_ws(V=511, ldw=511, **ok) >= head_ws(V=504, **ok) + 64 * 512 * 2
    if backward:  # always a copy of X
        assert head_ws(**ok) >= head_ws(backward=False) + 64 * 64 * 2
    else:
        assert head_ws(ldx=67) >= head_ws() + 64 * 64 * 2
    assert head_ws(layout=VOC, ldw=64, **ok) >= 256
    for bad in (dict(dt=3), dict(layout=2), dict(T=-1), dict(H=0), dict(V=0), dict(ldx=63),
                dict(ldw=511), dict(T=1 << 31), dict(ldw=1 << 23), dict(layout=VOC, ldw=63)):
        assert head_ws(**{**bad, **ok}) == 0, bad
    # the backward's G stays a piece of the vocabulary
    assert head_ws(T=8192, H=4096, V=1 << 20, ldx=4096, ldw=1 << 20, backward=True) < 1 << 30


def head(X=FAKE, W=FAKE, dt=1, layout=HID, target=FAKE, T=4, H=64, V=512, ldx=64, ldw=512, loss=FAKE,
         lse=FAKE, ws=FAKE, n=BIG):
    return L.fp4lin_head_loss(X, W, dt, layout, target, T, H, V, ldx, ldw, loss, lse, ws, n, None)


def head_back(X=FAKE, W=FAKE, dt=1, layout=HID, target=FAKE, T=4, H=64, V=512, ldx=64, ldw=512,
              lse=FAKE, dloss=FAKE, dX=FAKE, lddx=64, dW=FAKE, lddw=512, ws=FAKE, n=BIG):
    return L.fp4lin_head_loss_backward(X, W, dt, layout, target, lse, dloss, T, H, V, ldx, ldw, dX,
                                       lddx, dW, lddw, ws, n, None)


@pytest.mark.parametrize("call,pointers", [
    (head, ("X", "W", "target", "loss", "lse", "ws")),
    (head_back, ("X", "W", "target", "lse", "dloss", "dX", "dW", "ws"))])
def test_head_refusals(call, pointers):
    for name in pointers:
        assert call(**{name: None}) == _lib.ERR_NULL, name
    assert call(dt=2) == _lib.ERR_DTYPE
    for bad in (dict(layout=5), dict(T=-1), dict(H=0), dict(V=0), dict(ldx=63), dict(ldw=511)):
        assert call(**bad) == _lib.ERR_SHAPE, bad
    for name in ("X", "W", "ws"):
        assert call(**{name: MISALIGNED}) == _lib.ERR_ALIGN, name
    assert call(n=255) == _lib.ERR_WORKSPACE
    if call is head_back:
        assert call(lddx=63) == _lib.ERR_SHAPE
        assert call(lddw=511) == _lib.ERR_SHAPE
    else:
        assert call(T=0, X=None, target=None, loss=None, lse=None) == _lib.OK


# ---- clipping ----------------------------------------------------------------------
def grads(*entries):
    a = (_lib.Grad * max(len(entries), 1))()
    for i, e in enumerate(entries):
        a[i] = _lib.Grad(*e)
    return a, len(entries)


GOOD = (0x10000, 0x10000, 100, 0)


def norm(entries=(GOOD,), out=FAKE, ws=FAKE, n=BIG):
    a, count = grads(*entries)
    return L.fp4lin_grad_norm(a, count, out, ws, n, None)


def clip(entries=(GOOD,), out=FAKE, ws=FAKE, n=BIG, max_norm=1.0):
    a, count = grads(*entries)
    return L.fp4lin_clip_grads(a, count, max_norm, out, ws, n, None)


@pytest.mark.parametrize("call", [norm, clip])
def test_clip_refusals(call):
    assert call(out=None) == _lib.ERR_NULL
    assert call(ws=None) == _lib.ERR_NULL
    assert call(entries=[GOOD, (None, 0x10000, 1, 0)]) == _lib.ERR_NULL
    assert call(entries=[GOOD, (0x10000, 0x10000, -1, 0)]) == _lib.ERR_SHAPE
    assert call(entries=[GOOD, (0x10000, 0x10000, 1 << 47, 0)]) == _lib.ERR_SHAPE
    assert call(entries=[GOOD, (0x10000, 0x10000, 4, 2)]) == _lib.ERR_DTYPE
    assert call(entries=[GOOD, (0x10002, 0x10000, 4, 0)]) == _lib.ERR_ALIGN
    assert call(entries=[GOOD, (0x10001, 0x10000, 4, 1)]) == _lib.ERR_ALIGN
    assert call(ws=MISALIGNED) == _lib.ERR_ALIGN
    assert call(n=16) == _lib.ERR_WORKSPACE


def test_clip_max_norm():
    assert clip(max_norm=float("nan")) == _lib.ERR_VALUE
    assert clip(max_norm=-0.5) == _lib.ERR_VALUE
    assert clip(entries=[GOOD, (0x10000, None, 1, 0)]) == _lib.ERR_NULL
    assert clip(entries=[GOOD, (0x10000, 0x10002, 1, 0)]) == _lib.ERR_ALIGN


def test_clip_workspace_bytes():
    assert L.fp4lin_clip_workspace_bytes(-1, 4) == 0
    assert L.fp4lin_clip_workspace_bytes(1, -1) == 0
    assert L.fp4lin_clip_workspace_bytes(0, 0) >= 16
    # at most 2048 chunks and one more a tensor
    assert L.fp4lin_clip_workspace_bytes(100, 1 << 40) <= 16 + 8 * (2048 + 100) + 256
