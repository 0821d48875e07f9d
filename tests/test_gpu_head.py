"""GPU tests of the head loss and its gradients against a plain implementation
in float64.

Bounds. The products are fp32 sums of exact bfloat16 (or rounded fp32) products:
a logit of reduction H is off by at most (H + 2) * 2^-24 * sum |x w| =: dl. Then
  lse   dl + 2^-19 (exponentials and their fp32 sums, V <= 2^15 terms added in
        tiles, log, and the final fp32 roundings of |lse| < 16)
  loss  twice that
  G     |g| * (p * (2 * that + 2^-20) + 2^-23) + its rounding to the inputs' type
  dX, dW  the elementwise bound of G through |W| or |X|, plus the fp32 sums, plus
        the rounding of the result to the inputs' type.
All of them are evaluated in float64 element by element."""
import numpy as np
import pytest

import workloads as wl
from gpu_util import assert_bits_equal, host, log, padded, to_device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ql():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_linear_layer_amd as q
    q.lib()
    return q


def torch():
    import torch as t
    return t


def unit(dtype):
    """Relative rounding of the stored type."""
    return 2.0 ** -8 if dtype == wl.BF16 else U


def reference(X, W, target, dloss):
    """Everything in float64, W as H x V; rows left out where target is outside."""
    T, V = X.shape[0], W.shape[1]
    l = X @ W
    top = l.max(axis=1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(l - top).sum(axis=1))
    keep = (target >= 0) & (target < V)
    rows = np.nonzero(keep)[0]
    loss = np.zeros(T)
    loss[rows] = lse[rows] - l[rows, target[rows]]
    P = np.exp(l - lse[:, None])
    Z = P.copy()
    Z[rows, target[rows]] -= 1.0
    g = np.where(keep, dloss, 0.0)[:, None]
    G = Z * g
    return dict(l=l, lse=lse, loss=loss, P=P, G=G, g=np.abs(g), dX=G @ W.T, dW=X.T @ G)


def check(got, X, W, r, dtype):
    H, V, T = X.shape[1], W.shape[1], X.shape[0]
    dl = ((H + 2) * U * (np.abs(X) @ np.abs(W)))
    dlse = dl.max(axis=1) + 2.0 ** -19
    assert (np.abs(got["lse"] - r["lse"]) <= dlse).all(), "lse"
    assert (np.abs(got["loss"] - r["loss"]) <= dlse + dl.max(axis=1) + 2.0 ** -20).all(), "loss"
    if "dX" not in got:
        return
    dG = r["g"] * (r["P"] * (2 * (dlse[:, None] + dl) + 2.0 ** -20) + 2.0 ** -23)
    dG += unit(dtype) * (np.abs(r["G"]) + dG)
    for name, left, right, n in (("dX", None, np.abs(W).T, V), ("dW", np.abs(X).T, None, T)):
        mag = np.abs(r["G"]) + dG
        sums = (dG @ right + (n + 64) * U * (mag @ right)) if left is None else \
            (left @ dG + (n + 64) * U * (left @ mag))
        bound = sums + unit(dtype) * (np.abs(r[name]) + sums)
        bad = np.abs(got[name] - r[name]) > bound
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside the bound"


def inputs(T, H, V, dtype, seed=0, scale=1.0):
    rng = np.random.default_rng(seed + T + 3 * H + 5 * V)
    X = wl.random_matrix(rng, T, H, dtype, scale=scale)
    W = wl.random_matrix(rng, H, V, dtype, scale=0.05)
    target = rng.integers(0, V, T).astype(np.int32)
    dloss = (rng.standard_normal(T) / max(T, 1)).astype(np.float32)
    return X, W, target, dloss


def run(ql, X, W, target, dloss, by_vocab, pad=None):
    t = torch()
    Xd = to_device(X)
    Wd = to_device(W)
    if by_vocab:
        Wd = Wd.t().contiguous()
    if pad is not None:
        Xd, Wd = padded(Xd, Xd.shape[1] + pad), padded(Wd, Wd.shape[1] + pad)
    td = t.from_numpy(target).to("cuda:0")
    gd = t.from_numpy(dloss).to("cuda:0")
    loss, lse = ql.head_loss(Xd, Wd, td, by_vocab=by_vocab)
    dX, dW = ql.head_loss_backward(Xd, Wd, td, lse, gd, by_vocab=by_vocab)
    t.cuda.synchronize()
    return dict(loss=loss, lse=lse, dX=dX, dW=dW.t().contiguous() if by_vocab else dW)


def as64(out):
    return {k: host(v.float()).astype(np.float64) for k, v in out.items()}


SHAPES = [(1, 1, 1), (1, 64, 1000), (3, 33, 5), (31, 40, 131), (64, 128, 257), (65, 515, 300),
          (130, 256, 1031), (257, 96, 520), (300, 1032, 2056)]


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
@pytest.mark.parametrize("T,H,V", SHAPES)
def test_head_loss(ql, T, H, V, dtype, by_vocab):
    log(f"head loss {dtype} {T}x{H}x{V} {'VxH' if by_vocab else 'HxV'}")
    X, W, target, dloss = inputs(T, H, V, dtype)
    got = as64(run(ql, X, W, target, dloss, by_vocab))
    X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
    check(got, X64, W64, reference(X64, W64, target, dloss.astype(np.float64)), dtype)


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
def test_head_loss_large_tiles_and_pieces(ql, by_vocab):
    """Enough rows and columns for the largest tiles and for G in two pieces."""
    T, H, V = 2100, 136, 33000
    log(f"head loss in pieces {T}x{H}x{V}")
    X, W, target, dloss = inputs(T, H, V, wl.BF16)
    t = torch()
    Xd, Wd = to_device(X), to_device(W)
    out = run(ql, X, W, target, dloss, by_vocab)
    # the same in float64 on the GPU (products of float64 matrices)
    X64, W64 = Xd.double(), Wd.double()
    l = X64 @ W64
    lse = t.logsumexp(l, 1)
    tg = t.from_numpy(target).long().to("cuda:0")
    P = t.exp(l - lse[:, None])
    P[t.arange(T, device="cuda:0"), tg] -= 1.0
    P *= t.from_numpy(dloss).double().to("cuda:0")[:, None]
    loss = lse - l.gather(1, tg[:, None])[:, 0]
    # norms: fp32 sums for lse and loss; one rounding of G and one of the result
    # (2^-9 each at most, relative) for the gradients
    assert float((out["lse"].double() - lse).abs().max()) <= 2.0 ** -17
    assert float((out["loss"].double() - loss).abs().max()) <= 2.0 ** -16
    for name, want in (("dX", P @ W64.t()), ("dW", X64.t() @ P)):
        rel = float((out[name].double() - want).norm() / want.norm())
        assert rel <= 2.0 ** -8, f"{name}: {rel}"


def test_head_loss_mean_is_not_rounded_as_a_whole(ql):
    """All rows weighted alike by (1 + 2^-8) 2^-12, halfway between two bfloat16
    numbers: the gradients carry the roundings of G's and of their own entries,
    2^-9 / sqrt(3) of their norm each at most where they are independent, and not
    the 2^-8 of the weight. 1.5 * sqrt(2 / 3) * 2^-9 leaves room for half as much
    again."""
    T, H, V = 512, 256, 1024
    X, W, target, _ = inputs(T, H, V, wl.BF16, seed=3)
    dloss = np.full(T, (1 + 2.0 ** -8) * 2.0 ** -12, np.float32)
    got = as64(run(ql, X, W, target, dloss, False))
    r = reference(X.f32.astype(np.float64), W.f32.astype(np.float64), target, dloss.astype(np.float64))
    for k in ("dX", "dW"):
        rel = np.linalg.norm(got[k] - r[k]) / np.linalg.norm(r[k])
        log(f"head loss {k}: {rel:.2e}")
        assert rel <= 1.5 * np.sqrt(2 / 3) * 2.0 ** -9


@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_head_loss_left_out_rows(ql, dtype):
    """Targets outside the vocabulary: loss 0 and exactly no gradient; the rows
    that stay are not touched by them. Also all rows left out."""
    T, H, V = 140, 72, 333
    X, W, target, dloss = inputs(T, H, V, dtype)
    full = run(ql, X, W, target, dloss, False)
    out = target.copy()
    out[::3] = [-100, V, -1, 2 ** 31 - 1, -2 ** 31, V + 7] * 7 + [V] * (len(out[::3]) - 42)
    keep = (out >= 0) & (out < V)
    log(f"head loss {dtype}: {(~keep).sum()} rows left out")
    some = run(ql, X, W, out, dloss, False)
    for k in ("loss", "lse", "dX"):
        a, b = host(some[k].float()), host(full[k].float())
        assert_bits_equal(a[keep], b[keep], k)
    assert not host(some["loss"])[~keep].any()
    assert not host(some["dX"].float())[~keep].any()
    zeroed = run(ql, X, W, target, np.where(keep, dloss, 0).astype(np.float32), False)
    assert np.array_equal(host(some["dW"].float()), host(zeroed["dW"].float()))
    none = run(ql, X, W, np.full(T, -100, np.int32), dloss, False)
    assert not host(none["loss"]).any() and not host(none["dX"].float()).any()
    assert not host(none["dW"].float()).any()
    assert_bits_equal(host(none["lse"]), host(full["lse"]), "lse")


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("H", [72, 67])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_head_loss_left_out_rows_hold_anything(ql, dtype, H, by_vocab):
    """Infinities and NaN in X and dloss of rows that are left out: the losses and
    gradients are bit for bit those with finite numbers there."""
    T, V = 140, 333
    X, W, target, dloss = inputs(T, H, V, dtype, seed=7)
    target[1::4] = [-1, V] * 17 + [-100]
    out = (target < 0) | (target >= V)
    log(f"head loss {dtype}: {out.sum()} rows of infinities and NaN left out")
    want = run(ql, X, W, target, dloss, by_vocab)
    t = torch()
    rows = t.from_numpy(np.nonzero(out)[0]).to("cuda:0")
    Xd, Wd = to_device(X).clone(), to_device(W)
    Wd = Wd.t().contiguous() if by_vocab else Wd
    gd, td = t.from_numpy(dloss).to("cuda:0"), t.from_numpy(target).to("cuda:0")
    for bad in (float("nan"), float("inf"), -float("inf")):
        Xd[rows] = bad
        gd[rows] = bad
        loss, lse = ql.head_loss(Xd, Wd, td, by_vocab=by_vocab)
        dX, dW = ql.head_loss_backward(Xd, Wd, td, lse, gd, by_vocab=by_vocab)
        dW = dW.t().contiguous() if by_vocab else dW
        assert_bits_equal(host(loss), host(want["loss"]), "loss")
        assert_bits_equal(host(lse)[~out], host(want["lse"])[~out], "lse")
        assert_bits_equal(host(dX), host(want["dX"]), "dX")
        assert_bits_equal(host(dW), host(want["dW"]), "dW")


@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_head_loss_rows_keep_to_themselves(ql, dtype):
    """A NaN row of X and an infinite dloss that count: NaN in that row's loss
    and dX and in dW, and every other row's loss and dX as without them."""
    T, H, V = 70, 40, 300
    X, W, target, dloss = inputs(T, H, V, dtype, seed=9)
    dloss[:] = 0.5
    want = run(ql, X, W, target, dloss, False)
    t = torch()
    Xd, Wd = to_device(X).clone(), to_device(W)
    gd, td = t.from_numpy(dloss).to("cuda:0"), t.from_numpy(target).to("cuda:0")
    Xd[5] = float("nan")
    gd[33] = float("inf")
    log(f"head loss {dtype}: a NaN row and an infinite weight")
    loss, lse = ql.head_loss(Xd, Wd, td)
    dX, dW = ql.head_loss_backward(Xd, Wd, td, lse, gd)
    rest = np.ones(T, bool)
    rest[5] = False
    assert np.isnan(host(loss)[5])
    assert_bits_equal(host(loss)[rest], host(want["loss"])[rest], "loss")
    rest[33] = False
    d = host(dX.float())
    assert np.isnan(d[5]).all() and not np.isfinite(d[33]).any()
    assert_bits_equal(d[rest], host(want["dX"].float())[rest], "dX")
    assert not np.isfinite(host(dW.float())).any()


@pytest.mark.parametrize("scale", [1.0, 200.0])
def test_head_loss_large_logits(ql, scale):
    """Logits of some hundred, all negative or positive: no overflow, the
    largest dominates."""
    T, H, V = 70, 64, 300
    rng = np.random.default_rng(5)
    X = wl.from_f32(np.abs(rng.standard_normal((T, H))).astype(np.float32) * scale, wl.F32)
    for sign in (-1.0, 1.0):
        log(f"head loss logits around {sign * scale * 2}")
        W = wl.from_f32((sign * np.abs(rng.standard_normal((H, V)))).astype(np.float32) * 0.05, wl.F32)
        target = rng.integers(0, V, T).astype(np.int32)
        dloss = np.ones(T, np.float32)
        got = as64(run(ql, X, W, target, dloss, False))
        X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
        r = reference(X64, W64, target, np.ones(T))
        dl = (H + 2) * U * (np.abs(X64) @ np.abs(W64)).max(axis=1)
        lim = dl + 2.0 ** -19 + 4 * U * np.abs(r["lse"])
        assert (np.abs(got["lse"] - r["lse"]) <= lim).all()
        assert (np.abs(got["loss"] - r["loss"]) <= 2 * lim).all()
        assert np.isfinite(got["dX"]).all() and np.isfinite(got["dW"]).all()


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_head_loss_strides(ql, dtype, by_vocab):
    """Rows wider than their matrix, aligned and not, and a start that is not
    aligned: the same bits."""
    X, W, target, dloss = inputs(130, 96, 264, dtype)
    t = torch()
    want = run(ql, X, W, target, dloss, by_vocab)
    for pad in (8, 3):
        log(f"head loss strides {dtype}, {pad} more columns")
        got = run(ql, X, W, target, dloss, by_vocab, pad)
        for k in want:
            assert_bits_equal(host(got[k]), host(want[k]), k)
    Wd = to_device(W).t().contiguous() if by_vocab else to_device(W)
    buf = t.zeros(Wd.numel() + 1, dtype=Wd.dtype, device="cuda:0")
    view = buf[1:].view(Wd.shape)
    view.copy_(Wd)
    loss, lse = ql.head_loss(to_device(X), view, t.from_numpy(target).to("cuda:0"), by_vocab=by_vocab)
    assert_bits_equal(host(loss), host(want["loss"]), "loss")


def test_head_loss_difference_quotients(ql):
    """The gradients against differences of the loss itself, in float32: for
    directions u, (L(x + h u) - L(x - h u)) / 2h, h = 2^-6, to 2^-8 of the
    gradient's norm (curvature h^2 and rounding 2^-22 L / h)."""
    T, H, V = 20, 24, 50
    X, W, target, dloss = inputs(T, H, V, wl.F32)
    rng = np.random.default_rng(11)
    base = run(ql, X, W, target, dloss, False)
    t = torch()
    td = t.from_numpy(target).to("cuda:0")

    def total(x, w):
        return float((ql.head_loss(x, w, td)[0].double() * t.from_numpy(dloss).double().to("cuda:0")).sum())

    Xd, Wd = to_device(X), to_device(W)
    h = 2.0 ** -6
    for k in range(4):
        u = t.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to("cuda:0")
        u /= u.norm()
        slope = (total(Xd + h * u, Wd) - total(Xd - h * u, Wd)) / (2 * h)
        assert abs(slope - float((base["dX"] * u).sum())) <= 2.0 ** -8 * float(base["dX"].norm())
        u = t.from_numpy(rng.standard_normal((H, V)).astype(np.float32)).to("cuda:0")
        u /= u.norm()
        slope = (total(Xd, Wd + h * u) - total(Xd, Wd - h * u)) / (2 * h)
        assert abs(slope - float((base["dW"] * u).sum())) <= 2.0 ** -8 * float(base["dW"].norm())


def test_head_loss_no_rows(ql):
    t = torch()
    for by_vocab in (False, True):
        W = t.randn((40, 72) if not by_vocab else (72, 40), device="cuda:0")
        X = t.empty((0, 40), device="cuda:0")
        td = t.empty((0,), dtype=t.int32, device="cuda:0")
        loss, lse = ql.head_loss(X, W, td, by_vocab=by_vocab)
        assert loss.shape == (0,) and lse.shape == (0,)
        dX, dW = ql.head_loss_backward(X, W, td, lse, lse.clone(), by_vocab=by_vocab)
        assert dX.shape == (0, 40) and dW.shape == W.shape and not bool(dW.any())


def test_head_loss_repeats_stream_and_graph(ql):
    """The same bits every time: eager, on another stream, and in a graph that
    is replayed with eager work between."""
    t = torch()
    X, W, target, dloss = inputs(40, 520, 3000, wl.BF16)
    want = run(ql, X, W, target, dloss, False)
    again = run(ql, X, W, target, dloss, False)
    for k in want:
        assert_bits_equal(host(again[k]), host(want[k]), k)
    Xd, Wd = to_device(X), to_device(W)
    td, gd = t.from_numpy(target).to("cuda:0"), t.from_numpy(dloss).to("cuda:0")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    loss, lse = ql.head_loss(Xd, Wd, td, stream=s)
    dX, dW = ql.head_loss_backward(Xd, Wd, td, lse, gd, stream=s)
    t.cuda.current_stream().wait_stream(s)
    t.cuda.synchronize()
    assert_bits_equal(host(dW), host(want["dW"]), "dW on a stream")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        loss, lse = ql.head_loss(Xd, Wd, td)
        dX, dW = ql.head_loss_backward(Xd, Wd, td, lse, gd)
    for k in range(3):
        log(f"head loss graph replay {k}")
        for x in (loss, lse, dX, dW):
            x.fill_(5.0)
        g.replay()
        t.cuda.synchronize()
        for name, x in (("loss", loss), ("lse", lse), ("dX", dX), ("dW", dW)):
            assert_bits_equal(host(x), host(want[name]), f"{name} of replay {k}")
        run(ql, X, W, target, dloss, False)


def test_head_loss_binding_refusals(ql):
    t = torch()
    dev = "cuda:0"
    X, W = t.zeros((4, 16), device=dev), t.zeros((16, 24), device=dev)
    td = t.zeros(4, dtype=t.int32, device=dev)
    with pytest.raises(ValueError):
        ql.head_loss(X, W, td, by_vocab=True)
    with pytest.raises(TypeError):
        ql.head_loss(X, W, td.long())
    with pytest.raises(ValueError):
        ql.head_loss(X, W, td[:3])
    with pytest.raises(TypeError):
        ql.head_loss(X.bfloat16(), W, td)
    with pytest.raises(TypeError):
        ql.head_loss(X.half(), W.half(), td)
    with pytest.raises(ValueError):
        ql.head_loss(X, W.t(), td, by_vocab=True)
    with pytest.raises(ValueError):
        ql.head_loss(X.cpu(), W, td)
    f = t.zeros(4, device=dev)
    with pytest.raises(TypeError):
        ql.head_loss_backward(X, W, td, f, f.double())
    with pytest.raises(ql.Fp4linError):
        ql.fp4lin_head_loss(X, W, td, f, f.clone(), t.empty(16, dtype=t.uint8, device=dev))
