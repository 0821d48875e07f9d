"""GPU tests of the head loss against a teacher's top logits and of its gradients, against
a plain implementation in float64.

Bounds (U = 2^-24). A logit is off by at most (H + 2) * U * sum |x w| / temperature and
the roundings of the scale and of the product by it, 3 U |z|: dz. As in the head loss
  lse   dlse = dz + 2^-19 + 2 U |lse|
A teacher's u / temperature is off by 3 U |u / temperature|, and u - M by U |u - M| more:
du; the exponential by 2^-22, the sum of k of them by k U, the quotient by U:
  p     p * dp,  dp = 2 du + 2^-21 + (k + 4) U   (relative)
  loss  sum_j p dp (|log p| + |z| + |lse|) + sum_j p (dp + dz + dlse) + the fp32 sums,
        (k + 64) U of sum_j p (|log p| + |z| + |lse|)
  G     |g| * (q * (2 (dlse + dz) + 2^-20) + P * dp + 2^-22) + its rounding
  dX, dW  the elementwise bound of G through |W| or |X|, the fp32 sums and the rounding
        to the inputs' type.
All of them are evaluated in float64 element by element."""
import numpy as np
import pytest

import workloads as wl
from gpu_util import assert_bits_equal, host, log, padded, to_device
from test_gpu_head import U, as64, ql, torch, unit  # noqa: F401 (ql is a fixture)

pytestmark = pytest.mark.gpu


def inputs(T, H, V, k, dtype, seed=0, left=0.1):
    rng = np.random.default_rng(seed + T + 3 * H + 5 * V + 7 * k)
    X = wl.random_matrix(rng, T, H, dtype, scale=1.0)
    W = wl.random_matrix(rng, H, V, dtype, scale=0.05)
    # indices crowd together in half of the rows; some come twice, some lie outside
    index = rng.integers(0, V, (T, k))
    index[::2] = (rng.integers(0, V, (T, 1)) + rng.integers(0, 40, (T, k)))[::2] % V
    out = rng.random((T, k)) < left
    index[out] = rng.choice([-1, V, -2 ** 31, 2 ** 31 - 1], out.sum())
    teacher = (3 * rng.standard_normal((T, k))).astype(np.float32)
    dloss = (rng.standard_normal(T) / max(T, 1)).astype(np.float32)
    return X, W, index.astype(np.int32), teacher, dloss


def reference(X, W, index, teacher, dloss, tau):
    """Everything in float64, W as H x V."""
    T, V, k = X.shape[0], W.shape[1], index.shape[1]
    z = X @ W / tau
    top = z.max(axis=1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
    u = teacher.astype(np.float64) / tau
    kept = (index >= 0) & (index < V) & (u > -np.inf)
    some = kept.any(axis=1)
    M = np.where(kept, u, -np.inf).max(axis=1, initial=-np.inf, keepdims=True)
    M[~some] = 0
    e = np.where(kept, np.exp(np.where(kept, u, 0) - M), 0)
    s = e.sum(axis=1, keepdims=True)
    s[~some] = 1
    p = e / s
    logp = np.where(p > 0, np.where(kept, u, 0) - M - np.log(s), 0)
    at = np.where(kept, index, 0)
    zj = np.take_along_axis(z, at, 1)
    size = (p * (np.abs(logp) + np.abs(zj) + np.abs(lse[:, None]))).sum(axis=1)
    loss = (p * (logp - zj)).sum(axis=1) + lse * p.sum(axis=1)
    P = np.zeros((T, V))
    np.add.at(P, (np.arange(T)[:, None].repeat(k, 1), at), p)
    Q = np.exp(z - lse[:, None])
    g = np.where(some, dloss, 0.0)[:, None] / tau
    G = (Q - P) * g
    um = np.where(kept, np.abs(u), 0).max(axis=1, initial=0)
    du = 4 * U * (um + np.abs(M[:, 0])) + U * um
    return dict(z=z, lse=lse, loss=np.where(some, loss, 0), size=size, P=P, Q=Q, G=G, g=np.abs(g), p=p, at=at,
                dp=2 * du + 2.0 ** -21 + (k + 4) * U, dX=G @ W.T, dW=X.T @ G, k=k)


def check(got, X, W, r, dtype, tau):
    T, H, V, k = X.shape[0], X.shape[1], W.shape[1], r["k"]
    dz = (H + 2) * U * (np.abs(X) @ np.abs(W)) / tau + 3 * U * np.abs(r["z"])
    dlse = dz.max(axis=1) + 2.0 ** -19 + 2 * U * np.abs(r["lse"])
    assert (np.abs(got["lse"] - r["lse"]) <= dlse).all(), "lse"
    dzj = np.take_along_axis(dz, r["at"], 1)
    dloss = (r["dp"] + (k + 64) * U) * r["size"] + (r["p"] * (r["dp"][:, None] + dzj + dlse[:, None])).sum(axis=1)
    assert (np.abs(got["loss"] - r["loss"]) <= dloss).all(), "loss"
    if "dX" not in got:
        return
    dG = r["g"] * (r["Q"] * (2 * (dlse[:, None] + dz) + 2.0 ** -20) + r["P"] * r["dp"][:, None] + 2.0 ** -22)
    dG += unit(dtype) * (np.abs(r["G"]) + dG)
    mag = np.abs(r["G"]) + dG
    for name, sums in (("dX", dG @ np.abs(W).T + (V + 64) * U * (mag @ np.abs(W).T)),
                       ("dW", np.abs(X).T @ dG + (T + 64) * U * (np.abs(X).T @ mag))):
        bound = sums + unit(dtype) * (np.abs(r[name]) + sums)
        bad = np.abs(got[name] - r[name]) > bound
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside the bound"


def gpu(a):
    return torch().from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def run(ql, X, W, index, teacher, dloss, tau, by_vocab, pad=None):
    t = torch()
    Xd, Wd = to_device(X), to_device(W)
    if by_vocab:
        Wd = Wd.t().contiguous()
    if pad is not None:
        Xd, Wd = padded(Xd, Xd.shape[1] + pad), padded(Wd, Wd.shape[1] + pad)
    i, u, g = gpu(index), teacher if isinstance(teacher, t.Tensor) else gpu(teacher), gpu(dloss)
    loss, lse = ql.head_distill(Xd, Wd, i, u, tau, by_vocab=by_vocab)
    dX, dW = ql.head_distill_backward(Xd, Wd, i, u, lse, g, tau, by_vocab=by_vocab)
    t.cuda.synchronize()
    return dict(loss=loss, lse=lse, dX=dX, dW=dW.t().contiguous() if by_vocab else dW)


# rows, hidden, vocabulary, entries: each tile, the two ways to sort a list (up to 64
# entries, more) on both sides of their border, one entry, more entries than columns,
# vocabularies that are no multiple of 32
SHAPES = [(1, 1, 1, 1), (1, 64, 1000, 64), (3, 33, 5, 9), (31, 40, 131, 65), (64, 128, 257, 64), (65, 515, 300, 3),
          (130, 256, 1031, 100), (257, 96, 520, 1024), (300, 1032, 2056, 64), (20, 16, 4000, 1000)]


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
@pytest.mark.parametrize("T,H,V,k", SHAPES)
def test_distill(ql, T, H, V, k, dtype, by_vocab):
    X, W, index, teacher, dloss = inputs(T, H, V, k, dtype)
    X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
    for tau in (1.0, 2.5):
        log(f"distill {dtype} {T}x{H}x{V} {k} {'VxH' if by_vocab else 'HxV'} {tau}")
        got = as64(run(ql, X, W, index, teacher, dloss, tau, by_vocab))
        check(got, X64, W64, reference(X64, W64, index, teacher, dloss.astype(np.float64), tau), dtype, tau)


@pytest.mark.parametrize("T", [190, 600])
def test_distill_large_tiles_and_pieces(ql, T):
    """The largest tiles, and G in two pieces: the fewer rows as one of the others'."""
    t = torch()
    big = 2100
    H, V, k, tau = 136, 33000, 64, 2.0
    X, W, index, teacher, dloss = inputs(big, H, V, k, wl.BF16)
    index[0, 0], index[0, 1] = V - 1, 0
    log(f"distill in pieces {big}x{H}x{V}, {T} of them")
    all_rows = run(ql, X, W, index, teacher, dloss, tau, False)
    X64, W64 = X.f32[:T].astype(np.float64), W.f32.astype(np.float64)
    r = reference(X64, W64, index[:T], teacher[:T], dloss[:T].astype(np.float64), tau)
    got = {n: host(all_rows[n][:T].float()).astype(np.float64) for n in ("loss", "lse")}
    check(got, X64, W64, r, wl.BF16, tau)
    # all rows in float64 on the GPU (products of float64 matrices)
    Xd, Wd = to_device(X).double(), to_device(W).double()
    z = Xd @ Wd / tau
    lse = t.logsumexp(z, 1)
    idx = gpu(index).long()
    kept = (idx >= 0) & (idx < V)
    u = t.where(kept, gpu(teacher).double() / tau, -t.inf)
    some = kept.any(1)
    p = t.where(some[:, None], t.softmax(u, 1), 0.0)
    G = t.exp(z - lse[:, None])
    G.scatter_add_(1, t.where(kept, idx, 0), -p)
    G *= t.where(some, gpu(dloss).double() / tau, 0.0)[:, None]
    assert float((all_rows["lse"].double() - lse).abs().max()) <= 2.0 ** -17
    # one rounding of G and one of the result, half a step of 2^-7 each at most
    for name, want in (("dX", G @ Wd.t()), ("dW", Xd.t() @ G)):
        rel = float((all_rows[name].double() - want).norm() / want.norm())
        log(f"{name}: {rel:.2e}")
        assert rel <= 2.0 ** -8, f"{name}: {rel}"


@pytest.mark.parametrize("k", [40, 70])
def test_large_vocabulary(ql, k):
    """More groups of 32 columns than a list's threads count in one step (1024 and 4096)."""
    T, H, V = 3, 16, 140001
    X, W, index, teacher, dloss = inputs(T, H, V, k, wl.F32)
    index[:, :4] = [V - 1, 0, 131071, 131072]
    X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
    log(f"distill {T}x{H}x{V} {k}")
    got = as64(run(ql, X, W, index, teacher, dloss, 1.0, True))
    r = reference(X64, W64, index, teacher, dloss.astype(np.float64), 1.0)
    check(got, X64, W64, r, wl.F32, 1.0)


@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_one_entry_is_a_target(ql, dtype):
    """A list of one entry has probability 1: the head loss of that target.

    The logits are the same numbers in both (times 1), so the two lse differ by their
    sums alone, each 2^-19 + 2 U |lse| off that of these logits (see above): d. p is 1
    and its logarithm 0 exactly, so a loss is lse less the same logit, rounded once
    more: d + 2 U |loss|. Of G the softmax differs by the factor e^d - 1 < 2 d, and
    q - 1 is rounded before the product by dloss there and with it here, a rounding to
    the inputs' type at most on top: 2 d through |Q g|, and unit of the norm."""
    T, H, V = 140, 72, 333
    X, W, index, teacher, dloss = inputs(T, H, V, 1, dtype, left=0.2)
    t = torch()
    got = run(ql, X, W, index, teacher, dloss, 1.0, False)
    Xd, Wd, td = to_device(X), to_device(W), gpu(index[:, 0])
    loss, lse = ql.head_loss(Xd, Wd, td)
    dX, dW = ql.head_loss_backward(Xd, Wd, td, lse, gpu(dloss))
    t.cuda.synchronize()
    X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
    r = reference(X64, W64, index, teacher, dloss.astype(np.float64), 1.0)
    d = 2 * (2.0 ** -19 + 2 * U * np.abs(r["lse"]))
    a, b = as64(got), as64(dict(loss=loss, lse=lse, dX=dX, dW=dW))
    assert (np.abs(a["lse"] - b["lse"]) <= d).all()
    assert (np.abs(a["loss"] - b["loss"]) <= d + 2 * U * np.abs(b["loss"])).all()
    dG = 2 * d[:, None] * r["Q"] * r["g"]
    for name, more in (("dX", dG @ np.abs(W64).T), ("dW", np.abs(X64).T @ dG)):
        assert np.linalg.norm(a[name] - b[name]) <= unit(dtype) * np.linalg.norm(b[name]) + np.linalg.norm(more)


def test_bfloat16_teacher(ql):
    T, H, V, k = 50, 40, 600, 70
    X, W, index, teacher, dloss = inputs(T, H, V, k, wl.F32)
    u = gpu(teacher).bfloat16()
    a = run(ql, X, W, index, u, dloss, 2.0, False)
    b = run(ql, X, W, index, u.float(), dloss, 2.0, False)
    for n in a:
        assert_bits_equal(host(a[n]), host(b[n]), n)


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_left_out_rows_and_entries(ql, dtype, by_vocab):
    """Rows without an entry, by indices outside or teachers of -infinity: loss 0 and
    exactly no gradient, whatever X and dloss hold there; the others keep their bits."""
    T, H, V, k = 140, 67, 333, 20
    X, W, index, teacher, dloss = inputs(T, H, V, k, dtype)
    out = np.zeros(T, bool)
    out[::3] = True
    index[::6] = [-1, V] * (k // 2)
    teacher[3::6] = -np.inf
    teacher[1, :5] = -np.inf  # entries of a row that stays
    index[1, 5] = -7
    t = torch()
    want = run(ql, X, W, index, teacher, dloss, 2.0, by_vocab)
    log(f"distill {dtype}: {out.sum()} rows left out")
    assert not host(want["loss"])[out].any() and not host(want["dX"].float())[out].any()
    assert (host(want["loss"])[~out] != 0).all()
    zero = dloss.copy()
    zero[out] = 0
    X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
    check(as64(want), X64, W64, reference(X64, W64, index, teacher, zero.astype(np.float64), 2.0), dtype, 2.0)
    Xd, Wd = to_device(X).clone(), to_device(W)
    Wd = Wd.t().contiguous() if by_vocab else Wd
    gd = gpu(dloss)
    rows = gpu(np.nonzero(out)[0])
    for bad in (float("nan"), float("inf"), -float("inf")):
        Xd[rows] = bad
        gd[rows] = bad
        loss, lse = ql.head_distill(Xd, Wd, gpu(index), gpu(teacher), 2.0, by_vocab=by_vocab)
        dX, dW = ql.head_distill_backward(Xd, Wd, gpu(index), gpu(teacher), lse, gd, 2.0, by_vocab=by_vocab)
        dW = dW.t().contiguous() if by_vocab else dW
        assert_bits_equal(host(loss), host(want["loss"]), "loss")
        assert_bits_equal(host(lse)[~out], host(want["lse"])[~out], "lse")
        assert_bits_equal(host(dX), host(want["dX"]), "dX")
        assert_bits_equal(host(dW), host(want["dW"]), "dW")
    none = run(ql, X, W, np.full((T, k), -1, np.int32), teacher, dloss, 1.0, by_vocab)
    assert not host(none["loss"]).any() and not host(none["dX"].float()).any() and not host(none["dW"].float()).any()


@pytest.mark.parametrize("low", [-np.inf, np.finfo(np.float32).min, -1e30])
def test_masked_teacher_entries_are_as_if_not_listed(ql, low):
    """p = 0 at a student's logit of -infinity or NaN."""
    T, H, V, k = 30, 24, 100, 8
    X, W, index, teacher, dloss = inputs(T, H, V, k, wl.F32, left=0.0)
    index = np.stack([np.random.default_rng(i).permutation(V - 2)[:k] for i in range(T)]).astype(np.int32)
    with_mask = np.concatenate([index, np.full((T, 2), V - 1, np.int32)], 1)
    u = np.concatenate([teacher, np.full((T, 2), low, np.float32)], 1)
    Wx = W.f32.copy()
    Wx[:, V - 1] = 0
    Wm = wl.from_f32(Wx, wl.F32)
    a, b = run(ql, X, Wm, index, teacher, dloss, 0.5, False), run(ql, X, Wm, with_mask, u, dloss, 0.5, False)
    for n in a:
        assert_bits_equal(host(a[n]), host(b[n]), n)
    # the same place of the student at -infinity: X's first column 1, W's there -inf
    Xi = wl.from_f32(np.concatenate([np.ones((T, 1), np.float32), X.f32[:, 1:]], 1), wl.F32)
    Wx[0, V - 1] = -np.inf
    a, b = (ql.head_distill(to_device(Xi), to_device(wl.from_f32(Wx, wl.F32)), gpu(i), gpu(v), 0.5)
            for i, v in ((index, teacher), (with_mask, u)))
    assert np.isfinite(host(a[0])).all()
    for x, y in zip(a, b):
        assert_bits_equal(host(x), host(y), "loss, lse")
    # where the teacher has it, the loss is infinite
    has = index.copy()
    has[3, 2] = V - 1
    loss, _ = ql.head_distill(to_device(Xi), to_device(wl.from_f32(Wx, wl.F32)), gpu(has), gpu(teacher), 0.5)
    assert host(loss)[3] == np.inf and np.isfinite(np.delete(host(loss), 3)).all()


def test_rows_keep_to_themselves(ql):
    """A NaN in a teacher's list or in a row of X, an infinite dloss: that row's loss and
    dX and all of dW; every other row's loss and dX as without them."""
    T, H, V, k = 70, 40, 300, 10
    X, W, index, teacher, dloss = inputs(T, H, V, k, wl.BF16, left=0.0)
    dloss[:] = 0.5
    want = run(ql, X, W, index, teacher, dloss, 1.0, False)
    t = torch()
    teacher[5, 3], teacher[9, 0] = np.nan, np.inf
    dloss[33] = np.inf
    Xd, Wd = to_device(X).clone(), to_device(W)
    Xd[20] = float("nan")
    loss, lse = ql.head_distill(Xd, Wd, gpu(index), gpu(teacher))
    dX, dW = ql.head_distill_backward(Xd, Wd, gpu(index), gpu(teacher), lse, gpu(dloss))
    t.cuda.synchronize()
    rest = np.ones(T, bool)
    rest[[5, 9, 20]] = False
    assert np.isnan(host(loss)[~rest]).all()
    assert_bits_equal(host(loss)[rest], host(want["loss"])[rest], "loss")
    rest[33] = False
    d = host(dX.float())
    assert not np.isfinite(d[~rest]).any() and not np.isfinite(host(dW.float())).any()
    assert_bits_equal(d[rest], host(want["dX"].float())[rest], "dX")


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
def test_strides(ql, dtype, by_vocab):
    args = (*inputs(130, 96, 264, 12, dtype), 2.0, by_vocab)
    want = run(ql, *args)
    for pad in (8, 3):
        got = run(ql, *args, pad)
        for n in want:
            assert_bits_equal(host(got[n]), host(want[n]), n)


def test_difference_quotients(ql):
    """The gradients against differences of the loss itself, in float32: h = 2^-6, to 2^-8
    of the gradient's norm (curvature h^2 and rounding 2^-22 L / h)."""
    T, H, V, k = 20, 24, 50, 6
    X, W, index, teacher, dloss = inputs(T, H, V, k, wl.F32)
    rng = np.random.default_rng(11)
    base = run(ql, X, W, index, teacher, dloss, 1.5, False)
    t = torch()

    def total(x, w):
        loss, _ = ql.head_distill(x, w, gpu(index), gpu(teacher), 1.5)
        return float((loss.double() * gpu(dloss).double()).sum())

    Xd, Wd, h = to_device(X), to_device(W), 2.0 ** -6
    for _ in range(4):
        u = gpu(rng.standard_normal((T, H)).astype(np.float32))
        u /= u.norm()
        slope = (total(Xd + h * u, Wd) - total(Xd - h * u, Wd)) / (2 * h)
        assert abs(slope - float((base["dX"] * u).sum())) <= 2.0 ** -8 * float(base["dX"].norm())
        u = gpu(rng.standard_normal((H, V)).astype(np.float32))
        u /= u.norm()
        slope = (total(Xd, Wd + h * u) - total(Xd, Wd - h * u)) / (2 * h)
        assert abs(slope - float((base["dW"] * u).sum())) <= 2.0 ** -8 * float(base["dW"].norm())


def test_no_rows(ql):
    t = torch()
    for by_vocab in (False, True):
        W = t.randn((40, 72) if not by_vocab else (72, 40), device="cuda:0")
        X, i, u = t.empty((0, 40), device="cuda:0"), t.empty((0, 3), dtype=t.int32, device="cuda:0"), \
            t.empty((0, 3), device="cuda:0")
        loss, lse = ql.head_distill(X, W, i, u, by_vocab=by_vocab)
        assert loss.shape == (0,) and lse.shape == (0,)
        dX, dW = ql.head_distill_backward(X, W, i, u, lse, lse.clone(), by_vocab=by_vocab)
        assert dX.shape == (0, 40) and dW.shape == W.shape and not bool(dW.any())


def test_a_student_that_is_its_teacher(ql):
    """The teacher's own logits, all of them listed: the divergence is 0 up to the loss's
    bound, and so is its gradient."""
    T, H, V = 40, 32, 200
    X, W, _, _, dloss = inputs(T, H, V, 3, wl.F32)
    X64, W64 = X.f32.astype(np.float64), W.f32.astype(np.float64)
    teacher = (X64 @ W64).astype(np.float32)
    index = np.stack([np.random.default_rng(i).permutation(V) for i in range(T)]).astype(np.int32)
    teacher = np.take_along_axis(teacher, index, 1)
    got = as64(run(ql, X, W, index, teacher, dloss, 1.0, False))
    check(got, X64, W64, reference(X64, W64, index, teacher, dloss.astype(np.float64), 1.0), wl.F32, 1.0)
    assert np.abs(got["loss"]).max() < 1e-4
