"""GPU tests of the rows' way to the experts and back against a plain implementation
in float64.

Bounds. A dispatch copies: bits are equal. A combine adds k products and the
residual in fp32: every one of its k + 1 roundings is at most U = 2^-24 of a partial
sum, which the sum of the magnitudes bounds, and the result is rounded once more to
the output's type (half a step: 2^-8 for bfloat16, 2^-24 for float32). dY is one
fp32 product, rounded to its type. dweight is an fp32 sum of H products of stored
values: at most H roundings of a partial sum."""
import numpy as np
import pytest

from gpu_util import assert_bits_equal, host, log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UNIT = {"bf16": 2.0 ** -8, "f32": U}


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


def types():
    t = torch()
    return {"bf16": t.bfloat16, "f32": t.float32}


def randn(rng, rows, cols, dtype, pad=0, offset=0):
    """A rows x cols matrix on the GPU with `pad` columns after each row, its first
    element `offset` elements into its memory; the rest of the memory is NaN."""
    t = torch()
    flat = t.full((offset + rows * (cols + pad),), float("nan"), dtype=types()[dtype], device="cuda")
    m = flat[offset:].view(rows, cols + pad)[:, :cols]
    m.copy_(t.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to("cuda"))
    return m


def f64(x):
    return x.detach().to("cpu").double().numpy()


def experts_of(rng, T, k, E, left, k1=False):
    """(T, k) experts, repeats among them; a part of the slots out of range on both sides."""
    e = rng.integers(0, E, (T, k))
    out = rng.random((T, k)) < left
    e[out] = rng.choice([-1, -(2 ** 31), E, E + 5, 2 ** 31 - 1], out.sum())
    e = e.astype(np.int32)
    return e[:, 0].copy() if k1 else e


def plan(expert, E):
    """(slot_row, row_end) by a stable sort."""
    key = expert.reshape(-1).astype(np.int64)
    key = np.where((key >= 0) & (key < E), key, E)
    order = np.argsort(key, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(order.size)
    return row.astype(np.int32), np.cumsum(np.bincount(key, minlength=E + 1)[:E]).astype(np.int32)


def to_gpu(a):
    return torch().from_numpy(np.ascontiguousarray(a)).to("cuda")


# tokens, slots, experts, columns, part left out: one token to many; one slot up to more
# than are read together; the two ways to sort (up to 1024 slots, more) on both sides of
# their border; rows narrower than a thread's group, odd, and longer than a workgroup's
SIZES = [(1, 1, 1, 1, 0.0), (1, 2, 8, 2048, 0.0), (3, 2, 4, 7, 0.5), (17, 4, 65, 64, 0.1), (64, 2, 8, 4096, 0.0),
         (128, 8, 16, 136, 0.0), (341, 3, 5, 515, 0.2), (342, 3, 5, 515, 0.2), (1001, 3, 5, 130, 0.1),
         (700, 5, 300, 33, 0.3), (200, 9, 7, 2056, 0.1), (50, 1, 3, 8193, 0.3), (2000, 1, 700, 24, 0.05),
         (4096, 2, 600, 40, 1.0), (5000, 2, 1, 16, 0.0), (9, 70, 5, 12, 0.2),
         (1, 2, 256, 48, 0.0), (1, 2, 257, 48, 0.0), (2, 3, 65534, 24, 0.3), (170, 3, 2000, 9, 0.1), (171, 3, 255, 9, 0.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,H,left", SIZES)
def test_dispatch(ql, T, k, E, H, left, dtype):
    rng = np.random.default_rng(T + 7 * k + 11 * H)
    log(f"dispatch {T} {k} {E} {H} {left} {dtype}")
    e = experts_of(rng, T, k, E, left)
    row, end = plan(e, E)
    for pad, offset in ((0, 0), (3, 1)):
        X = randn(rng, T, H, dtype, pad, offset)
        Xs, row_end, slot_row = ql.experts_dispatch(X, to_gpu(e), E)
        assert_bits_equal(host(slot_row).reshape(-1), row, "slot_row")
        assert_bits_equal(host(row_end), end, "row_end")
        want = np.zeros_like(host(Xs))
        kept = row < end[-1]
        want[row[kept]] = np.repeat(host(X), k, axis=0)[kept]
        assert_bits_equal(host(Xs), want, "Xs")


def combine_reference(Y, row, end, k, weight, residual):
    T = row.size // k
    out = np.zeros((T, Y.shape[1])) if residual is None else residual.copy()
    mag = np.abs(out)
    for j in range(k):
        r = row.reshape(T, k)[:, j]
        kept = r < end[-1]
        w = np.ones(T) if weight is None else weight.reshape(T, k)[:, j].astype(np.float64)
        out[kept] += w[kept, None] * Y[r[kept]]
        mag[kept] += np.abs(w[kept, None] * Y[r[kept]])
    return out, mag


@pytest.mark.parametrize("dtypes", ["bf16 bf16", "f32 bf16", "f32 f32", "bf16 f32"])
@pytest.mark.parametrize("T,k,E,H,left", SIZES)
def test_combine(ql, T, k, E, H, left, dtypes):
    ydt, odt = dtypes.split()
    rng = np.random.default_rng(T + 7 * k + 11 * H + 1)
    log(f"combine {T} {k} {E} {H} {left} {dtypes}")
    row, end = plan(experts_of(rng, T, k, E, left), E)
    for weighted, res, pad, offset in ((True, True, 0, 0), (True, False, 5, 3), (False, True, 1, 1),
                                       (False, False, 0, 0)):
        Y = randn(rng, T * k, H, ydt, pad, offset)
        Y[end[-1]:] = float("nan")  # rows that no expert has made have no part
        w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
        if weighted:
            w.reshape(-1)[row >= end[-1]] = np.inf
        r = randn(rng, T, H, odt, pad, offset) if res else None
        out = ql.experts_combine(Y, to_gpu(row.reshape(T, k)), to_gpu(end), None if w is None else to_gpu(w), r,
                                 out_dtype=types()[odt])
        want, mag = combine_reference(f64(Y), row, end, k, w, None if r is None else f64(r))
        bound = (k + 1) * U * mag
        bound += UNIT[odt] * (np.abs(want) + bound) + 2.0 ** -140
        assert (np.abs(f64(out) - want) <= bound).all(), (weighted, res)


def test_combine_in_place_of_its_residual(ql):
    rng = np.random.default_rng(5)
    T, k, E, H = 77, 2, 4, 523
    row, end = plan(experts_of(rng, T, k, E, 0.1), E)
    Y, r, w = randn(rng, T * k, H, "f32"), randn(rng, T, H, "bf16", 3, 1), to_gpu(rng.random((T, k), dtype=np.float32))
    args = (Y, to_gpu(row.reshape(T, k)), to_gpu(end))
    want = ql.experts_combine(*args, w, r)
    ql.fp4lin_experts_combine(*args, r, w, r)
    assert_bits_equal(host(r), host(want), "in place")


@pytest.mark.parametrize("dtypes", ["bf16 f32 bf16", "bf16 bf16 bf16", "f32 f32 f32", "f32 bf16 bf16", "bf16 f32 f32"])
@pytest.mark.parametrize("T,k,E,H,left", SIZES)
def test_combine_backward(ql, T, k, E, H, left, dtypes):
    """dout's, Y's and dY's types."""
    odt, ydt, gdt = dtypes.split()
    rng = np.random.default_rng(T + 7 * k + 11 * H + 2)
    log(f"combine backward {T} {k} {E} {H} {left} {dtypes}")
    row, end = plan(experts_of(rng, T, k, E, left), E)
    n = end[-1]
    kept = row < n
    for weighted, pad, offset in ((True, 0, 0), (True, 3, 1), (False, 0, 0)):
        d, Y = randn(rng, T, H, odt, pad, offset), randn(rng, T * k, H, ydt, pad, offset)
        Y[n:] = float("nan")
        w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
        if weighted:
            w.reshape(-1)[~kept] = np.nan
        dY, dw = ql.experts_combine_backward(d, Y if weighted else None, to_gpu(row.reshape(T, k)), to_gpu(end),
                                             None if w is None else to_gpu(w), out_dtype=types()[gdt])
        d64, Y64 = np.repeat(f64(d), k, axis=0)[kept], f64(Y)[row[kept]]
        want = np.zeros((T * k, H))
        want[row[kept]] = d64 if w is None else w.reshape(-1)[kept, None].astype(np.float64) * d64
        bound = U * np.abs(want)
        bound += UNIT[gdt] * (np.abs(want) + bound) + 2.0 ** -140
        assert (np.abs(f64(dY) - want) <= bound).all()
        if w is None:
            assert dw is None
            continue
        want, bound = np.zeros(T * k), np.zeros(T * k)
        want[kept] = (d64 * Y64).sum(1)
        bound[kept] = H * U * np.abs(d64 * Y64).sum(1)
        assert (np.abs(f64(dw).reshape(-1) - want) <= bound).all()


def test_gradients_by_differences(ql):
    """The gradient of a fixed linear function of the layer's output, float32: central
    differences of a function linear in X and in w are exact up to the roundings of the
    two values, at most (k + H + 4) * U of the magnitudes each, over the step."""
    t = torch()
    rng = np.random.default_rng(9)
    T, k, E, H = 13, 3, 4, 37
    e = to_gpu(experts_of(rng, T, k, E, 0.2))
    X, c = randn(rng, T, H, "f32"), randn(rng, T, H, "f32")
    w = to_gpu(rng.standard_normal((T, k)).astype(np.float32))

    def value(X, w):
        Xs, row_end, slot_row = ql.experts_dispatch(X, e, E)
        out = ql.experts_combine(Xs, slot_row, row_end, w)
        return float((out.double() * c.double()).sum()), (Xs, row_end, slot_row)

    _, (Xs, row_end, slot_row) = value(X, w)
    dXs, dw = ql.experts_combine_backward(c, Xs, slot_row, row_end, w)
    dX = ql.experts_combine(dXs, slot_row, row_end)
    step = 0.5
    size = float((t.abs(c).double() * ql.experts_combine(Xs.abs(), slot_row, row_end, w.abs()).double()).sum())
    size += step * float(c.abs().max() * (w.abs().sum() + X.abs().max() * k))
    tol = 2 * (k + H + 4) * U * size / (2 * step)
    for x, g in ((X, dX), (w, dw)):
        for at in [(0, 0), (5, 1), (12, 2), (7, 2)]:
            old = float(x[at])
            x[at] = old + step
            up, _ = value(X, w)
            x[at] = old - step
            down, _ = value(X, w)
            x[at] = old
            assert abs((up - down) / (2 * step) - float(g[at])) <= tol


def test_no_tokens(ql):
    t = torch()
    X = t.empty((0, 16), device="cuda")
    Xs, row_end, slot_row = ql.experts_dispatch(X, t.empty((0, 2), dtype=t.int32, device="cuda"), 5)
    assert Xs.shape == (0, 16) and row_end.tolist() == [0] * 5 and slot_row.shape == (0, 2)
    assert ql.experts_combine(Xs, slot_row, row_end).shape == (0, 16)
    dY, dw = ql.experts_combine_backward(X, Xs, slot_row, row_end, t.empty((0, 2), device="cuda"))
    assert dY.shape == (0, 16) and dw.shape == (0, 2)


def test_one_slot_vectors(ql):
    """expert as a vector: one slot a token."""
    rng = np.random.default_rng(3)
    e = experts_of(rng, 90, 1, 6, 0.1, k1=True)
    X = randn(rng, 90, 40, "bf16")
    a, b = ql.experts_dispatch(X, to_gpu(e), 6), ql.experts_dispatch(X, to_gpu(e[:, None]), 6)
    assert a[2].shape == (90,)
    for x, y in zip(a, b):
        assert_bits_equal(host(x).reshape(-1), host(y).reshape(-1), "one slot")


def test_wrong_rows_are_left_out(ql):
    """Rows outside the M are as slots that carry nothing, a last end past M as M."""
    t = torch()
    T, k, H = 20, 2, 24
    rng = np.random.default_rng(8)
    Y, d = randn(rng, T * k, H, "f32"), randn(rng, T, H, "f32")
    row = np.arange(T * k, dtype=np.int32)
    row[3], row[6], row[10] = -1, T * k, 2 ** 31 - 1
    end = to_gpu(np.array([7, 10 ** 6], np.int32))
    out = ql.experts_combine(Y, to_gpu(row.reshape(T, k)), end)
    want = f64(Y)
    want[[3, 6, 10]] = 0
    assert np.abs(f64(out) - want.reshape(T, k, H).sum(1)).max() <= 2 * U * np.abs(want).max() * k
    dY = t.full((T * k, H), 7.0, device="cuda")
    dw = t.full((T, k), 7.0, device="cuda")
    ql.fp4lin_experts_combine_backward(d, Y, to_gpu(row.reshape(T, k)), end, dY, None, dw)
    want = np.repeat(f64(d), k, axis=0)
    want[[3, 6, 10]] = 7.0  # rows that no slot names
    assert_bits_equal(host(dY), want.astype(np.float32), "dY")
    assert (host(dw).reshape(-1)[[3, 6, 10]] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_of_experts(ql, dtype):
    """The calls together, as a layer's training step makes them: the products take the
    rows, ends and zeros of the dispatch as they are, and every result is that of the
    same calls on rows sorted by torch."""
    t = torch()
    T, k, E, H, N = 150, 2, 4, 128, 96
    rng = np.random.default_rng(21)
    e = experts_of(rng, T, k, E, 0.05)
    row, end = plan(e, E)
    X, d = randn(rng, T, H, dtype), randn(rng, T, H, dtype)
    up, down = (to_gpu(rng.standard_normal(s).astype(np.float32) * 0.1).to(X.dtype) for s in ((E, H, N), (E, N, H)))
    w = to_gpu(rng.random((T, k), dtype=np.float32))
    Xs, row_end, slot_row = ql.experts_dispatch(X, to_gpu(e), E)
    sorted_rows = t.zeros_like(Xs)
    kept = row < end[-1]
    sorted_rows[to_gpu(row[kept]).long()] = X.repeat_interleave(k, 0)[to_gpu(kept)]
    assert_bits_equal(host(Xs), host(sorted_rows), "rows")
    u = ql.experts_forward_mx(Xs, up, row_end, out_dtype=X.dtype)
    Y = ql.experts_forward_mx(u, down, row_end)
    out = ql.experts_combine(Y, slot_row, row_end, w, X)
    assert out.dtype == X.dtype
    dY, dw = ql.experts_combine_backward(d, Y, slot_row, row_end, w)
    ddown = ql.experts_wgrad_mx(u, dY, row_end)
    du = ql.experts_dgrad_mx(dY, down, row_end, out_dtype=X.dtype)
    dup = ql.experts_wgrad_mx(Xs, du, row_end)
    dXs = ql.experts_dgrad_mx(du, up, row_end, out_dtype=X.dtype)
    dX = ql.experts_combine(dXs, slot_row, row_end, residual=d)
    end_t = to_gpu(end)
    u2 = ql.experts_forward_mx(sorted_rows, up, end_t, out_dtype=X.dtype)
    Y2 = ql.experts_forward_mx(u2, down, end_t)
    assert_bits_equal(host(Y), host(Y2), "products")
    want, mag = combine_reference(f64(Y2), row, end, k, host(w), f64(X))
    bound = (k + 1) * U * mag
    assert (np.abs(f64(out) - want) <= bound + UNIT[dtype] * (np.abs(want) + bound)).all()
    want, mag = combine_reference(f64(dXs), row, end, k, None, f64(d))
    bound = (k + 1) * U * mag
    assert (np.abs(f64(dX) - want) <= bound + UNIT[dtype] * (np.abs(want) + bound)).all()
    for g in (dup, ddown, dw):
        assert t.isfinite(g).all()


def test_rows_past_32_bit_offsets(ql):
    """Xs of more than 2^31 elements: the last expert's rows."""
    t = torch()
    T, k, H, E = 1 << 18, 2, 4104, 3
    e = t.zeros((T, k), dtype=t.int32, device="cuda")
    e[:, 1] = 2
    e[-1, 1] = 7
    X = t.empty((T, H), dtype=t.bfloat16, device="cuda")
    X.copy_(t.arange(T, device="cuda").remainder(251).to(t.bfloat16).unsqueeze(1).expand(T, H))
    Xs, row_end, slot_row = ql.experts_dispatch(X, e, E)
    assert row_end.tolist() == [T, T, 2 * T - 1]
    assert int(slot_row[-1, 1]) == 2 * T - 1 and int(slot_row[5, 1]) == T + 5
    assert bool((Xs[:T] == X).all()) and bool((Xs[T:-1] == X[:-1]).all()) and bool((Xs[-1] == 0).all())
    out = ql.experts_combine(Xs, slot_row, row_end)
    assert bool((out[:-1] == 2 * X[:-1]).all()) and bool((out[-1] == X[-1]).all())
    dY, _ = ql.experts_combine_backward(X, None, slot_row, row_end)
    assert bool((dY == Xs).all())
