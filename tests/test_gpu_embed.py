"""GPU tests of the embedding and its gradient against a plain implementation in
float64.

Bounds (U = 2^-24, the roundings to a type at half a step: 2^-8 for bfloat16). The
lookup is one fp32 product by the scale (itself rounded to fp32: one U more) and
its rounding. A row of the gradient adds n rows in fp32, pieces of a long list
first: at most n roundings of partial sums that the sum of the magnitudes bounds,
then the scale and its rounding, what was there, and the rounding to the type."""
import numpy as np
import pytest

from gpu_util import assert_bits_equal, host, log
from test_gpu_route import UNIT, U, f64, randn, to_gpu, types

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_linear_layer_amd as q
    q.lib()
    return q


def tokens_of(rng, T, V, kind):
    if kind == "uniform":
        t = rng.integers(0, V, T)
    elif kind == "text":
        t = rng.permutation(V)[np.minimum(rng.zipf(1.3, T) - 1, V - 1)]
    elif kind == "same":
        t = np.full(T, V // 2)
    elif kind == "low":  # all in the first keys
        t = rng.integers(0, min(V, 97), T)
    else:
        t = np.sort(rng.integers(0, V, T))
    out = rng.random(T) < (0.0 if kind == "same" else 0.1)
    t[out] = rng.choice([-1, V, V + 9, -(2 ** 31), 2 ** 31 - 1], out.sum())
    return t.astype(np.int32)


@pytest.mark.parametrize("dtypes", ["bf16 bf16", "f32 f32", "bf16 f32", "f32 bf16"])
@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 1000, 2048), (64, 300, 515), (1000, 77, 40), (33, 5, 4104)])
def test_lookup(ql, T, V, H, dtypes):
    dt, odt = dtypes.split()
    rng = np.random.default_rng(T + V + H)
    log(f"embed {T} {V} {H} {dtypes}")
    tok = tokens_of(rng, T, V, "uniform")
    kept = (tok >= 0) & (tok < V)
    for scale, pad, offset in ((1.0, 0, 0), (H ** 0.5, 3, 1), (-0.3, 0, 0), (0.0, 0, 0)):
        E = randn(rng, V, H, dt, pad, offset)
        out = ql.embed(E, to_gpu(tok), scale, out_dtype=types()[odt])
        want = np.zeros((T, H))
        want[kept] = f64(E)[tok[kept]] * scale
        bound = 2 * U * np.abs(want)
        bound += UNIT[odt] * (np.abs(want) + bound) + 2.0 ** -140
        assert (np.abs(f64(out) - want) <= bound).all(), scale
        if scale == 1.0 and dt == odt:
            assert_bits_equal(host(out)[kept], host(E)[tok[kept]], "rows")


def test_lookup_shape(ql):
    rng = np.random.default_rng(1)
    E = randn(rng, 50, 24, "bf16")
    tok = tokens_of(rng, 12, 50, "uniform")
    out = ql.embed(E, to_gpu(tok.reshape(3, 4)))
    assert out.shape == (3, 4, 24)
    assert_bits_equal(host(out.view(12, 24)), host(ql.embed(E, to_gpu(tok))), "batch")


def gradient(dX, tok, V, scale, base=None):
    """(dE, bound before the last rounding) in float64."""
    kept = (tok >= 0) & (tok < V)
    d, mag, n = np.zeros((V, dX.shape[1])), np.zeros((V, dX.shape[1])), np.zeros(V)
    np.add.at(d, tok[kept], dX[kept])
    np.add.at(mag, tok[kept], np.abs(dX[kept]))
    np.add.at(n, tok[kept], 1)
    bound = (n[:, None] + 3) * U * abs(scale) * mag
    d *= scale
    if base is not None:
        d += base
        bound += U * (np.abs(d) + bound)
    return d, bound, n


# positions, vocabulary, columns: no piece, lists at and past a piece's length, one
# piece more; a vocabulary of one, of more than a workgroup's keys each, of less
BACK = [(1, 1, 1, "uniform"), (1, 1000, 2048, "uniform"), (32, 3, 40, "same"), (33, 3, 40, "same"), (65, 1, 515, "same"),
        (1000, 77, 33, "uniform"), (1001, 5003, 515, "text"), (4096, 3000, 64, "text"), (8192, 2, 16, "uniform"),
        (2000, 40000, 24, "low"), (3000, 300, 4104, "sorted"), (5000, 131100, 8, "uniform"), (1025, 257, 9, "text"),
        # few positions, in one launch: at and past the most of them, and the most rows of one
        # token that a thread may come to add; slices of a long list, sweeps over the columns,
        # rows that end inside a group of eight; many rows to fill
        (256, 50, 515, "same"), (257, 50, 515, "text"), (256, 50, 500, "same"), (256, 9, 2048, "same"),
        (255, 9, 2049, "text"), (128, 9, 4096, "same"), (129, 9, 4096, "same"), (64, 9, 8192, "low"),
        (32, 9, 8200, "same"), (33, 9, 8200, "same"), (256, 40000, 8, "uniform"), (200, 5000, 130, "low"),
        (128, 70000, 264, "text"), (8, 3, 2048, "same"), (9, 3, 1000, "same"), (256, 1, 7, "same"),
        (100, 2, 17, "low"), (1000, 50, 515, "same"), (384, 9, 2048, "same"), (1024, 40000, 8, "uniform")]


@pytest.mark.parametrize("dtypes", ["bf16 bf16", "f32 f32", "bf16 f32", "f32 bf16"])
@pytest.mark.parametrize("T,V,H,kind", BACK)
def test_gradient(ql, T, V, H, kind, dtypes):
    dt, edt = dtypes.split()
    rng = np.random.default_rng(T + V + H)
    log(f"embed backward {T} {V} {H} {kind} {dtypes}")
    tok = tokens_of(rng, T, V, kind)
    left = (tok < 0) | (tok >= V)
    for scale, pad, offset in ((1.0, 0, 0), (H ** 0.5, 3, 1)):
        dX = randn(rng, T, H, dt, pad, offset)
        dX[to_gpu(left)] = float("nan")  # no part
        got = ql.embed_backward(dX, to_gpu(tok), V, scale, out_dtype=types()[edt])
        want, bound, n = gradient(f64(dX), tok, V, scale)
        bound += UNIT[edt] * (np.abs(want) + bound) + 2.0 ** -140
        assert (np.abs(f64(got) - want) <= bound).all()
        assert not host(got)[n == 0].any()
        # again: the same bits; and on top of a gradient, whose other rows stay
        assert_bits_equal(host(ql.embed_backward(dX, to_gpu(tok), V, scale, out_dtype=types()[edt])), host(got), "again")
        base = randn(rng, V, H, edt, pad, offset)
        old = host(base).copy()
        base64 = f64(base)
        assert ql.embed_backward(dX, to_gpu(tok), V, scale, add_to=base) is base
        want, bound, n = gradient(f64(dX), tok, V, scale, base64)
        bound += UNIT[edt] * (np.abs(want) + bound) + 2.0 ** -140
        ok = np.abs(f64(base) - want) <= bound
        assert ok[n > 0].all()
        assert_bits_equal(host(base)[n == 0], old[n == 0], "rows without a position")


def test_gradient_by_differences(ql):
    """The lookup is linear in the table: central differences are exact up to the two
    values' roundings (2 U of the magnitudes each) over the step."""
    rng = np.random.default_rng(4)
    T, V, H, step = 40, 9, 11, 0.5
    tok = to_gpu(tokens_of(rng, T, V, "uniform"))
    E, c = randn(rng, V, H, "f32"), randn(rng, T, H, "f32")
    g = ql.embed_backward(c, tok, V, 1.7)
    size = float((ql.embed(E.abs(), tok, 1.7) * c.abs()).double().sum()) + 1.7 * step * float(c.abs().sum())
    for at in [(0, 0), (3, 10), (8, 5), (4, 4)]:
        old = float(E[at])
        values = []
        for x in (old + step, old - step):
            E[at] = x
            values.append(float((ql.embed(E, tok, 1.7).double() * c.double()).sum()))
        E[at] = old
        assert abs((values[0] - values[1]) / (2 * step) - float(g[at])) <= (4 / (2 * step) + T) * U * size


def test_no_positions(ql):
    import torch as t
    none = t.empty(0, dtype=t.int32, device="cuda")
    assert ql.embed(t.ones((5, 3), device="cuda"), none).shape == (0, 3)
    d = ql.embed_backward(t.empty((0, 3), device="cuda"), none, 5)
    assert d.shape == (5, 3) and not host(d).any()
    base = t.ones((5, 3), device="cuda")
    ql.embed_backward(t.empty((0, 3), device="cuda"), none, 5, add_to=base)
    assert (host(base) == 1).all()


def test_tied_with_the_head(ql):
    """The table shared with the head: its gradient of the loss and of the lookup in one
    array, as a training step of a tied model leaves it."""
    import torch as t
    rng = np.random.default_rng(6)
    T, V, H = 70, 130, 48
    E = randn(rng, V, H, "f32")
    tok, target = (to_gpu(tokens_of(rng, T, V, "uniform")) for _ in range(2))
    X = ql.embed(E, tok, 2.0)
    loss, lse = ql.head_loss(X, E, target, by_vocab=True)
    dloss = t.full_like(loss, 1.0 / T)
    dX, dE = ql.head_loss_backward(X, E, target, lse, dloss, by_vocab=True)
    head = f64(dE)
    ql.embed_backward(dX, tok, V, 2.0, add_to=dE)
    want, bound, _ = gradient(f64(dX), host(tok), V, 2.0, head)
    assert (np.abs(f64(dE) - want) <= bound + U * (np.abs(want) + bound)).all()


def test_rows_past_32_bit_offsets(ql):
    """A table of more than 2^31 elements."""
    import torch as t
    V, H = 530000, 4096
    E = t.empty((V, H), dtype=t.bfloat16, device="cuda")
    E.copy_(t.arange(V, device="cuda").remainder(253).to(t.bfloat16).unsqueeze(1).expand(V, H))
    tok = t.tensor([V - 1, 0, 524289, V - 1, V, 524287], dtype=t.int32, device="cuda")
    out = ql.embed(E, tok)
    assert out[:, 7].float().tolist() == [(V - 1) % 253, 0, 524289 % 253, (V - 1) % 253, 0, 524287 % 253]
    d = ql.embed_backward(out, tok, V)
    assert bool((d[V - 1] == 2 * out[0]).all()) and bool((d[524289] == out[2]).all())
    assert bool((d[524287] == out[5]).all()) and float(d[1:524287].float().abs().max()) == 0
