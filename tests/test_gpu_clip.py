"""GPU tests of the global gradient norm and clipping against float64.

The norm is a double sum rounded once to float: 2^-23 relative. The coefficient
is an fp32 quotient of it (2^-22), an output one product more and the rounding to
its type."""
import math

import numpy as np
import pytest

from gpu_util import assert_bits_equal, host, log

pytestmark = pytest.mark.gpu


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


def make(sizes, dtypes, seed=0, std=1.0):
    t = torch()
    g = t.Generator().manual_seed(seed)
    return [(t.randn(n, generator=g) * std).to(d).to("cuda:0") for n, d in zip(sizes, dtypes)]


def expected_norm(tensors):
    return math.sqrt(math.fsum(float(x.double().square().sum()) for x in tensors))


def check(ql, tensors, max_norm):
    t = torch()
    before = [x.clone() for x in tensors]
    norm64 = expected_norm(tensors)
    c = min(1.0, max_norm / (norm64 + 1e-6))
    assert abs(float(ql.grad_norm(tensors)) - norm64) <= 2.0 ** -23 * norm64
    out = [t.full_like(x, 9.0) for x in tensors]
    norm = ql.clip_grads(tensors, max_norm, out=out)
    assert abs(float(norm) - norm64) <= 2.0 ** -23 * norm64
    for x, b, o in zip(tensors, before, out):
        assert t.equal(x, b), "gradients were written"
        want = b.double() * c
        unit = 2.0 ** -8 if x.dtype == t.bfloat16 else 2.0 ** -22
        lim = (unit + 2.0 ** -21) * want.abs() + 2.0 ** -126
        assert bool(((o.double() - want).abs() <= lim).all())
    norm2 = ql.clip_grads(tensors, max_norm)
    assert_bits_equal(host(norm2), host(norm), "norm in place")
    for x, o in zip(tensors, out):
        assert t.equal(x, o), "in place and out of place differ"


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [0, 5, 0], [8191, 8192, 8193, 1, 100000],
                                   [3000001, 17], [33] * 300])
def test_clip(ql, sizes, max_norm):
    t = torch()
    log(f"clip {len(sizes)} tensors of {sum(sizes)} elements, max_norm {max_norm}")
    kinds = [t.float32, t.bfloat16]
    check(ql, make(sizes, [kinds[i % 2] for i in range(len(sizes))]), max_norm)


def test_clip_unaligned_and_shaped(ql):
    """Views that start off 16 bytes, transposed (dense) tensors, scalars."""
    t = torch()
    base = make([5000, 5001], [t.float32, t.bfloat16])
    views = [base[0][1:4000], base[1][3:4999], make([1200], [t.float32], 3)[0].view(30, 40).t(),
             make([1], [t.bfloat16], 4)[0].reshape(())]
    log("clip unaligned views")
    norm64 = expected_norm(views)
    rest = base[0][:1].clone(), base[0][4000:].clone(), base[1][:3].clone()
    want = [v.double() * (0.25 / (norm64 + 1e-6)) for v in views]
    norm = ql.clip_grads(views, 0.25)
    assert abs(float(norm) - norm64) <= 2.0 ** -23 * norm64
    for v, w in zip(views, want):
        unit = 2.0 ** -8 if v.dtype == t.bfloat16 else 2.0 ** -21
        assert bool(((v.double() - w).abs() <= unit * w.abs()).all())
    assert t.equal(rest[0], base[0][:1]) and t.equal(rest[1], base[0][4000:])
    assert t.equal(rest[2], base[1][:3])


def test_clip_extreme_values(ql):
    """Squares beyond fp32's range on both sides; infinities and NaN as the
    formula gives them; all zeros."""
    t = torch()
    for v in (1e30, 1e-30):
        log(f"clip values of {v}")
        x = t.full((5000,), v, device="cuda:0")
        assert abs(float(ql.grad_norm([x])) / (v * math.sqrt(5000)) - 1) <= 2.0 ** -20
    x = t.full((100,), 1e30, device="cuda:0")
    ql.clip_grads([x], 1.0)
    assert bool(((x - 0.1).abs() < 1e-6).all())
    z = t.zeros(1000, device="cuda:0")
    assert float(ql.clip_grads([z], 1.0)) == 0.0 and not bool(z.any())
    y = t.ones(1000, device="cuda:0")
    y[17] = float("inf")
    assert float(ql.clip_grads([y, z], 1.0)) == float("inf")
    assert math.isnan(float(y[17])) and not bool(y[:17].any()) and not bool(z.any())
    y = t.ones(1000, device="cuda:0")
    y[999] = float("nan")
    w = t.ones(10, device="cuda:0", dtype=t.bfloat16)
    assert math.isnan(float(ql.clip_grads([y, w], 1.0)))
    assert bool(y.isnan().all()) and bool(w.isnan().all())


def test_clip_repeats_stream_and_graph(ql):
    t = torch()
    tensors = make([100000, 31, 70000], [t.float32, t.bfloat16, t.bfloat16])
    out = [t.empty_like(x) for x in tensors]
    want = host(ql.clip_grads(tensors, 1.0, out=out)), [host(o) for o in out]
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    norm = ql.clip_grads(tensors, 1.0, out=out, stream=s)
    t.cuda.current_stream().wait_stream(s)
    t.cuda.synchronize()
    assert_bits_equal(host(norm), want[0], "norm on a stream")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        norm = ql.clip_grads(tensors, 1.0, out=out)
    for k in range(3):
        log(f"clip graph replay {k}")
        norm.fill_(-1.0)
        for o in out:
            o.zero_()
        g.replay()
        t.cuda.synchronize()
        assert_bits_equal(host(norm), want[0], "norm of a replay")
        for o, w in zip(out, want[1]):
            assert_bits_equal(host(o), w, "output of a replay")
        ql.grad_norm(tensors)


def test_clip_binding_refusals(ql):
    t = torch()
    x = t.ones((4, 6), device="cuda:0")
    with pytest.raises(ValueError):
        ql.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        ql.clip_grads([x[:, :3]], 1.0)
    with pytest.raises(ValueError):
        ql.clip_grads([x.cpu()], 1.0)
    with pytest.raises(TypeError):
        ql.clip_grads([x.half()], 1.0)
    with pytest.raises(TypeError):
        ql.clip_grads([x], 1.0, out=[x.bfloat16()])
    with pytest.raises(ValueError):
        ql.clip_grads([x], 1.0, out=[])
    with pytest.raises(ValueError):
        ql.clip_grads([x], 1.0, out=[t.empty((6, 4), device="cuda:0")])
    for bad in (float("nan"), -1.0):
        with pytest.raises(ql.Fp4linError):
            ql.clip_grads([x], bad)
    assert bool((x == 1).all())
