"""GPU tests of what the binding accepts and refuses: strides that a single row
need not have, and buffers that do not fit a call."""
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


@pytest.mark.parametrize("length", [70000, 70001])
def test_one_row_of_a_long_sequence(ql, length):
    """The last position of one sequence, hidden[:, -1]: one row whose stride is
    the whole sequence, beyond the largest leading dimension."""
    t = torch()
    H, V, N = 65, 300, 40
    log(f"one row with a stride of {length * H}")
    hidden = t.randn((1, length, H), device="cuda:0").bfloat16()
    x = hidden[:, -1]
    assert x.stride(0) == length * H
    W = (t.randn((H, V), device="cuda:0") * 0.05).bfloat16()
    target, dloss = t.tensor([7], dtype=t.int32, device="cuda:0"), t.ones(1, device="cuda:0")
    y = x.clone(memory_format=t.contiguous_format)
    for a, b in zip(ql.head_loss(x, W, target), ql.head_loss(y, W, target)):
        assert_bits_equal(host(a), host(b), "loss")
    lse = ql.head_loss(y, W, target)[1]
    for a, b in zip(ql.head_loss_backward(x, W, target, lse, dloss), ql.head_loss_backward(y, W, target, lse, dloss)):
        assert_bits_equal(host(a), host(b), "gradients")
    E = t.randn((2, H, N), device="cuda:0").bfloat16()
    re = t.tensor([0, 1], dtype=t.int32, device="cuda:0")
    assert_bits_equal(host(ql.experts_forward_mx(x, E, re)), host(ql.experts_forward_mx(y, E, re)), "Y")


def test_weights_of_one_row_an_expert(ql):
    """K = 1: the row stride is the experts', whatever the middle stride says."""
    t = torch()
    E, N = 3, 24
    W = t.randn((E, 5, N), device="cuda:0")[:, 2:3]
    A, re = t.randn((4, 1), device="cuda:0"), t.tensor([1, 1, 4], dtype=t.int32, device="cuda:0")
    log("experts of one row each")
    want = ql.experts_forward_mx(A, W.contiguous(), re)
    assert_bits_equal(host(ql.experts_forward_mx(A, W, re)), host(want), "Y")


def test_clip_norm_buffer(ql):
    """norm takes one float32: other types and sizes are refused, and nothing is
    written then."""
    t = torch()
    g = t.full((100,), 3.0, device="cuda:0")
    ws = t.empty(ql.clip_workspace_bytes(1, 100), dtype=t.uint8, device="cuda:0")
    log("norm buffers of other types and sizes")
    for bad, error in ((t.zeros((), dtype=t.float64, device="cuda:0"), TypeError),
                       (t.zeros((), dtype=t.bfloat16, device="cuda:0"), TypeError),
                       (t.zeros(0, device="cuda:0"), ValueError), (t.zeros(2, device="cuda:0"), ValueError),
                       (t.zeros(()), ValueError)):
        with pytest.raises(error):
            ql.fp4lin_grad_norm([g], bad, ws)
        with pytest.raises(error):
            ql.fp4lin_clip_grads([g], 1.0, bad, ws)
        assert not bool(bad.any()) and bool((g == 3.0).all())
    for norm in (t.zeros((), device="cuda:0"), t.zeros((1, 1), device="cuda:0")):
        ql.fp4lin_grad_norm([g], norm, ws)
        assert float(norm) == 30.0


def test_packed_weight_buffers(ql):
    """Buffers for quantized weights that are too small are refused."""
    t = torch()
    W = t.randn((3, 130, 5), device="cuda:0")
    Wq, Ws = ql.experts_quantize_weight_mx(W)
    log("packed weights into given buffers")
    for q, s in ((Wq[:2], Ws), (Wq, Ws[:1]), (Wq[:, ::2], Ws)):
        with pytest.raises(ValueError):
            ql.fp4lin_experts_quantize_weight_mx(W, q, s)
    q, s = t.full_like(Wq, 255), t.full_like(Ws, 255)
    ql.fp4lin_experts_quantize_weight_mx(W, q, s)
    assert_bits_equal(host(q), host(Wq), "codes")
    assert_bits_equal(host(s), host(Ws), "scales")


def test_clip_refuses_shared_memory(ql):
    """Two workgroups would scale the same elements: an output listed twice, or one
    that is another output's gradient. The norm alone may count a tensor twice, and
    tensors without elements may share their address."""
    t = torch()
    a, b = t.full((100,), 3.0, device="cuda:0"), t.full((100,), 4.0, device="cuda:0")
    none = t.empty(0, device="cuda:0")
    log("clipping of shared memory")
    c, d = t.empty_like(a), t.empty_like(a)
    ws, norm = t.empty(4096, dtype=t.uint8, device="cuda:0"), t.zeros((), device="cuda:0")
    for grads, out in (([a, b, a], None), ([a, b], [c, c]), ([a, b], [b, c]), ([a, b], [b, a]), ([a, a], [a, c]),
                       ([a[1:]], [a[:-1]])):
        with pytest.raises(ql.Fp4linError):
            ql.clip_grads(grads, 1.0, out=out)
        with pytest.raises(ql.Fp4linError):
            ql.fp4lin_clip_grads(grads, 1.0, norm, ws, out=out)
    assert bool((a == 3.0).all()) and bool((b == 4.0).all())
    assert float(ql.grad_norm([a, a])) == pytest.approx(1800 ** 0.5)
    assert float(ql.clip_grads([a, none, b, none], 1e9, out=[c, none, d, none])) == 50.0
    assert t.equal(a, c) and t.equal(b, d)
    ql.clip_grads([a, a], 1e9, out=[c, d])
    ql.clip_grads([a, b, none], 1e9, out=[a, c, none])
    ql.clip_grads([none, a, none, b], 1e9)
    assert t.equal(b, c) and t.equal(a, d) and bool((a == 3.0).all())
