"""GPU tests of infinite logits in the head loss: -infinity is a probability of 0,
+infinity makes NaN of its row alone (its gradients: of its dX and of dW)."""
import pytest

from gpu_util import log

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


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [20, 200])
def test_column_of_minus_infinity(ql, T, dtype, by_vocab):
    """W[3, 17] = -inf and positive X[:, 3]: the losses are those without column 17 (a
    logit is off by at most (H + 2) * 2^-24 * sum |x w| =: d, a loss by 2 d + 2^-18),
    +infinity where it is the target; dX is not finite in column 3 alone, dW finite."""
    t = torch()
    H, V = 40, 300
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    log(f"head loss {dtype}, {T} rows, a column of -inf")
    g = t.Generator(device="cuda").manual_seed(T)
    X = t.randn((T, H), generator=g, device="cuda").to(dt)
    X[:, 3] = X[:, 3].abs() + 0.5
    W = (t.randn((H, V), generator=g, device="cuda") * 0.1).to(dt)
    W[3, 17] = -float("inf")
    target = t.randint(0, V, (T,), generator=g, device="cuda", dtype=t.int32)
    target[target == 17] = 18
    target[5] = 17
    Wd = W.t().contiguous() if by_vocab else W
    loss, lse = ql.head_loss(X, Wd, target, by_vocab=by_vocab)
    rest = [v for v in range(V) if v != 17]
    l = X.double() @ W[:, rest].double()
    want = t.logsumexp(l, 1)
    d = (H + 2) * 2.0 ** -24 * (X.double().abs() @ W[:, rest].double().abs()).amax(1)
    assert bool(((lse.double() - want).abs() <= d + 2.0 ** -19).all())
    at = target.long() - (target > 17).long()
    want -= l.gather(1, at.clamp(max=V - 2)[:, None])[:, 0]
    others = t.arange(T, device="cuda") != 5
    assert bool(((loss.double() - want).abs() <= 2 * d + 2.0 ** -18)[others].all())
    assert float(loss[5]) == float("inf")
    dX, dW = ql.head_loss_backward(X, Wd, target, lse, t.ones_like(loss), by_vocab=by_vocab)
    # the product with W[3, 17] = -inf: G = 0 (NaN), in row 5 G = -1 (+inf)
    assert bool(dX[:, 3][others].isnan().all()) and float(dX[5, 3]) == float("inf")
    assert bool(dW.isfinite().all())
    assert bool(t.cat((dX[:, :3], dX[:, 4:]), 1).isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_row_of_infinity(ql, dtype, value):
    """One X[6, 3] = inf (or NaN), W[3, :] positive in one column only: that row's loss
    and dX are NaN, and dW; no other row's."""
    t = torch()
    T, H, V = 70, 40, 300
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    log(f"head loss {dtype}, a logit of {value}")
    g = t.Generator(device="cuda").manual_seed(7)
    X = t.randn((T, H), generator=g, device="cuda").to(dt)
    W = (t.randn((H, V), generator=g, device="cuda") * 0.1).to(dt)
    W[3] = -1.0
    W[3, 44] = 1.0
    target = t.randint(0, V, (T,), generator=g, device="cuda", dtype=t.int32)
    want = ql.head_loss(X, W, target)[0]
    X[6, 3] = value
    loss, lse = ql.head_loss(X, W, target)
    others = t.arange(T, device="cuda") != 6
    assert bool(loss[6].isnan()) and t.equal(loss[others], want[others])
    dX, dW = ql.head_loss_backward(X, W, target, lse, t.ones_like(loss))
    assert bool(dX[6].isnan().all()) and bool(dX[others].isfinite().all())
    assert bool(dW.isnan().all())
