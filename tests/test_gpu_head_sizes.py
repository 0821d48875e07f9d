"""GPU tests of the head loss and its gradients at the sizes where each tile, split
and piece is taken, against float64 on the GPU, element by element.

Bounds (as for the small sizes): a logit of reduction H is an fp32 sum of exact
(bfloat16) or rounded products, off by at most (H + 2) * 2^-24 * sum |x w| =: dl;
lse by dl + 2^-19 and the final rounding 2^-21; the loss by twice that; G by
|g| * (p * (2 * that + 2^-20) + 2^-23) and its rounding to the inputs' type; dX and
dW by G's bound through |W| or |X|, an fp32 sum of n terms (slices and pieces added
once each: n + 64 roundings) and the result's rounding to the inputs' type."""
import pytest

from gpu_util import log

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


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound"


def check(ql, T, H, V, dtype, by_vocab):
    t = torch()
    log(f"head loss {dtype} {T}x{H}x{V} {'VxH' if by_vocab else 'HxV'}")
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    g = t.Generator(device="cuda").manual_seed(T + H + V)
    X = t.randn((T, H), generator=g, device="cuda").to(dt)
    W = (t.randn((V, H) if by_vocab else (H, V), generator=g, device="cuda") * 0.02).to(dt)
    target = t.randint(0, V, (T,), generator=g, device="cuda", dtype=t.int32)
    target[5::11] = -100
    target[3] = V - 1
    dloss = t.randn((T,), generator=g, device="cuda") / T
    loss, lse = ql.head_loss(X, W, target, by_vocab=by_vocab)
    dX, dW = ql.head_loss_backward(X, W, target, lse, dloss, by_vocab=by_vocab)
    if by_vocab:
        W, dW = W.t(), dW.t()
    # float64
    X, W = X.double(), W.double()
    l = X @ W
    want_lse = t.logsumexp(l, 1)
    dl = (H + 2) * U * (X.abs() @ W.abs())
    dlse = dl.amax(1) + 2.0 ** -19 + 2.0 ** -21
    within(lse, want_lse, dlse, "lse")
    keep = (target >= 0) & (target < V)
    at = t.where(keep, target, 0).long()[:, None]
    want = t.where(keep, want_lse - l.gather(1, at)[:, 0], 0.0)
    within(loss, want, dlse + dl.amax(1) + 2.0 ** -20, "loss")
    P = t.exp(l - want_lse[:, None])
    del l
    gr = t.where(keep, dloss.double(), 0.0)[:, None]
    dG = gr.abs() * (P * (2 * (dlse[:, None] + dl) + 2.0 ** -20) + 2.0 ** -23)
    del dl
    G = P.scatter_add_(1, at, t.full_like(at, -1, dtype=t.float64)).mul_(gr)
    unit = 2.0 ** -8 if dtype == "bf16" else U
    dG += unit * (G.abs() + dG)
    mag = G.abs() + dG
    for name, got, want, err, terms, n in (
            ("dX", dX, G @ W.t(), dG @ W.abs().t(), mag @ W.abs().t(), V),
            ("dW", dW, X.t() @ G, X.abs().t() @ dG, X.abs().t() @ mag, T)):
        err += (n + 64) * U * terms
        within(got, want, err + unit * (want.abs() + err), name)
    assert not bool(dX[~keep].any())


@pytest.mark.parametrize("by_vocab", [False, True], ids=["HxV", "VxH"])
@pytest.mark.parametrize("T,H,V,dtype", [
    # 9 x 33 tiles of 256 x 256 of dW, ten K steps; dX of the same tiles in 15 slices
    (300, 2056, 8200, "bf16"),
    # 17 x 17 tiles of 256 x 256 of dX, unsplit, over two pieces of the vocabulary
    (4100, 4104, 17000, "bf16"),
    # two pieces, the second ending inside a tile, and dX in slices
    (2100, 136, 33001, "bf16"),
    # float32: two pieces (H = 40: dX in slices, 64 x 64 tiles)
    (1100, 40, 33000, "f32"),
    # float32 128 x 128 tiles of the logits, dX (two slices) and dW, nothing a multiple
    (2040, 2043, 2041, "f32"),
])
def test_head_loss_by_tile(ql, T, H, V, dtype, by_vocab):
    check(ql, T, H, V, dtype, by_vocab)
