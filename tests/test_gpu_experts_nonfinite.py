"""GPU tests of infinities and NaN in the operands of the experts' products: the
block of 32 that holds one has no scale (byte 255), so that every element of the
result that the block has a part in is NaN, in each form of each product, and
every other element keeps its bits."""
import numpy as np
import pytest

from gpu_util import assert_bits_equal, host, log

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]


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


def same_but(got, want, nan, what):
    """got is NaN exactly where `nan` says, and bit for bit want elsewhere."""
    t = torch()
    assert t.equal(got.isnan(), nan), f"{what}: {int(got.isnan().sum())} NaN, not {int(nan.sum())}"
    assert t.equal(got[~nan], want[~nan]), what


def make(M, K, N, dtype):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(M + K + N)
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    A = t.randn((M, K), generator=g, device="cuda").to(dt)
    dY = (t.randn((M, N), generator=g, device="cuda") * 1e-3).to(dt)
    W = (t.randn((3, K, N), generator=g, device="cuda") * 0.02).to(dt)
    ends = [M // 4, M // 4, M - 2]
    return A, dY, W, ends, t.tensor(ends, dtype=t.int32, device="cuda")


# 12 rows of 256: the forms for few rows; 300 of 261: tiles and unaligned loads;
# 8300 of 2056: four rows a thread in the row quantizers
SIZES = [(12, 256, 130), (300, 261, 136), (8300, 2056, 4096)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_nonfinite_activation(ql, M, K, N, dtype):
    t = torch()
    A, dY, W, ends, re = make(M, K, N, dtype)
    W[:, :, 5] = 0.0  # a product with zeros is NaN as well
    Wq, Ws = ql.experts_quantize_weight_mx(W)

    def results():
        return (ql.experts_forward_mx(A, W, re), ql.experts_apply_mx(A, Wq, Ws, re),
                ql.experts_forward_mx(A, W, re, out_dtype=t.bfloat16), ql.experts_wgrad_mx(A, dY, re))

    want = results()
    row, col = ends[0] + 1, K - 3
    nan = t.zeros((M, N), dtype=t.bool, device="cuda")
    nan[row] = True
    nan_w = t.zeros((3, K, N), dtype=t.bool, device="cuda")
    nan_w[2, col] = True
    saved = A[row, col].item()
    for bad in BAD:
        log(f"experts {dtype} {M}x{K}x{N}: {bad} in A")
        A[row, col] = bad
        got = results()
        for name, x, y in zip(("forward", "apply", "forward in bfloat16"), got, want):
            same_but(x, y, nan, name)
        same_but(got[3], want[3], nan_w, "wgrad")
    A[row, col] = saved


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_nonfinite_gradient(ql, M, K, N, dtype):
    t = torch()
    A, dY, W, ends, re = make(M, K, N, dtype)
    want = ql.experts_dgrad_mx(dY, W, re), ql.experts_wgrad_mx(A, dY, re)
    row, col = ends[0] - 1, N - 1
    nan = t.zeros((M, K), dtype=t.bool, device="cuda")
    nan[row] = True
    nan_w = t.zeros((3, K, N), dtype=t.bool, device="cuda")
    nan_w[0, :, col] = True
    for bad in BAD:
        log(f"experts {dtype} {M}x{K}x{N}: {bad} in dY")
        dY[row, col] = bad
        same_but(ql.experts_dgrad_mx(dY, W, re), want[0], nan, "dgrad")
        same_but(ql.experts_wgrad_mx(A, dY, re), want[1], nan_w, "wgrad")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_nonfinite_weight(ql, M, K, N, dtype):
    t = torch()
    A, dY, W, ends, re = make(M, K, N, dtype)

    def results():
        Wq, Ws = ql.experts_quantize_weight_mx(W)
        return (ql.experts_forward_mx(A, W, re), ql.experts_apply_mx(A, Wq, Ws, re),
                ql.experts_dgrad_mx(dY, W, re), Ws)

    want = results()
    k, n = 33, N - 2
    nan = t.zeros((M, N), dtype=t.bool, device="cuda")
    nan[ends[1]:ends[2], n] = True
    nan_x = t.zeros((M, K), dtype=t.bool, device="cuda")
    nan_x[ends[1]:ends[2], k] = True
    for bad in BAD:
        log(f"experts {dtype} {M}x{K}x{N}: {bad} in W")
        W[2, k, n] = bad
        got = results()
        same_but(got[0], want[0], nan, "forward")
        same_but(got[1], want[1], nan, "apply")
        same_but(got[2], want[2], nan_x, "dgrad")
        scales = host(want[3]).copy()
        scales[k // 128, 2, n, k // 32 % 4] = 255
        assert_bits_equal(host(got[3]), scales, "scale bytes")
