"""GPU tests of the experts' products at the sizes where each tile and quantizer
is taken, against a float64 reference on the GPU, and of the weights' forms that
serve few rows.

The reference quantizes from the definition (blocks of 32 along the reduction,
2^e the least power of two with 6 * 2^e >= the block's maximum, nearest E2M1
value, ties away from zero) and multiplies in float64, one expert at a time. An
element is held to the fp32 accumulation bound of the micro-scaled GEMM,
(2 * blocks + 2) * 2^-24 * sum of |terms|; a bfloat16 output is bit for bit the
fp32 one rounded once."""
import numpy as np
import pytest

import oracle as O
import workloads as wl
from gpu_util import assert_bits_equal, host, log, to_device

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


def quantized(x, dim):
    """x quantized in blocks of 32 along dim, as the values that the codes stand for."""
    t = torch()
    x = x.double().movedim(dim, -1)
    n = x.shape[-1]
    b = t.nn.functional.pad(x, (0, -n % 32)).unflatten(-1, (-1, 32))
    m, p = t.frexp(b.abs().amax(-1, keepdim=True) / 6.0)
    e = t.where(m == 0.5, p - 1, p)
    e = t.where(m == 0.0, -127, e).clamp(min=-127).double()
    y = b.abs() * t.exp2(-e)
    mids = t.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), dtype=t.float64, device=x.device)
    grid = t.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), dtype=t.float64, device=x.device)
    v = grid[t.bucketize(y.contiguous(), mids, right=True)] * t.exp2(e) * t.sign(b)
    return v.flatten(-2)[..., :n].movedim(-1, dim)


def randn(shape, dtype, seed, std=1.0):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return (t.randn(shape, generator=g, device="cuda") * std).to(dtype)


def activations(shape, dtype, seed):
    """Normal values, every 37th column 50 times as large."""
    x = randn(shape, torch().float32, seed)
    x[:, ::37] *= 50.0
    return x.to(dtype)


def ends_of(counts):
    return torch().tensor(np.cumsum(counts), dtype=torch().int32, device="cuda:0")


def spans(counts):
    at = 0
    for n in counts:
        yield at, at + n
        at += n


def assert_within(got, want, mag, L, what):
    """mag: the sum of the terms' magnitudes, L the length of the reduction."""
    blocks = -(-L // 128) * 4
    bad = (got.double() - want).abs() > (2 * blocks + 2) * 2.0 ** -24 * mag
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound"


def check_rows(got, x, weights, counts, along, what):
    """got: x's rows times their expert's matrix; weights[e] is quantized along
    dimension `along`, which the product runs over."""
    t = torch()
    L = x.shape[1]
    for e, (b, n) in enumerate(spans(counts)):
        if n > b:
            q, w = quantized(x[b:n], 1), quantized(weights[e], along)
            w = w if along == 0 else w.t()
            assert_within(got[b:n], q @ w, q.abs() @ w.abs(), L, f"{what}, expert {e}")
    assert not bool(t.any(got[sum(counts):])), f"{what}: rows past the last expert"


def test_reference_quantizes_as_the_oracle():
    pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    x = wl.random_matrix(rng, 70, 100, wl.F32, dist="t3")
    q = quantized(torch().from_numpy(x.f32.copy()), 1).numpy()
    _, _, codes, e = O.quantize_act_mx(x.f32)
    grid = np.array((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0))
    value = grid[codes % 8] * np.where(codes >= 8, -1.0, 1.0)
    scale = np.exp2(np.asarray(e, np.float64)).repeat(32, axis=1)[:, :value.shape[1]]
    assert np.array_equal(q, value * scale)


# rows an expert, rows past the last one, reduction, output columns
ROWS = {
    # 17 x 33 tiles of 256 x 256, five K steps
    "256x256": ([1500, 0, 2077, 1, 510], 12, 520, 8200),
    # 17 x 17 tiles of 128 x 256 (153 of 256 x 256), three K steps
    "128x256": ([700, 0, 1300, 91], 9, 300, 4100),
    # 64 x 128 tiles; 8 MiB of codes of the rows: four rows a thread
    "64x128, many rows": ([4000, 0, 4187], 10, 2048, 300),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ROWS)
def test_experts_rows_by_tile(ql, name, dtype):
    """Forward, apply and dgrad, in float32 and bfloat16 output."""
    t = torch()
    counts, extra, L, n = ROWS[name]
    M, E, dt = sum(counts) + extra, len(counts), t.bfloat16 if dtype == "bf16" else t.float32
    log(f"experts {name} {dtype}: {M} rows, {E} experts, {L} -> {n}")
    x, re = activations((M, L), dt, 3), ends_of(counts)
    W = randn((E, L, n), dt, 4, 0.02)
    Y = ql.experts_forward_mx(x, W, re)
    check_rows(Y, x, W, counts, 0, "forward")
    Yb = ql.experts_forward_mx(x, W, re, out_dtype=t.bfloat16)
    assert t.equal(Yb, Y.bfloat16()), "forward in bfloat16"
    Wq, Ws = ql.experts_quantize_weight_mx(W)
    Z = ql.experts_apply_mx(x, Wq, Ws, re)
    check_rows(Z, x, W, counts, 0, "apply")
    Zb = ql.experts_apply_mx(x, Wq, Ws, re, out_dtype=t.bfloat16)
    assert t.equal(Zb, Z.bfloat16()), "apply in bfloat16"
    del W, Wq, Ws, Y, Yb, Z, Zb
    V = randn((E, n, L), dt, 5, 0.02)  # dgrad's weights: reduction along their rows
    dX = ql.experts_dgrad_mx(x, V, re)
    check_rows(dX, x, V, counts, 1, "dgrad")
    dXb = ql.experts_dgrad_mx(x, V, re, out_dtype=t.bfloat16)
    assert t.equal(dXb, dX.bfloat16()), "dgrad in bfloat16"


@pytest.mark.parametrize("counts,extra", [([100, 0, 33, 200], 0), ([2000, 4, 0, 2100], 0)],
                         ids=["333 rows", "4104 rows"])
def test_experts_dgrad_of_many_weights(ql, counts, extra):
    """8 MiB of codes of the weights (and, with 4104 rows, of dY): four rows a
    thread, over matrices of 1030 rows, so that such four lie in two experts."""
    t = torch()
    E, K, N = len(counts), 1030, 4096
    log(f"experts dgrad of {E} x {K} x {N}, {sum(counts)} rows")
    dY, V, re = randn((sum(counts), N), t.bfloat16, 6, 1e-3), randn((E, K, N), t.bfloat16, 7, 0.02), ends_of(counts)
    check_rows(ql.experts_dgrad_mx(dY, V, re), dY, V, counts, 1, "dgrad")


@pytest.mark.parametrize("counts,extra,K,N", [([130, 0, 1, 64, 257, 33, 515, 128], 9, 2050, 2056),
                                              ([300, 0, 40], 0, 2050, 1100)],
                         ids=["256x256", "128x256"])
def test_experts_wgrad_by_tile(ql, counts, extra, K, N):
    """8 x 9 x 9 tiles of 256 x 256, one to five K steps; 3 x 17 x 5 of 128 x 256."""
    t = torch()
    M = sum(counts) + extra
    log(f"experts wgrad {K} x {N}, {M} rows of {len(counts)} experts")
    A, dY, re = activations((M, K), t.bfloat16, 8), randn((M, N), t.bfloat16, 9, 1e-3), ends_of(counts)
    dW = ql.experts_wgrad_mx(A, dY, re)
    for e, (b, n) in enumerate(spans(counts)):
        if n == b:
            assert not bool(dW[e].any())
            continue
        a, d = quantized(A[b:n], 0), quantized(dY[b:n], 0)
        assert_within(dW[e], a.t() @ d, a.abs().t() @ d.abs(), n - b, f"dW of expert {e}")
    assert t.equal(ql.experts_wgrad_mx(A, dY, re, out_dtype=t.bfloat16), dW.bfloat16())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,E,K,N", [(1, 3, 8192, 130), (1, 2, 4101, 40), (3, 2, 2050, 17), (16, 5, 512, 70),
                                     (64, 8, 515, 300)])
def test_experts_apply_spread_exponents(ql, M, E, K, N, dtype):
    """Blocks whose scales lie up to 2^24 apart, so that the fp32 sums round: four
    waves, eight waves (K > 4096) and tiles; float32 and bfloat16 output."""
    t = torch()
    rng = np.random.default_rng(M + K)
    counts = rng.multinomial(M, np.full(E, 1.0 / E)).tolist()
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    log(f"experts apply {dtype} {M}x{K}x{N}, rows {counts}")
    power = t.from_numpy(rng.integers(-12, 13, (M, -(-K // 32))).astype(np.float32)).to("cuda:0")
    x = (randn((M, K), t.float32, 10) * t.exp2(power).repeat_interleave(32, 1)[:, :K]).to(dt)
    W, re = randn((E, K, N), dt, 11, 0.02), ends_of(counts)
    Wq, Ws = ql.experts_quantize_weight_mx(W)
    Y = ql.experts_apply_mx(x, Wq, Ws, re)
    check_rows(Y, x, W, counts, 0, "apply")
    Yb = ql.experts_apply_mx(x, Wq, Ws, re, out_dtype=t.bfloat16)
    assert_bits_equal(host(Yb), host(Y.bfloat16()), "apply in bfloat16")
    check_rows(ql.experts_forward_mx(x, W, re), x, W, counts, 0, "forward")


@pytest.mark.parametrize("name", ["forward", "apply"])
def test_experts_offsets_near_32_bits(ql, name):
    """2.05 GB of codes of the rows: the offsets of rows outside an expert and of late
    K steps together pass 2^31. The rows around each expert's ends."""
    t = torch()
    counts, K, n = [250001, 0, 249990], 8192, 40
    M = sum(counts) + 7
    log(f"experts {name} of {M} x {K}")
    x = t.empty((M, K), dtype=t.bfloat16, device="cuda:0")
    g = t.Generator(device="cuda").manual_seed(12)
    for part in x.split(50000):
        part.copy_(t.randn(part.shape, generator=g, device="cuda"))
    W, re = randn((len(counts), K, n), t.bfloat16, 13, 0.02), ends_of(counts)
    if name == "apply":
        Y = ql.experts_apply_mx(x, *ql.experts_quantize_weight_mx(W), re)
    else:
        Y = ql.experts_forward_mx(x, W, re)
    assert not bool(Y[sum(counts):].any())
    for e, (b, end) in enumerate(spans(counts)):
        w = quantized(W[e], 0)
        for rows in (slice(b, min(b + 300, end)), slice(max(b, end - 300), end)):
            if rows.stop > rows.start:
                q = quantized(x[rows], 1)
                assert_within(Y[rows], q @ w, q.abs() @ w.abs(), K, f"expert {e}, rows {rows}")
