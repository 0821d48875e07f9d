"""GPU parity of the products grouped by expert (fp4lin_experts_*_mx) against
the CPU oracle, one expert at a time: quantize the expert's rows (for the
weight gradient: its columns, in blocks counted from its first row) and multiply
in float64.

Codes and scale bytes are bit-exact. An output element is held to the fp32
accumulation bound of the micro-scaled GEMM, (2 * blocks + 2) * 2^-24 * sum of
|block terms|, plus half a unit in the last place where the output is bfloat16
(2^-8 of its magnitude)."""
import numpy as np
import pytest

import oracle as O
import workloads as wl
from gpu_util import assert_bits_equal, host, log, padded, to_device

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


def ends_of(counts):
    return np.cumsum(np.asarray(counts), dtype=np.int64).astype(np.int32)


def upload_ends(ends):
    return torch().from_numpy(np.asarray(ends, np.int32)).to("cuda:0")


def groups(ends, M):
    """[(begin, end)] of each expert as the kernels read row_end."""
    out, at = [], 0
    for n in ends:
        n = max(at, min(max(int(n), 0), M))
        out.append((at, n))
        at = n
    return out


def stack3(parts, dtype):
    """Host matrices (one an expert) as one 3-D device tensor."""
    t = torch().stack([to_device(p) for p in parts])
    return t


def bound(mag, L, want, bf16):
    blocks = O.packed_ld(L) // 16
    b = (2 * blocks + 2) * 2.0 ** -24 * mag
    return b + (2.0 ** -8 * (np.abs(want) + b) if bf16 else 0.0)


def assert_within(got, want, mag, L, bf16, what):
    bad = np.abs(got - want) > bound(mag, L, want, bf16)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} elements outside the bound"


def as64(t):
    return host(t.float()).astype(np.float64)


def expect_rows(X32, W32s, ends, transposed):
    """(Y, |terms|) of forward (transposed false: W along its rows) or dgrad."""
    M = X32.shape[0]
    n = W32s[0].shape[0 if transposed else 1]
    y, mag = np.zeros((M, n)), np.zeros((M, n))
    for (b, e), W in zip(groups(ends, M), W32s):
        if e > b:
            qx = O.quantize_act_mx(X32[b:e])
            qw = O.quantize_act_mx(W) if transposed else O.quantize_weight_mx(W)
            y[b:e], mag[b:e] = O.mx_product(qx[2], qx[3], qw[2], qw[3])
    return y, mag


def expect_wgrad(A32, dY32, ends):
    out = []
    M, K, N = A32.shape[0], A32.shape[1], dY32.shape[1]
    for b, e in groups(ends, M):
        if e > b:
            out.append(O.wgrad_mx(A32[b:e], dY32[b:e])[:2])
        else:
            out.append((np.zeros((K, N)), np.zeros((K, N))))
    return out


# counts of rows an expert (some experts empty), rows past the last expert, K, N
SHAPES = [
    ([1], 0, 1, 1),
    ([2, 0, 1], 0, 33, 17),
    ([0, 0, 5], 0, 129, 260),
    ([16, 1, 0, 17, 3], 2, 515, 130),
    ([40, 0, 75, 33], 0, 300, 515),
    ([130, 257, 0, 64], 9, 200, 300),
    ([300, 5, 520], 0, 640, 264),
    ([3] * 70 + [0] * 3 + [40], 0, 96, 40),
]


def make(shape, dtype, seed=0):
    counts, extra, K, N = shape
    rng = np.random.default_rng(seed + sum(counts) + K + N)
    M = sum(counts) + extra
    A = wl.random_matrix(rng, M, K, dtype, dist="t3")
    dY = wl.random_matrix(rng, M, N, dtype, scale=1e-3)
    W = [wl.random_matrix(rng, K, N, dtype, scale=0.02) for _ in counts]
    return A, dY, W, ends_of(counts)


@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{sum(s[0])}x{s[2]}x{s[3]}")
def test_experts_forward_dgrad_wgrad(ql, shape, dtype):
    A, dY, W, ends = make(shape, dtype)
    log(f"experts {dtype} {shape}")
    K, N = shape[2], shape[3]
    Ad, dYd, Wd, re = to_device(A), to_device(dY), stack3(W, dtype), upload_ends(ends)
    Y = ql.experts_forward_mx(Ad, Wd, re)
    dX = ql.experts_dgrad_mx(dYd, Wd, re)
    dW = ql.experts_wgrad_mx(Ad, dYd, re)
    torch().cuda.synchronize()
    want, mag = expect_rows(A.f32, [w.f32 for w in W], ends, False)
    assert_within(as64(Y), want, mag, K, False, "Y")
    want, mag = expect_rows(dY.f32, [w.f32 for w in W], ends, True)
    assert_within(as64(dX), want, mag, N, False, "dX")
    got = as64(dW)
    for e, (want, mag) in enumerate(expect_wgrad(A.f32, dY.f32, ends)):
        assert_within(got[e], want, mag, A.shape[0], False, f"dW of expert {e}")


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[5], SHAPES[6]], ids=["few", "tiles", "large"])
def test_experts_bf16_outputs(ql, shape):
    A, dY, W, ends = make(shape, wl.BF16, 1)
    log(f"experts bf16 outputs {shape}")
    bf = torch().bfloat16
    Ad, dYd, Wd, re = to_device(A), to_device(dY), stack3(W, wl.BF16), upload_ends(ends)
    Y = ql.experts_forward_mx(Ad, Wd, re, out_dtype=bf)
    dX = ql.experts_dgrad_mx(dYd, Wd, re, out_dtype=bf)
    dW = ql.experts_wgrad_mx(Ad, dYd, re, out_dtype=bf)
    # the same sums as the fp32 outputs, rounded once
    assert_bits_equal(host(Y), host(ql.experts_forward_mx(Ad, Wd, re).to(bf)), "Y")
    assert_bits_equal(host(dX), host(ql.experts_dgrad_mx(dYd, Wd, re).to(bf)), "dX")
    assert_bits_equal(host(dW), host(ql.experts_wgrad_mx(Ad, dYd, re).to(bf)), "dW")


@pytest.mark.parametrize("dtype", [wl.F32, wl.BF16])
@pytest.mark.parametrize("M,E,K,N", [(1, 1, 64, 40), (2, 8, 2048, 130), (5, 3, 1030, 17),
                                     (64, 8, 515, 300), (200, 4, 260, 515)])
def test_experts_apply(ql, M, E, K, N, dtype):
    """Weights quantized before: codes and scale bytes bit for bit the oracle's
    of each expert, and the product that of experts_forward_mx."""
    log(f"experts apply {dtype} {M}x{K}x{N}, {E} experts")
    rng = np.random.default_rng(M + E + K + N)
    counts = rng.multinomial(M, np.full(E, 1.0 / E))
    ends = ends_of(counts)
    A = wl.random_matrix(rng, M, K, dtype, dist="t3")
    W = [wl.random_matrix(rng, K, N, dtype, scale=0.02) for _ in range(E)]
    Ad, Wd, re = to_device(A), stack3(W, dtype), upload_ends(ends)
    Wq, Ws = ql.experts_quantize_weight_mx(Wd)
    for e in range(E):
        q = O.quantize_weight_mx(W[e].f32)
        assert_bits_equal(host(Wq)[e], q[0], f"codes of expert {e}")
        s = host(Ws)[:, e].transpose(1, 0, 2).reshape(N, -1)
        assert_bits_equal(s, q[1], f"scale bytes of expert {e}")
    Y = ql.experts_apply_mx(Ad, Wq, Ws, re)
    want, mag = expect_rows(A.f32, [w.f32 for w in W], ends, False)
    assert_within(as64(Y), want, mag, K, False, "Y")
    assert_bits_equal(host(Y), host(ql.experts_forward_mx(Ad, Wd, re)), "Y against the forward")


@pytest.mark.parametrize("M,counts", [(40, [10, 30]), (700, [200, 500])])
def test_experts_strides(ql, M, counts):
    """Row strides that are wider than the rows, aligned and not, in and out."""
    K, N = 200, 264
    rng = np.random.default_rng(M)
    A = wl.random_matrix(rng, M, K, wl.BF16, dist="t3")
    dY = wl.random_matrix(rng, M, N, wl.BF16, scale=1e-3)
    W = [wl.random_matrix(rng, K, N, wl.BF16, scale=0.02) for _ in counts]
    re = upload_ends(ends_of(counts))
    Ad, dYd, Wd = to_device(A), to_device(dY), stack3(W, wl.BF16)
    Y, dX, dW = (ql.experts_forward_mx(Ad, Wd, re), ql.experts_dgrad_mx(dYd, Wd, re),
                 ql.experts_wgrad_mx(Ad, dYd, re))
    t = torch()
    for pad in (8, 3):
        log(f"experts strides {M} rows, {pad} more columns")
        Ap, dYp = padded(Ad, K + pad), padded(dYd, N + pad)
        Wp = padded(Wd.reshape(-1, N), N + pad).unflatten(0, (len(counts), K))
        assert_bits_equal(host(ql.experts_forward_mx(Ap, Wp, re)), host(Y), "Y")
        assert_bits_equal(host(ql.experts_dgrad_mx(dYp, Wp, re)), host(dX), "dX")
        assert_bits_equal(host(ql.experts_wgrad_mx(Ap, dYp, re)), host(dW), "dW")
        # outputs into wider buffers: nothing past a row's end is written
        out = t.full((M, N + pad), 7.0, device="cuda:0")
        ws = t.empty(ql.experts_workspace_bytes(0, len(counts), M, K, N), dtype=t.uint8, device="cuda:0")
        ql.fp4lin_experts_forward_mx(Ap, Wp, re, out[:, :N], ws)
        assert_bits_equal(host(out[:, :N].contiguous()), host(Y), "Y in a wider buffer")
        assert bool((out[:, N:] == 7.0).all())


@pytest.mark.parametrize("M", [24, 300])
def test_experts_row_end_is_clamped(ql, M):
    """Ends that descend, are negative or lie past M read as a running maximum
    in [0, M]; the rows past the last end are zeros."""
    K, N = 96, 130
    rng = np.random.default_rng(M)
    A = wl.random_matrix(rng, M, K, wl.F32)
    dY = wl.random_matrix(rng, M, N, wl.F32)
    W = [wl.random_matrix(rng, K, N, wl.F32, scale=0.02) for _ in range(4)]
    Ad, dYd, Wd = to_device(A), to_device(dY), stack3(W, wl.F32)
    for ends in ([5, 3, M - 6, M - 8], [-4, 7, 2 ** 31 - 1, 1], [0, 0, 0, 0], [M, M, M, M]):
        log(f"experts ends {ends} of {M}")
        re = upload_ends(ends)
        want, mag = expect_rows(A.f32, [w.f32 for w in W], ends, False)
        got = as64(ql.experts_forward_mx(Ad, Wd, re))
        assert_within(got, want, mag, K, False, "Y")
        assert not got[groups(ends, M)[-1][1]:].any()
        dW = as64(ql.experts_wgrad_mx(Ad, dYd, re))
        for e, (want, mag) in enumerate(expect_wgrad(A.f32, dY.f32, ends)):
            assert_within(dW[e], want, mag, M, False, f"dW of expert {e}")


@pytest.mark.parametrize("M", [16, 300])
def test_experts_rows_keep_to_themselves(ql, M):
    """Infinities and NaN past the last expert's end reach nothing, those of one
    expert's rows none of the others' results."""
    K, N = 256, 130
    rng = np.random.default_rng(M + 1)
    A = wl.random_matrix(rng, M, K, wl.F32)
    dY = wl.random_matrix(rng, M, N, wl.F32)
    W = [wl.random_matrix(rng, K, N, wl.F32, scale=0.02) for _ in range(3)]
    ends = [M // 4, M // 4 + 5, M - 3]
    Ad, dYd, Wd, re = to_device(A), to_device(dY), stack3(W, wl.F32), upload_ends(ends)
    Wq, Ws = ql.experts_quantize_weight_mx(Wd)

    def all_of():
        return (ql.experts_forward_mx(Ad, Wd, re), ql.experts_apply_mx(Ad, Wq, Ws, re),
                ql.experts_dgrad_mx(dYd, Wd, re), ql.experts_wgrad_mx(Ad, dYd, re))

    want = [host(x) for x in all_of()]
    for bad in (float("nan"), float("inf"), -float("inf")):
        log(f"experts {M} rows, {bad} past the last end, then in one expert")
        Ad[ends[2]:], dYd[ends[2]:] = bad, bad
        for name, x, y in zip(("Y", "Y applied", "dX", "dW"), all_of(), want):
            assert_bits_equal(host(x), y, name)
        saved = Ad[ends[0]:ends[1]].clone(), dYd[ends[0]:ends[1]].clone()
        Ad[ends[0]:ends[1]], dYd[ends[0]:ends[1]] = bad, bad
        *rows, dW = (host(x) for x in all_of())
        for name, x, y in zip(("Y", "Y applied", "dX"), rows, want):
            assert_bits_equal(x[:ends[0]], y[:ends[0]], name)
            assert_bits_equal(x[ends[1]:], y[ends[1]:], name)
        for e in (0, 2):
            assert_bits_equal(dW[e], want[3][e], f"dW of expert {e}")
        Ad[ends[0]:ends[1]], dYd[ends[0]:ends[1]] = saved


def test_experts_no_rows(ql):
    """A batch without rows: empty outputs, a zero weight gradient."""
    t = torch()
    E, K, N = 3, 40, 70
    W = t.randn((E, K, N), device="cuda:0")
    re = upload_ends([0] * E)
    A, dY = t.empty((0, K), device="cuda:0"), t.empty((0, N), device="cuda:0")
    assert ql.experts_forward_mx(A, W, re).shape == (0, N)
    assert ql.experts_dgrad_mx(dY, W, re).shape == (0, K)
    Wq, Ws = ql.experts_quantize_weight_mx(W)
    assert ql.experts_apply_mx(A, Wq, Ws, re).shape == (0, N)
    dW = ql.experts_wgrad_mx(A, dY, re)
    assert dW.shape == (E, K, N) and not bool(dW.any())


def test_experts_match_the_layer_calls(ql):
    """One expert with all rows is the micro-scaled layer of the public calls."""
    M, K, N = 700, 300, 520
    rng = np.random.default_rng(9)
    A = wl.random_matrix(rng, M, K, wl.BF16, dist="t3")
    W = wl.random_matrix(rng, K, N, wl.BF16, scale=0.02)
    Ad, Wd = to_device(A), to_device(W)
    aq, asc = ql.quantize_act_mx(Ad)
    wq, wsc = ql.quantize_weight_mx(Wd)
    want = ql.gemm_mx(aq, asc, wq, wsc, M, N, K)
    got = ql.experts_forward_mx(Ad, Wd.unsqueeze(0), upload_ends([M]))
    assert_bits_equal(host(got), host(want), "Y")


def test_experts_stream_and_graph(ql):
    """On a stream of the caller's, and captured in a graph that is replayed
    with eager work between."""
    t = torch()
    shape = ([40, 0, 75, 33], 4, 300, 264)
    A, dY, W, ends = make(shape, wl.BF16, 3)
    Ad, dYd, Wd, re = to_device(A), to_device(dY), stack3(W, wl.BF16), upload_ends(ends)
    want = host(ql.experts_forward_mx(Ad, Wd, re)), host(ql.experts_wgrad_mx(Ad, dYd, re))
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    Y = ql.experts_forward_mx(Ad, Wd, re, stream=s)
    t.cuda.current_stream().wait_stream(s)
    t.cuda.synchronize()
    assert_bits_equal(host(Y), want[0], "Y on a stream")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        Y = ql.experts_forward_mx(Ad, Wd, re)
        dW = ql.experts_wgrad_mx(Ad, dYd, re)
    for k in range(3):
        log(f"experts graph replay {k}")
        Y.zero_()
        dW.fill_(3.0)
        g.replay()
        t.cuda.synchronize()
        assert_bits_equal(host(Y), want[0], f"Y of replay {k}")
        assert_bits_equal(host(dW), want[1], f"dW of replay {k}")
        assert_bits_equal(host(ql.experts_forward_mx(Ad, Wd, re)), want[0], "Y")


def test_experts_binding_refusals(ql):
    t = torch()
    dev = "cuda:0"
    A, W = t.zeros((4, 32), device=dev), t.zeros((2, 32, 16), device=dev)
    re = upload_ends([2, 4])
    with pytest.raises(ValueError):
        ql.experts_forward_mx(A[:, :31], W, re)
    with pytest.raises(ValueError):
        ql.experts_forward_mx(A, W, re[:1])
    with pytest.raises(TypeError):
        ql.experts_forward_mx(A, W, re.long())
    with pytest.raises(TypeError):
        ql.experts_forward_mx(A.bfloat16(), W, re)
    with pytest.raises(TypeError):
        ql.experts_forward_mx(A.half(), W.half(), re)
    with pytest.raises(ValueError):
        ql.experts_forward_mx(A, W.transpose(1, 2), re)
    with pytest.raises(ValueError):
        ql.experts_forward_mx(A.cpu(), W, re)
    with pytest.raises(ValueError):
        ql.experts_wgrad_mx(A, t.zeros((3, 16), device=dev), re)
    Wq, Ws = ql.experts_quantize_weight_mx(W)
    with pytest.raises(ValueError):
        ql.experts_apply_mx(A, Wq[:, :, :32].contiguous(), Ws, re)
    ws = t.empty(16, dtype=t.uint8, device=dev)
    with pytest.raises(ql.Fp4linError):
        ql.fp4lin_experts_forward_mx(A, W, re, t.empty((4, 16), device=dev), ws)
