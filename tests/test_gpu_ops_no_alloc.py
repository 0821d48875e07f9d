"""GPU tests that the raw calls of the experts' products, the head loss and the
clipping allocate nothing and can be captured: neither the device's free memory nor
the number of torch's allocations changes over them, and a graph of all of them,
replayed with eager work between, gives the eager results bit for bit."""
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


class Step:
    """Buffers for one call of each entry, on given inputs."""

    def __init__(self, ql, dtype, M, few):
        import torch as t
        self.ql, E, K, N, H, V, T = ql, 3, 200, 136, 72, 1000, 90
        g = t.Generator(device="cuda").manual_seed(M)

        def randn(*shape):
            return t.randn(shape, generator=g, device="cuda").to(dtype)

        def empty(*shape, dtype=t.float32):
            return t.empty(shape, device="cuda", dtype=dtype)

        def ws(n):
            assert n > 0
            return empty(n, dtype=t.uint8)

        self.A, self.dY, self.W = randn(M, K), randn(M, N), randn(E, K, N)
        self.a = randn(few, K)
        self.re = t.tensor([M // 3, M // 3, M - 1], dtype=t.int32, device="cuda")
        self.few_re = t.tensor([0, few - 1, few], dtype=t.int32, device="cuda")
        steps = (K + 127) // 128
        self.Wq, self.Ws = empty(E, N, steps * 64, dtype=t.uint8), empty(steps, E, N, 4, dtype=t.uint8)
        self.Y, self.Yb, self.Z, self.z = empty(M, N), empty(M, N, dtype=t.bfloat16), empty(M, N), empty(few, N)
        self.dX, self.dW = empty(M, K), empty(E, K, N)
        self.ws = [ws(ql.experts_workspace_bytes(p, E, M, K, N)) for p in range(4)]
        self.few_ws = ws(ql.experts_workspace_bytes(3, E, few, K, N))
        self.X, self.Wh, self.target = randn(T, H), randn(H, V), t.randint(0, V, (T,), generator=g, device="cuda",
                                                                          dtype=t.int32)
        self.loss, self.lse, self.dloss = empty(T), empty(T), t.ones(T, device="cuda")
        self.dXh, self.dWh = empty(T, H, dtype=dtype), empty(H, V, dtype=dtype)
        code = ql.BF16 if dtype == t.bfloat16 else ql.F32
        self.head_ws = [ws(ql.head_loss_workspace_bytes(code, False, T, H, V, H, V, b)) for b in (False, True)]
        self.grads = [self.dXh, self.dWh, self.dW, self.dX]
        self.out = [t.empty_like(x) for x in self.grads]
        self.clip_ws = ws(ql.clip_workspace_bytes(4, sum(x.numel() for x in self.grads)))
        self.norm, self.norm2 = empty(), empty()

    def run(self):
        q = self.ql
        q.fp4lin_experts_forward_mx(self.A, self.W, self.re, self.Y, self.ws[0])
        q.fp4lin_experts_forward_mx(self.A, self.W, self.re, self.Yb, self.ws[0])
        q.fp4lin_experts_quantize_weight_mx(self.W, self.Wq, self.Ws)
        q.fp4lin_experts_apply_mx(self.A, self.Wq, self.Ws, self.re, self.Z, self.ws[3])
        q.fp4lin_experts_apply_mx(self.a, self.Wq, self.Ws, self.few_re, self.z, self.few_ws)
        q.fp4lin_experts_dgrad_mx(self.dY, self.W, self.re, self.dX, self.ws[1])
        q.fp4lin_experts_wgrad_mx(self.A, self.dY, self.re, self.dW, self.ws[2])
        q.fp4lin_head_loss(self.X, self.Wh, self.target, self.loss, self.lse, self.head_ws[0])
        q.fp4lin_head_loss_backward(self.X, self.Wh, self.target, self.lse, self.dloss, self.dXh, self.dWh,
                                    self.head_ws[1])
        q.fp4lin_grad_norm(self.grads, self.norm, self.clip_ws)
        q.fp4lin_clip_grads(self.grads, 0.5, self.norm2, self.clip_ws, out=self.out)

    def results(self):
        return [self.Y, self.Yb, self.Wq, self.Ws, self.Z, self.z, self.dX, self.dW, self.loss, self.lse, self.dXh,
                self.dWh, self.norm, self.norm2, *self.out]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_raw_calls_allocate_nothing(ql, dtype):
    import torch as t
    s = Step(ql, t.bfloat16 if dtype == "bf16" else t.float32, 300, 4)
    s.run()  # loads the kernels
    t.cuda.synchronize()
    want = [host(x).copy() for x in s.results()]
    free, made = t.cuda.mem_get_info()[0], t.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        s.run()
    t.cuda.synchronize()
    log(f"raw calls {dtype}: {free} bytes free before, {t.cuda.mem_get_info()[0]} after")
    assert t.cuda.mem_get_info()[0] == free
    assert t.cuda.memory_stats()["allocation.all.allocated"] == made
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        s.run()
    for k in range(3):
        for x in s.results():
            x.fill_(3)
        g.replay()
        t.cuda.synchronize()
        for i, (x, w) in enumerate(zip(s.results(), want)):
            assert_bits_equal(host(x), w, f"result {i} of replay {k}")
        s.run()
