"""GPU tests that the raw calls of the experts' routing, the embedding and the distillation
allocate nothing and can be captured, and that calls on two streams keep to themselves:
a graph of all of them, replayed with eager work between, gives the eager results bit
for bit, and so do two streams that run them at once, each on buffers of its own."""
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

    def __init__(self, ql, dtype, T, k, E, H=136, V=1000, list_k=70, seed=0):
        import torch as t
        self.ql = ql
        g = t.Generator(device="cuda").manual_seed(seed + T)

        def randn(*shape, dtype=dtype):
            return t.randn(shape, generator=g, device="cuda").to(dtype)

        def ints(low, high, *shape):
            return t.randint(low, high, shape, generator=g, device="cuda", dtype=t.int32)

        def empty(*shape, dtype=t.float32):
            return t.full(shape, 3, device="cuda", dtype=dtype)

        def ws(n):
            assert n > 0
            return t.empty(n, device="cuda", dtype=t.uint8)

        self.X, self.expert = randn(T, H), ints(-1, E + 1, T, k)
        self.Xs, self.row_end, self.slot_row = empty(T * k, H, dtype=dtype), empty(E, dtype=t.int32), \
            empty(T, k, dtype=t.int32)
        self.weight, self.out, self.outb = randn(T, k, dtype=t.float32), empty(T, H), empty(T, H, dtype=dtype)
        self.dY, self.dw = empty(T * k, H, dtype=t.bfloat16), empty(T, k)
        self.table, self.token = randn(V, H), ints(-1, V // 3, T)
        self.token[: T // 2] = 5  # a long list
        self.rows, self.dE, self.sum = empty(T, H, dtype=dtype), empty(V, H), empty(V, H, dtype=dtype)
        self.ws = ws(ql.embed_backward_workspace_bytes(T, V, H))
        self.W, self.index = randn(H, V), ints(-1, V, T, list_k)
        self.teacher, self.dloss = randn(T, list_k, dtype=t.float32), randn(T, dtype=t.float32)
        self.loss, self.lse = empty(T), empty(T)
        self.dX, self.dW = empty(T, H, dtype=dtype), empty(H, V, dtype=dtype)
        code = ql.BF16 if dtype == t.bfloat16 else ql.F32
        self.head_ws = [ws(ql.head_distill_workspace_bytes(code, False, T, H, V, list_k, H, V, b)) for b in (False, True)]

    def run(self, stream=None):
        q, s = self.ql, dict(stream=stream)
        q.fp4lin_experts_dispatch(self.X, self.expert, self.Xs, self.row_end, self.slot_row, **s)
        q.fp4lin_experts_combine(self.Xs, self.slot_row, self.row_end, self.out, self.weight, **s)
        q.fp4lin_experts_combine(self.Xs, self.slot_row, self.row_end, self.outb, None, self.X, **s)
        q.fp4lin_experts_combine_backward(self.out, self.Xs, self.slot_row, self.row_end, self.dY, self.weight,
                                          self.dw, **s)
        q.fp4lin_embed(self.table, self.token, self.rows, 2.5, **s)
        q.fp4lin_embed_backward(self.rows, self.token, self.dE, self.ws, 1.5, **s)
        q.fp4lin_embed_backward(self.rows, self.token, self.sum, self.ws, **s)
        q.fp4lin_embed_backward(self.X, self.token, self.sum, self.ws, add=True, **s)
        q.fp4lin_head_distill(self.X, self.W, self.index, self.teacher, self.loss, self.lse, self.head_ws[0], 2.0, **s)
        q.fp4lin_head_distill_backward(self.X, self.W, self.index, self.teacher, self.lse, self.dloss, self.dX, self.dW,
                                       self.head_ws[1], 2.0, **s)

    def results(self):
        return [self.Xs, self.row_end, self.slot_row, self.out, self.outb, self.dY, self.dw, self.rows, self.dE, self.sum,
                self.loss, self.lse, self.dX, self.dW]


# the sort and the move in one launch and in two, with one key a workgroup and with more
SIZES = [(90, 2, 5), (700, 3, 5), (700, 3, 600)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_raw_calls_allocate_nothing(ql, T, k, E, dtype):
    import torch as t
    s = Step(ql, t.bfloat16 if dtype == "bf16" else t.float32, T, k, E)
    s.run()  # loads the kernels
    t.cuda.synchronize()
    want = [host(x).copy() for x in s.results()]
    free, made = t.cuda.mem_get_info()[0], t.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        s.run()
    t.cuda.synchronize()
    log(f"raw calls {T} {k} {E} {dtype}: {free} bytes free before, {t.cuda.mem_get_info()[0]} after")
    assert t.cuda.mem_get_info()[0] == free
    assert t.cuda.memory_stats()["allocation.all.allocated"] == made
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        s.run()
    for n in range(3):
        for x in s.results():
            x.fill_(3)
        g.replay()
        t.cuda.synchronize()
        for i, (x, w) in enumerate(zip(s.results(), want)):
            assert_bits_equal(host(x), w, f"result {i} of replay {n}")
        s.run()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(ql, dtype):
    """Also the helpers, given a stream: what they allocate belongs to it."""
    import torch as t
    kind = t.bfloat16 if dtype == "bf16" else t.float32
    steps = [Step(ql, kind, 700, 3, 5, seed=i) for i in range(2)]
    for s in steps:
        s.run()
    t.cuda.synchronize()
    want = [[host(x).copy() for x in s.results()] for s in steps]
    streams = [t.cuda.Stream() for _ in range(2)]
    for n in range(3):
        for s in steps:
            for x in s.results():
                x.fill_(3)
        t.cuda.synchronize()
        for s, q in zip(steps, streams):
            s.run(q)
        t.cuda.synchronize()
        for s, w in zip(steps, want):
            for i, (x, y) in enumerate(zip(s.results(), w)):
                assert_bits_equal(host(x), y, f"result {i}, turn {n}")
    got = []
    for s, q in zip(steps, streams):
        Xs, row_end, slot_row = ql.experts_dispatch(s.X, s.expert, 5, stream=q)
        out = ql.experts_combine(Xs, slot_row, row_end, s.weight, out_dtype=t.float32, stream=q)
        dY, dw = ql.experts_combine_backward(out, Xs, slot_row, row_end, s.weight, out_dtype=t.bfloat16, stream=q)
        rows = ql.embed(s.table, s.token, 2.5, stream=q)
        dE = ql.embed_backward(rows, s.token, 1000, 1.5, out_dtype=t.float32, stream=q)
        loss, lse = ql.head_distill(s.X, s.W, s.index, s.teacher, 2.0, stream=q)
        dX, dW = ql.head_distill_backward(s.X, s.W, s.index, s.teacher, lse, s.dloss, 2.0, stream=q)
        got.append([Xs, row_end, slot_row, out, None, dY, dw, rows, dE, None, loss, lse, dX, dW])
    t.cuda.synchronize()
    for g, w in zip(got, want):
        for i, (x, y) in enumerate(zip(g, w)):
            if x is not None:
                assert_bits_equal(host(x), y, f"helper's result {i}")


def test_graphs_that_share_a_workspace(ql):
    """Two captured gradients on one workspace, replayed one after the other: each call
    writes what it reads of it."""
    import torch as t
    a, b = Step(ql, t.float32, 700, 1, 5, seed=1), Step(ql, t.float32, 700, 1, 5, seed=2)
    b.ws, b.head_ws = a.ws, a.head_ws
    want = []
    for s in (a, b):
        s.run()
        t.cuda.synchronize()
        want.append([host(x).copy() for x in s.results()])
    graphs = []
    for s in (a, b):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            s.run()
        graphs.append(g)
    for n in range(3):
        for g in graphs:
            g.replay()
        t.cuda.synchronize()
        for s, w in zip((a, b), want):
            for i, (x, y) in enumerate(zip(s.results(), w)):
                assert_bits_equal(host(x), y, f"result {i} of replay {n}")
        a.X.mul_(1.0)
