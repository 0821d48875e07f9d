"""Host tests of the binding's checks (no GPU): which device a call runs on and
which buffers it refuses, with stand-ins for tensors on several GPUs."""
import contextlib

import pytest

ql = pytest.importorskip("quantized_linear_layer_amd")
torch = pytest.importorskip("torch")


class On:
    """A tensor's surface, on a GPU by number."""

    def __init__(self, device, dtype=torch.float32, n=1):
        self.number, self.dtype, self.n = device, dtype, n
        self.device = f"cuda:{device}"
        self.is_cuda = True

    def get_device(self):
        return self.number

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True


def test_norm_and_workspace_on_the_gradients_gpu():
    ql._norm_out(On(1), On(1), 1)
    for norm, ws in ((On(0), On(0)), (On(0), On(1)), (On(1), On(0))):
        with pytest.raises(ValueError):
            ql._norm_out(norm, ws, 1)
    with pytest.raises(TypeError):
        ql._norm_out(On(1, torch.float64), On(1), 1)
    with pytest.raises(ValueError):
        ql._norm_out(On(1, n=2), On(1), 1)


class Library:
    """Notes the calls of the C entries, and on which GPU they were made."""

    def __init__(self):
        self.calls, self.gpus, self.current = [], [], 0

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            self.gpus.append(self.current)
            return 0
        return call

    @contextlib.contextmanager
    def device(self, number):
        before, self.current = self.current, number
        yield
        self.current = before


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(ql, "lib", lambda: lib)
    monkeypatch.setattr(ql, "_queue", lambda stream, device: 0)
    monkeypatch.setattr(ql, "_current", lambda: lib.current)
    monkeypatch.setattr(torch.cuda, "device", lib.device)
    return lib


def test_packed_weight_buffers_are_large_enough(library, monkeypatch):
    """E = 3 matrices of 130 x 5: two steps of 64 bytes of codes and 4 scales a column."""
    monkeypatch.setattr(ql, "_gpu", lambda *tensors: 0)
    W = torch.zeros((3, 130, 5))
    codes, scales = 3 * 5 * 2 * 64, 3 * 5 * 2 * 4

    def buffers(c, s):
        return torch.zeros(c, dtype=torch.uint8), torch.zeros(s, dtype=torch.uint8)

    for c, s in ((codes - 1, scales), (codes, scales - 1), (0, scales), (codes, 0)):
        with pytest.raises(ValueError):
            ql.fp4lin_experts_quantize_weight_mx(W, *buffers(c, s))
    with pytest.raises(ValueError):
        ql.fp4lin_experts_quantize_weight_mx(W, torch.zeros(2 * codes, dtype=torch.uint8)[::2], buffers(0, scales)[1])
    assert library.calls == []
    ql.fp4lin_experts_quantize_weight_mx(W, *buffers(codes, scales))
    ql.fp4lin_experts_quantize_weight_mx(W, *buffers(codes + 64, scales + 64))
    assert library.calls == ["fp4lin_experts_quantize_weight_mx"] * 2


@pytest.mark.parametrize("gpu", [0, 1])
def test_raw_calls_run_on_the_tensors_gpu(library, monkeypatch, gpu):
    """With GPU 0 current: the null stream of a GPU is the current one's."""
    monkeypatch.setattr(ql, "_gpu", lambda *tensors: gpu)
    monkeypatch.setattr(ql, "_grads", lambda tensors, out: (None, 1, 4, gpu))
    A, dY, W = torch.zeros((4, 8)), torch.zeros((4, 6)), torch.zeros((2, 8, 6))
    re, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    Wq, Ws = torch.zeros((2, 6, 64), dtype=torch.uint8), torch.zeros((1, 2, 6, 4), dtype=torch.uint8)
    target, f, H = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros((8, 6))
    norm = torch.zeros(())
    ql.fp4lin_experts_quantize_weight_mx(W, Wq, Ws)
    ql.fp4lin_experts_forward_mx(A, W, re, dY, ws)
    ql.fp4lin_experts_apply_mx(A, Wq, Ws, re, dY, ws)
    ql.fp4lin_experts_dgrad_mx(dY, W, re, A, ws)
    ql.fp4lin_experts_wgrad_mx(A, dY, re, W, ws)
    ql.fp4lin_head_loss(A, H, target, f, f, ws)
    ql.fp4lin_head_loss_backward(A, H, target, f, f, A, H, ws)
    ql.fp4lin_grad_norm([A], norm, ws)
    ql.fp4lin_clip_grads([A], 1.0, norm, ws)
    assert len(library.calls) == 9 and library.gpus == [gpu] * 9 and library.current == 0
