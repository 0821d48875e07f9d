"""Host tests of the binding's checks (no GPU): which device a call runs on and
which buffers it refuses, with stand-ins for tensors on several GPUs."""
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
    """Notes the calls of the C entries."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(ql, "lib", lambda: lib)
    monkeypatch.setattr(ql, "_queue", lambda stream, device: 0)
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
