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
        return 4


def test_norm_and_workspace_on_the_gradients_gpu():
    ql._norm_out(On(1), On(1), 1)
    for norm, ws in ((On(0), On(0)), (On(0), On(1)), (On(1), On(0))):
        with pytest.raises(ValueError):
            ql._norm_out(norm, ws, 1)
    with pytest.raises(TypeError):
        ql._norm_out(On(1, torch.float64), On(1), 1)
    with pytest.raises(ValueError):
        ql._norm_out(On(1, n=2), On(1), 1)
