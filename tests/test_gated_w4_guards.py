"""Calls of the gated block and of 4-bit weights with operands on a device that is not current are
refused before any pointer reaches the library, which launches on the current device. CPU only: the
current device's index is patched and operands are stood in for."""
import pytest
import torch

from gemm_epilogues_epilog_amd import gated, mx, w4


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a device."""
    @staticmethod
    def make(shape, dtype, device):
        t = torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)
        t.place = torch.device(device)
        return t

    is_cuda = property(lambda self: True)
    device = property(lambda self: self.place)

    def get_device(self):
        return self.place.index


@pytest.fixture
def current(monkeypatch):
    """Sets the index of the current device, and fails on any use of the library."""
    def used(*a, **k):
        raise AssertionError("the library was reached")
    for module in (mx, gated, w4):
        monkeypatch.setattr(module, "load", used)

    def to(index):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: index, raising=False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: index)
    return to


def weight(rows, k, gated_, device):
    q = w4.W4Tensor.__new__(w4.W4Tensor)
    q.rows, q.k, q.group, q.gated, q.dtype, q.device = rows, k, 32, gated_, torch.float16, torch.device(device)
    q._buf, q._parts, q.ptrs = OnDevice.make((1024,), torch.uint8, device), None, (1 << 20,) * 3
    return q


@pytest.mark.parametrize("on,now", [(1, 0), (0, 1)])
def test_operands_of_another_device(current, on, now):
    def f(*shape, dtype=torch.float16, device=on):
        return OnDevice.make(shape, dtype, f"cuda:{device}")
    current(now)
    x, W, G = f(4, 64), weight(8, 64, False, f"cuda:{on}"), weight(8, 64, True, f"cuda:{on}")
    for call in (lambda: gated.gated_forward(x, f(16, 64)), lambda: gated.gated_down(x, f(8, 64)),
                 lambda: gated.gated_backward(f(4, 8), x, f(16, 64), f(4, 16)),
                 lambda: w4.w4_quantize(x, 32), lambda: w4.w4_pack(f(8, 32, dtype=torch.uint8), f(8, 2)),
                 lambda: w4.w4_dequantize(W), lambda: w4.w4_matmul(x, W), lambda: w4.w4_gated(x, G)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_weights_of_another_device(current):
    current(0)
    x = OnDevice.make((4, 64), torch.float16, "cuda:0")
    for call in (lambda: w4.w4_matmul(x, weight(8, 64, False, "cuda:1")), lambda: w4.w4_gated(x, weight(8, 64, True, "cuda:1")),
                 lambda: gated.gated_down(x, OnDevice.make((8, 64), torch.float16, "cuda:1")),
                 lambda: gated.gated_forward(x, OnDevice.make((16, 64), torch.float16, "cuda:1"))):
        with pytest.raises(ValueError):
            call()
