"""An execute on a device that is not current is refused before any pointer reaches the
library, which launches on the current device: the kernel would run there, on another
device's memory and in no order with that device's work. CPU only: the current device's
index is patched and operands are stood in for."""
import pytest
import torch

from gemm_epilogues_epilog_amd import mx


@pytest.fixture
def current(monkeypatch):
    """Sets the index of the current device, and fails on any use of the library."""
    def used(*a, **k):
        raise AssertionError("the library was reached")
    monkeypatch.setattr(mx, "load", used)
    def to(index):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: index, raising=False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: index)
    return to


def operand(rows, k, fmt, device):
    q = mx.MXTensor.__new__(mx.MXTensor)
    q.rows, q.k, q.format, q.experts, q.device = rows, k, fmt, None, torch.device(device)
    q.code_ptr = q.scale_ptr = 1 << 20
    return q


def test_microscaled_product(current):
    for plan_on, now in ((1, 0), (0, 1)):
        mm = mx.MXMatmul(64, 96, "mxfp8", "NONE", "bf16")
        mm.handle, mm.device = 1 << 20, torch.device("cuda", plan_on)   # as plan() leaves it
        X, W = operand(4, 96, "mxfp8", mm.device), operand(64, 96, "mxfp4", mm.device)
        out = operand(4, 64, "mxfp8", mm.device)
        current(now)
        with pytest.raises(ValueError, match="current device"):
            mm.execute(X, W)
        m8 = mx.MXMatmul(64, 96, "mxfp8", "NONE", "mxfp8")
        m8.handle, m8.device = 1 << 20, mm.device
        with pytest.raises(ValueError, match="current device"):
            m8.execute(X, W, out=out)
        mm.handle = m8.handle = None
