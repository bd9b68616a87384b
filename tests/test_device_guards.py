"""An execute on a device that is not current is refused before any pointer reaches the
library, which launches on the current device: the kernel would run there, on another
device's memory and in no order with that device's work. CPU only: the current device's
index is patched and operands are stood in for."""
import pytest
import torch

import gemm_epilogues_epilog_amd as ge
from gemm_epilogues_epilog_amd import mx
from tests.test_binding_checks import FakeDev


@pytest.fixture
def current(monkeypatch):
    """Sets the index of the current device, and fails on any use of the library."""
    def used(*a, **k):
        raise AssertionError("the library was reached")
    monkeypatch.setattr(mx, "load", used)
    monkeypatch.setattr(ge, "load", used)
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


def test_fused_product(current):
    def operands(index):
        return [FakeDev(s, torch.float16, device=f"cuda:{index}") for s in ((64, 32), (32, 48), (64,), (64, 48))]
    for plan_on, now in ((1, 0), (0, 1)):
        A, B, bias, out = operands(plan_on)
        current(now)
        for planned in (True, False):   # planning also goes to the current device
            m = ge.Matmul(64, 48, 32, "f16", "BIAS")
            if planned:
                m.handle, m.device_index = 1 << 20, plan_on   # as plan() leaves it
            for call in (m.execute, m.autotune):
                with pytest.raises(ValueError, match="current device"):
                    call(A, B, bias, out=out)
            assert planned or m.handle is None
            m.handle = None
    # a plan of another device than the operands'
    A, B, bias, out = operands(0)
    current(0)
    m = ge.Matmul(64, 48, 32, "f16", "BIAS")
    m.handle, m.device_index = 1 << 20, 1
    with pytest.raises(ValueError, match="planned on"):
        m.execute(A, B, bias, out=out)
    m.handle = None
