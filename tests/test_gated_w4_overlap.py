"""Results that the caller gives and that lie over an operand are refused before the library is reached:
workgroups would read what others have written. CPU only, with operands stood in for as in
test_gated_w4_guards.py."""
import pytest
import torch

from gemm_epilogues_epilog_amd import gated, w4
from tests.test_gated_w4_guards import OnDevice, current, weight   # noqa: F401


class View(OnDevice):
    """Elements `at` onwards of a buffer, in a shape."""
    @staticmethod
    def of(buf, at, *shape):
        n = 1
        for s in shape:
            n *= s
        t = buf.as_subclass(torch.Tensor)[at:at + n].view(*shape).as_subclass(View)
        t.place = buf.place
        return t


def test_overlapping_results(current):   # noqa: F811
    current(0)
    buf = OnDevice.make((4096,), torch.float16, "cuda:0")
    x, w = View.of(buf, 0, 4, 16), View.of(buf, 256, 32, 16)
    h, wd = View.of(buf, 1024, 4, 16), View.of(buf, 2048, 16, 16)
    z, apart = View.of(buf, 3200, 4, 32), View.of(buf, 3600, 4, 16)
    W, G = weight(16, 16, False, "cuda:0"), weight(32, 16, True, "cuda:0")
    W._buf = View.of(buf, 1536, 256)
    G._buf = View.of(buf, 1536, 256)
    for call in (lambda: gated.gated_forward(x, w, out=x), lambda: gated.gated_forward(x, w, out=View.of(buf, 63, 4, 16)),
                 lambda: gated.gated_forward(x, w, out=View.of(buf, 300, 4, 16)),
                 lambda: gated.gated_forward(x, w, out=h, z_out=View.of(buf, 1080, 4, 32)),
                 lambda: gated.gated_forward(x, w, out=h, z_out=View.of(buf, 700, 4, 32)),
                 lambda: gated.gated_forward(x, w, View.of(buf, 1030, 32), out=h),
                 lambda: gated.gated_down(h, wd, out=h), lambda: gated.gated_down(h, wd, out=View.of(buf, 2200, 4, 16)),
                 lambda: w4.w4_matmul(x, W, out=x), lambda: w4.w4_gated(x, G, out=x),
                 lambda: w4.w4_matmul(x, W, out=View.of(buf, 1540, 4, 16)), lambda: w4.w4_dequantize(W, out=View.of(buf, 1700, 16, 16))):
        with pytest.raises(ValueError, match="overlap"):
            call()
    # beside them: as far as the library
    for call in (lambda: gated.gated_forward(x, w, out=View.of(buf, 64, 4, 16), z_out=z), lambda: gated.gated_down(h, wd, out=apart),
                 lambda: w4.w4_matmul(x, W, out=apart)):
        with pytest.raises(AssertionError, match="reached"):
            call()
