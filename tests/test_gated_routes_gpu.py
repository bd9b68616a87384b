"""The kernels of the gated block and of 4-bit weights that only larger shapes reach (gated_shapes.py),
against the formulas in 64 bits, by the bounds of test_gated_gpu.py and test_w4_gpu.py."""
import pytest
import torch

from gemm_epilogues_epilog_amd import gated
from tests import gated_shapes as S
from tests import test_gated_gpu as G
from tests import test_w4_gpu as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,t", S.FORWARD)
def test_forward(gpu, m, n, k, t):
    dtype = S.NAMES[t]
    for act, bias in (("SILU", True), ("GELU", False), ("RELU", True)):
        x, w, b = G.make(m, n, k, dtype, m + n + k, bias=bias)
        h, z = gated.gated_forward(x, w, b, act=act, save=True)
        G.check_forward(x, w, b, act, dtype, h, z, act)
        assert torch.equal(gated.gated_forward(x, w, b, act=act)[0], h)


@pytest.mark.parametrize("m,d,n,t", S.DOWN)
def test_down(gpu, m, d, n, t):
    dtype = S.NAMES[t]
    g = torch.Generator().manual_seed(m + d)
    h = torch.randn(m, n, generator=g).to(G.T[dtype]).cuda()
    w = (torch.randn(d, n, generator=g) * n ** -0.5).to(G.T[dtype]).cuda()
    y = gated.gated_down(h, w)
    G.close(y, h.double() @ w.double().t(), G.sum_error(h.double(), w.double().t()), dtype)
    assert torch.equal(gated.gated_down(h, w), y)


@pytest.mark.parametrize("m,n,k,d,t", S.BACKWARD)
def test_backward(gpu, m, n, k, d, t):
    dtype = S.NAMES[t]
    for act in G.ACTS:
        x, w, b = G.make(m, n, k, dtype, m + n + k)
        g = torch.Generator().manual_seed(d)
        h, z = gated.gated_forward(x, w, b, act=act, save=True)
        wd = (torch.randn(d, n, generator=g) * n ** -0.5).to(G.T[dtype]).cuda()
        dy = (torch.randn(m, d, generator=g) * 0.3).to(G.T[dtype]).cuda()
        out = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, act=act, bias_grad="f32")
        G.check_backward(dy, x, w, z, wd, h, act, dtype, out, act)
        again = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, act=act, bias_grad="f32")
        assert all(torch.equal(p, q) for p, q in zip(out, again))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,group,halves", S.W4)
def test_w4(gpu, m, n, k, group, halves, dtype):
    a = Q.make(m, n, k, group, dtype, m + n + k, gated=halves)
    if halves:
        Q.check_gated(*a, dtype, [("SILU", True), ("RELU", False)])
    else:
        Q.check(*a, dtype, [("GELU_BIAS", None), ("NONE", "f32")])
