"""The bias's gradient sums dZ before its rounding to 16 bits: against the formula in 64 bits, by the
errors of fp32 alone (bounds as in test_gated_gpu.py without the half steps of dZ), in every kernel that
computes dZ."""
import math

import pytest
import torch

from gemm_epilogues_epilog_amd import gated
from tests import test_gated_gpu as G

pytestmark = pytest.mark.gpu


def expect(dy, z, wd, act):
    """Column sums of dZ and their bound."""
    n = z.shape[1] // 2
    D = dy.double()
    dh, eh = D, torch.zeros(1, dtype=torch.float64, device="cuda")
    if wd is not None:
        dh, eh = D @ wd.double(), G.sum_error(D, wd.double())
    g, u = z.double()[:, :n], z.double()[:, n:]
    a, da = G.act64(g, act)
    dz = torch.cat((dh * u * da, dh * a), 1)
    slack, lead = (16 + 4 * g.abs()) * G.U, 1 + g.abs() * 1.2
    ez = torch.cat(((eh * da.abs() + slack * dh.abs() * lead) * u.abs(), eh * a.abs() + slack * (dh * a).abs()), 1)
    return dz.sum(0), 8 * torch.sqrt((ez * ez).sum(0)) + (8 * math.sqrt(dz.shape[0]) + 4) * G.U * dz.abs().sum(0)


# tiles of 128 x 128 (two and three stages), 128, 192 and 256 x 256, one round of them and several, and
# ragged ones; more rows of sums than one kernel adds up; the general kernels; a few rows; d small, so that
# the errors of dH do not hide those of the sums
SHAPES = [(77, 1000, 40), (1, 64, 16), (130, 264, 1600), (1999, 4344, 64), (2048, 8192, 128), (2048, 4352, 128), (1801, 4400, 72),
          (1152, 4096, 256), (20011, 136, 24), (300, 251, 24), (2048, 2050, 33), (40, 33, 7), (3, 5, 2), (9000, 24, 11)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,d", SHAPES)
def test_sums_before_rounding(gpu, m, n, d, dtype):
    for act in G.ACTS:
        x, w, _ = G.make(m, n, 8, dtype, m + n + d, bias=False)
        g = torch.Generator().manual_seed(d)
        h, z = gated.gated_forward(x, w, act=act, save=True)
        wd = (torch.randn(d, n, generator=g) * d ** -0.5).to(G.T[dtype]).cuda()
        dy = (torch.randn(m, d, generator=g) * 0.3).to(G.T[dtype]).cuda()
        dh = (torch.randn(m, n, generator=g) * 0.3).to(G.T[dtype]).cuda()
        for grad, down in ((dy, wd), (dh, None)):
            want, err = expect(grad, z, down, act)
            for t in {"f32", dtype}:
                out = gated.gated_backward(grad, x, w, z, w_down=down, act=act, bias_grad=t)
                G.close(out.dbias, want, err, t, (act, t, down is None))
                alone = gated.gated_backward(grad, x, w, z, w_down=down, act=act, bias_grad=t, need_dx=False, need_dw=False)
                assert torch.equal(out.dbias, alone.dbias)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_unaligned(gpu, dtype):
    """Whole 16-byte rows behind pointers that are not on 16 bytes."""
    m, n, d = 150, 264, 24
    x, w, _ = G.make(m, n, 8, dtype, 3, bias=False)
    _, z = gated.gated_forward(x, w, save=True)
    wd = (torch.randn(d, n, device="cuda") * d ** -0.5).to(G.T[dtype])
    buf = torch.randn(m * d + 1, device="cuda").to(G.T[dtype])
    dy = buf[1:].view(m, d)
    want, err = expect(dy, z, wd, "SILU")
    G.close(gated.gated_backward(dy, x, w, z, w_down=wd, bias_grad="f32").dbias, want, err, "f32")


@pytest.mark.parametrize("m", [77, 2000])
def test_infinite_weights_and_the_tiles_last_rows(gpu, m):
    """An infinity in Wd: infinite sums of its column, no NaN from a tile's rows past the last token."""
    n, d = 2056, 72
    z = torch.ones(m, 2 * n, device="cuda").bfloat16()
    wd = torch.ones(d, n, device="cuda").bfloat16()
    wd[3, 5] = float("inf")
    dy = torch.ones(m, d, device="cuda").bfloat16()
    x, w = torch.ones(m, 8, device="cuda").bfloat16(), torch.ones(2 * n, 8, device="cuda").bfloat16()
    db = gated.gated_backward(dy, x, w, z, w_down=wd, act="SILU", bias_grad="f32").dbias
    bad = torch.zeros(2 * n, dtype=torch.bool, device="cuda")
    bad[5] = bad[n + 5] = True
    assert (db[bad] == float("inf")).all() and torch.isfinite(db[~bad]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_down_gradient_alone(gpu, dtype):
    """Through the C interface, where the others' operands may be left out: the same gradient, with Z and
    the rest of the operands missing and the part of the workspace that holds dZ untouched."""
    m, n, k, d = 100, 264, 40, 72
    x, w, _ = G.make(m, n, k, dtype, 1, bias=False)
    h, z = gated.gated_forward(x, w, save=True)
    wd, dy = torch.randn(d, n, device="cuda").to(G.T[dtype]), torch.randn(m, d, device="cuda").to(G.T[dtype])
    want = gated.gated_backward(dy, x, w, z, w_down=wd, h=h)
    L, t = gpu.load(), gpu.DTYPES[dtype]
    size = L.gemm_epilog_gated_workspace_bytes(m, n, k, d, t)
    ws, out = torch.full((size,), 7, dtype=torch.uint8, device="cuda"), torch.empty_like(want.dw_down)
    assert L.gemm_epilog_gated_backward(m, n, k, d, t, 0, dy.data_ptr(), None, None, None, h.data_ptr(), wd.data_ptr(), None, None,
                                        out.data_ptr(), None, 0, ws.data_ptr(), size,
                                        torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want.dw_down)
    assert (ws[:m * 2 * n * (4 if dtype == "f32" else 2)] == 7).all()
    # without Z the others are refused
    assert L.gemm_epilog_gated_backward(m, n, k, d, t, 0, dy.data_ptr(), x.data_ptr(), w.data_ptr(), None, h.data_ptr(), wd.data_ptr(),
                                        want.dx.data_ptr(), None, None, None, 0, ws.data_ptr(), size, None) == 3
