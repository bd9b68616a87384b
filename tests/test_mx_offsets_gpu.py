"""Experts' offsets that do not ascend: each range is held to the rows, and to those past the
furthest end of the ranges before it, so that every row has one expert at most. Whole numbers, so
every product is exact and says which expert a row had."""
import numpy as np
import pytest
import torch

from gemm_epilogues_epilog_amd import mx

pytestmark = pytest.mark.gpu


def owners(offsets, m):
    """The expert of each row, -1 for none."""
    own, end = np.full(m, -1), 0
    hold = [min(max(o, 0), m) for o in offsets]
    for e in range(len(offsets) - 1):
        lo, hi = hold[e], hold[e + 1]
        if hi > lo:
            own[max(lo, end):max(hi, end)] = e
            end = max(end, hi)
    return own


def test_owners():
    assert owners([0, 2, 2, 5], 6).tolist() == [0, 0, 2, 2, 2, -1]
    assert owners([0, 4, 0, 4], 4).tolist() == [0, 0, 0, 0]
    assert owners([3, 1, 2, 9], 5).tolist() == [-1, 1, 2, 2, 2]
    assert owners([4, 6, 1, 7], 8).tolist() == [-1, -1, -1, -1, 0, 0, 2, -1]


def lists(m, seed):
    r = np.random.default_rng(seed)
    yield [0, m] * 6
    yield [0, m // 2, 0, m, 0, m, 0, m]
    yield [0, m, m // 3, m, m // 3]
    yield r.integers(-5, m + 6, 9).tolist()
    yield [0, m] * 65 + [3]                                    # 130 experts, two loads of a wave and more
    yield [m // 2] * 64 + [m // 4, m // 2 + 3, 0, m, m]        # nothing in the first 64
    yield sorted(r.integers(0, m // 2, 70).tolist()) + r.integers(0, m + 1, 31).tolist()


@pytest.mark.parametrize("which", range(7))
@pytest.mark.parametrize("m,n", [(40, 96), (300, 1100), (700, 96), (1012, 16400)])
def test_rows_have_one_expert(gpu, m, n, which):
    offsets = list(lists(m, m))[which]
    E, k = len(offsets) - 1, 64
    w = torch.zeros(E, n, k, device="cuda")
    e = torch.arange(E, device="cuda")   # three digits of e, as values that MXFP4 holds beside 6
    for j in range(3):
        w[:, :, j] = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0], device="cuda")[e // 6 ** j % 6].view(E, 1)
    w[:, :, 3] = 6.0
    W = mx.mx_quantize(w, "mxfp4")
    assert torch.equal(mx.mx_dequantize(W, "f32"), w)
    own = owners(offsets, m)
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    with mx.MXMatmul(n, k, "mxfp8", "NONE", "f32", experts=E) as mm:
        for j in range(3):
            xj = torch.zeros(m, k, device="cuda")
            xj[:, j] = 1.0
            D = torch.full((m, n), 9.0, device="cuda")
            mm.execute(mx.mx_quantize(xj, "mxfp8"), W, offsets=o, out=D)
            at = torch.tensor(own, device="cuda")
            want = torch.where(at >= 0, w[:, 0, j][at.clamp(min=0)], 9.0)
            assert torch.equal(D, want.view(m, 1).expand(m, n))
