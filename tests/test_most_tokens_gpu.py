"""As many tokens as the header allows, 2^31 - 1, more than one launch has lanes for: rows from the first
launch, from around its end and from the last one. Whole numbers, so results are exact."""
import pytest
import torch

from gemm_epilogues_epilog_amd import gated, w4

pytestmark = pytest.mark.gpu

M = (1 << 31) - 1
# around the ends of launches of every kernel here (2^30, 3 2^29 rows and what is left), and the ends
ROWS = [0, 1, 12345, (1 << 30) - 513, (1 << 30) - 257, (1 << 30) - 256, (1 << 30) - 1, 1 << 30, (1 << 30) + 300, 3 * (1 << 29) - 193,
        3 * (1 << 29) - 1, 3 * (1 << 29), M - 600, M - 257, M - 256, M - 129, M - 2, M - 1]


def tokens(k):
    """(M, k) of f16 zeros but for ROWS: whole numbers there."""
    x = torch.zeros(M, k, dtype=torch.float16, device="cuda")
    v = torch.randint(-3, 4, (len(ROWS), k), generator=torch.Generator().manual_seed(k)).to(torch.float16).cuda()
    x[ROWS] = v
    return x, v


def check(d, want):
    assert torch.equal(d[ROWS].double(), want)
    # the other rows hold zeros
    total = sum(int((part != 0).any(1).sum()) for part in d.split(1 << 28))
    assert total == int((want != 0).any(1).sum())


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,k", [(1, 1), (8, 8)])
def test_gated(gpu, n, k):
    x, v = tokens(k)
    w = torch.randint(-2, 3, (2 * n, k), generator=torch.Generator().manual_seed(n)).to(torch.float16).cuda()
    w[:, 0] = 1
    h, _ = gated.gated_forward(x, w, act="RELU")
    z = v.double() @ w.double().t()
    check(h, z[:, :n].clamp(min=0) * z[:, n:])


@pytest.mark.parametrize("d,n", [(1, 1), (8, 8)])
def test_down(gpu, d, n):
    h, v = tokens(n)
    w = torch.randint(-2, 3, (d, n), generator=torch.Generator().manual_seed(n)).to(torch.float16).cuda()
    w[:, 0] = 1
    check(gated.gated_down(h, w), v.double() @ w.double().t())


@pytest.mark.parametrize("group", [32, 64])
def test_w4(gpu, group):
    x, v = tokens(8)
    q = torch.randint(0, 16, (1, 4), generator=torch.Generator().manual_seed(1)).to(torch.uint8)
    W = w4.w4_pack(q.cuda(), torch.ones(1, 1, dtype=torch.float16, device="cuda"), None, group)
    check(w4.w4_matmul(x, W), v.double() @ w4.w4_dequantize(W, "f32").double().t())
