"""4-bit weights at the ends of the types' range, on the GPU.

Codes of fp32 weights are the exact quotient's: a border h + 1/2 of a 16-bit scale s, h below 16, is the
product of 5 and 11 bits, an fp32 number itself; any other fp32 value lies a step of 2^-23 or 2^-24 of
itself away (below a power of two), and its quotient as far from the border in proportion, more than
the half step, below 2^-24 of the border (which is no power of two), that a rounded quotient may be off.

Products: scales outside of [2^-14, 2^11] (fp16), and bf16's from its smallest subnormal numbers to 2^126,
beside each other in a row. Bounds as in test_w4_gpu.py; where terms are subnormal, each of the k
products and k additions is off by at most 2^-150 as well."""
import math

import pytest
import torch

from gemm_epilogues_epilog_amd import w4
from tests import test_w4_gpu as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_f32_codes_at_borders(gpu, dtype, symmetric):
    g = torch.Generator().manual_seed(5)
    rows, group = 3000, 64
    s = (torch.exp2(torch.randint(-9, 3, (rows, 1), generator=g).float()) * (1 + torch.rand(rows, 1, generator=g))).to(Q.T[dtype]).float()
    z = torch.full((rows, 1), 7.0) if symmetric else torch.randint(0, 16, (rows, 1), generator=g).float()
    h = torch.randint(-7, 7, (rows, group), generator=g) + 0.5
    h = torch.minimum(torch.maximum(h, 0.5 - z), (14.5 - z).clamp(min=0.5) if not symmetric else torch.tensor(6.5))
    x = h * s                                                        # on the borders, exactly
    kind = torch.randint(0, 3, x.shape, generator=g)
    x = torch.where(kind == 0, torch.nextafter(x, torch.full_like(x, -9e9)), torch.where(kind == 1, torch.nextafter(x, torch.full_like(x, 9e9)), x))
    if symmetric:
        x[:, 0] = 7 * s[:, 0]
    else:
        x[:, 0], x[:, 1] = (15 - z[:, 0]) * s[:, 0], -z[:, 0] * s[:, 0]
    inside = (x.amin(1) >= -z[:, 0] * s[:, 0]) & (x.amax(1) <= ((15 - z) if not symmetric else z)[:, 0] * s[:, 0])
    x = x[inside]
    assert x.shape[0] > 2000
    W = w4.w4_quantize(x.cuda(), group, symmetric=symmetric, dtype=dtype)
    got, want = Q.unpack(W), Q.quantize64(x.double(), group, symmetric, dtype)
    assert torch.equal(got[1].double(), want[1]) and torch.equal(got[1].float(), s[inside])
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_f32_codes(gpu, dtype):
    x = torch.randn(2000, 512, generator=torch.Generator().manual_seed(6))
    for group in (32, 128, 256):
        got, want = Q.unpack(w4.w4_quantize(x.cuda(), group, dtype=dtype)), Q.quantize64(x.double(), group, False, dtype)
        assert torch.equal(got[1].double(), want[1]) and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


# (exponents of the scales from .. to, of x): f > 1 alone; f16's whole range; bf16's largest; its smallest
# alone, with x that makes normal and subnormal products; both ends and the middle
RANGES = {"f16": [(12, 16, -6), (-24, 16, -4)],
          "bf16": [(101, 127, -20), (-133, -99, 8), (-133, -120, -4), (-133, 127, -20)]}


@pytest.mark.parametrize("dtype,i", [(d, i) for d in RANGES for i in range(len(RANGES[d]))])
@pytest.mark.parametrize("m", [1, 20, 100, 600, 2100])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_at_the_ends(gpu, m, group, dtype, i):
    lo, hi, xe = RANGES[dtype][i]
    n, k = 4200, 512
    g = torch.Generator().manual_seed(m + i)
    G = k // group
    q = torch.randint(0, 16, (n, k), generator=g).to(torch.uint8)
    z = torch.randint(0, 16, (n, G), generator=g).to(torch.uint8)
    s = torch.exp2(torch.randint(lo, hi, (n, G), generator=g).double()) * (1 + torch.randint(0, 8, (n, G), generator=g) / 8)
    s = (s * torch.where(torch.rand(n, G, generator=g) < 0.3, -1.0, 1.0)).to(Q.T[dtype])
    assert torch.isfinite(s).all()
    x = (torch.randn(m, k, generator=g) * 2.0 ** xe).to(Q.T[dtype])
    got = w4.w4_matmul(x.cuda(), w4.w4_pack(Q.nibbles(q).cuda(), s.cuda(), z.cuda(), group), out_dtype="f32")
    full = Q.values64(q, s, z, group).cuda()
    mags = ((q.double() + z.double().repeat_interleave(group, 1)) * s.double().abs().repeat_interleave(group, 1)).cuda()
    X = x.double().cuda()
    Q.close(got, X @ full.t(), (8 * math.sqrt(k) + 8) * Q.U * (X.abs() @ mags.t()) + 2 * k * 2.0 ** -150, "f32", (lo, hi))


def test_scales_beyond_the_type(gpu):
    x = torch.ones(20, 256)
    x[3, :128], x[5, 128:], x[7, 128] = 1e6, -2e6, 9.9e5
    for symmetric in (False, True):
        v = w4.w4_dequantize(w4.w4_quantize(x.cuda(), 128, symmetric=symmetric, dtype="f16"), "f32").cpu()
        bad = torch.zeros(20, 2, dtype=torch.bool)
        bad[3, 0] = bad[5, 1] = bad[7, 1] = True
        assert torch.equal(v.view(20, 2, 128).isnan().all(-1), bad) and torch.isfinite(v.view(20, 2, 128)[~bad]).all()
