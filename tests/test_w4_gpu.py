"""4-bit weights with group scales on the GPU against the formulas in 64 bits.

Quantising is exact arithmetic on 16-bit weights (a quotient of two 16-bit numbers lies either
on a border between codes or 2^-16 of itself away from it, so the fp32 quotient rounds as the
exact one) and is compared code by code. Products: each sum is taken over q and over z apart,
so its terms' magnitudes add up to S = sum s |x| (q + z); k additions in fp32 stay within
8 sqrt(k) 2^-24 S (independent rounding errors, 8 standard deviations), then the activation's few
units and 2 |g| of them through its exponential, and half a step of the result."""
import math

import numpy as np
import pytest
import torch

from gemm_epilogues_epilog_amd import w4

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}
U = 2.0 ** -24


def quantize64(x, group, symmetric, dtype):
    """Row-major codes, scales and zeros of x (rows, k) in 64 bits."""
    rows, k = x.shape
    G = -(-k // group)
    q, s, z = torch.zeros(rows, k), torch.zeros(rows, G, dtype=torch.float64), torch.zeros(rows, G)
    for g in range(G):
        v = x[:, g * group:(g + 1) * group]
        lo, hi = v.min(1).values.clamp(max=0), v.max(1).values.clamp(min=0)
        w = torch.maximum(-lo, hi) / 7 if symmetric else (hi - lo) / 15
        w = w.float().to(T[dtype]).double()
        one = torch.where(w > 0, w, torch.ones_like(w))
        zz = torch.full_like(w, 8.0) if symmetric else torch.round(-lo / one).clamp(max=15)
        c = (torch.round(v / one[:, None]) + zz[:, None]).clamp(0, 15)
        c = torch.where(w[:, None] > 0, c, zz[:, None].expand_as(c))
        bad = ~torch.isfinite(v).all(1)
        w[bad] = float("nan")
        zz[bad] = 8.0 if symmetric else 0.0
        c[bad] = zz[bad][:, None]
        q[:, g * group:(g + 1) * group], s[:, g], z[:, g] = c, w, zz
    return q.to(torch.uint8), s, z.to(torch.uint8)


def nibbles(q):
    """(rows, k) codes two to a byte, even k low."""
    rows, k = q.shape
    p = torch.zeros(rows, k + k % 2, dtype=torch.uint8)
    p[:, :k] = q
    return p[:, 0::2] | (p[:, 1::2] << 4)


def unpack(W):
    """Row-major codes, scales, zeros of the layout, each element looked up where the header says."""
    halves = 2 if W.gated else 1
    n, kt, G = W.rows // halves, -(-W.k // 128), -(-W.k // W.group)
    rg = -(-n // 16)
    r, k = torch.arange(n)[:, None], torch.arange(W.k)[None, :]
    codes, scales, zeros = W.codes.cpu(), W.scales.cpu(), W.zeros.cpu()
    out = []
    for h in range(halves):
        at = ((h * rg + r // 16) * kt + k // 128) * 1024 + (k % 32 // 8) * 256 + (r % 16) * 16 + (k % 128 // 32) * 4 + k % 4
        c = (codes[at] >> torch.where(k % 8 < 4, 0, 4).to(torch.uint8)) & 15
        g = torch.arange(G)[None, :]
        i = ((h * rg + r // 16) * G + g) * 16 + r % 16
        out.append((c, scales[i], zeros[i]))
    return [torch.cat([o[i] for o in out]) for i in range(3)]


def values64(q, s, z, group):
    k = q.shape[1]
    return (q.double() - z.double().repeat_interleave(group, 1)[:, :k]) * s.double().repeat_interleave(group, 1)[:, :k]


WEIGHTS = [(1, 1, 32), (3, 31, 32), (16, 128, 128), (17, 129, 64), (40, 200, 32), (33, 300, 128), (50, 1000, 256),
           (20, 777, 1024), (130, 520, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,k,group", WEIGHTS)
def test_quantize_and_back(gpu, rows, k, group, dtype):
    g = torch.Generator().manual_seed(rows + k)
    x = (torch.randn(rows, k, generator=g) * torch.rand(rows, 1, generator=g)).to(T[dtype])
    x[rows // 2] = 0
    x[-1, :1] = 3.0
    for sym in (False, True):
        for gated in (False, True):
            if gated and rows % 2:
                continue
            W = w4.w4_quantize(x.cuda(), group, symmetric=sym, gated=gated)
            got = unpack(W)
            want = quantize64(x.double(), group, sym, dtype)
            assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
            assert torch.equal(got[1].double(), want[1])
            v = values64(*want, group)
            assert torch.equal(w4.w4_dequantize(W, "f32").cpu(), v.float())
            assert torch.equal(w4.w4_dequantize(W).cpu(), v.float().to(T[dtype]))
            P = w4.w4_pack(nibbles(want[0]).cuda(), want[1].to(T[dtype]).cuda(), want[2].cuda(), group, k, gated)
            for p, q in ((P.codes, W.codes), (P.scales, W.scales), (P.zeros, W.zeros)):
                assert torch.equal(p, q)
    P = w4.w4_pack(nibbles(want[0]).cuda(), want[1].to(T[dtype]).cuda(), None, group, k)
    assert (unpack(P)[2] == 8).all()


def test_quantize_f32_strides_and_special(gpu):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(37, 300, generator=g)
    x[0, 5], x[1, 200], x[2] = float("nan"), float("inf"), 0
    x[3, :128] = -2.0
    x[4, :128] = 5.0
    big = torch.full((37, 310), 9.0, device="cuda")
    big[:, 3:303] = x.cuda()
    for dtype in ("f16", "bf16"):
        W = w4.w4_quantize(big[:, 3:303], 128, dtype=dtype)
        q, s, z = unpack(W)
        wq, ws, wz = quantize64(x.double(), 128, False, dtype)
        # (an fp32 quotient may round to a border that the exact one misses: one step there)
        assert (q.int() - wq.int()).abs().max() <= 1 and (q != wq).float().mean() < 1e-3
        assert torch.equal(torch.nan_to_num(s.double(), -1), torch.nan_to_num(ws, -1)) and torch.equal(z, wz)
        v = w4.w4_dequantize(W, "f32").cpu()
        assert v[0, :128].isnan().all() and not v[0, 128:].isnan().any() and v[1, 128:256].isnan().all()
        assert (v[2] == 0).all()
        assert (v[3, :128] + 2).abs().max() <= 2 * HALF[dtype] and (v[4, :128] - 5).abs().max() <= 5 * HALF[dtype]
        row = torch.empty(1, 300, device="cuda").copy_(x[5:6].cuda()).expand(3, 300)   # one row for all
        assert torch.equal(w4.w4_dequantize(w4.w4_quantize(row, 64, dtype=dtype)),
                           w4.w4_dequantize(w4.w4_quantize(row.contiguous(), 64, dtype=dtype)))


def make(m, n, k, group, dtype, seed, gated=False, zeros=True):
    g = torch.Generator().manual_seed(seed)
    rows = 2 * n if gated else n
    q = torch.randint(0, 16, (rows, k), generator=g).to(torch.uint8)
    G = -(-k // group)
    s = ((0.5 + torch.rand(rows, G, generator=g)) * k ** -0.5 / 4).to(T[dtype])
    z = torch.randint(0, 16, (rows, G), generator=g).to(torch.uint8) if zeros else torch.full((rows, G), 8, dtype=torch.uint8)
    x = torch.randn(m, k, generator=g).to(T[dtype])
    b = (torch.randn(rows, generator=g) * 0.5).to(T[dtype])
    W = w4.w4_pack(nibbles(q).cuda(), s.cuda(), z.cuda() if zeros else None, group, k, gated)
    full = values64(q, s, z, group).cuda()
    mags = (q.double() + z.double().repeat_interleave(group, 1)[:, :k]).cuda() * \
        s.double().repeat_interleave(group, 1)[:, :k].cuda()
    return x.cuda(), W, b.cuda(), full, mags


def act64(v, act):
    if act in ("NONE", "BIAS"):
        return v
    if act.startswith("RELU"):
        return v.clamp(min=0)
    return v * torch.sigmoid(v if act == "SILU" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))


def close(got, want, err, dtype, where=""):
    e = (got.double() - want).abs()
    bound = err * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + TINY[dtype]
    assert torch.isfinite(got.double()).all(), where
    assert (e <= bound).all(), (where, float((e / bound).max()))


def check(x, W, b, full, mags, dtype, eps, where=""):
    k = x.shape[1]
    X = x.double()
    for ep, out in eps:
        bias = None if ep == "NONE" else b
        got = w4.w4_matmul(x, W, bias, epilog=ep, out_dtype=out)
        v = X @ full.t() + (0 if bias is None else b.double())
        err = (8 * math.sqrt(k) + 8) * U * (X.abs() @ mags.t() + b.double().abs())
        a = act64(v, ep)
        if ep == "GELU_BIAS":
            err = 1.13 * err + (10 + 4 * v.abs()) * U * a.abs()
        close(got, a, err, out or dtype, (where, ep, out))


def check_gated(x, W, b, full, mags, dtype, acts, where=""):
    n, k = full.shape[0] // 2, x.shape[1]
    X = x.double()
    for act, bias in acts:
        got = w4.w4_gated(x, W, b if bias else None, act=act)
        v = X @ full.t() + (b.double() if bias else 0)
        err = (8 * math.sqrt(k) + 8) * U * (X.abs() @ mags.t() + b.double().abs())
        G, V = v[:, :n], v[:, n:]
        a = act64(G, act)
        e = 1.13 * err[:, :n] * (V.abs() + err[:, n:]) + a.abs() * err[:, n:] + (10 + 4 * G.abs()) * U * (a * V).abs()
        close(got, a * V, e, dtype, (where, act))


SHAPES = [(1, 1, 1, 32), (1, 16, 128, 128), (1, 100, 1000, 64), (3, 33, 31, 32), (16, 48, 384, 128), (17, 70, 136, 32),
          (24, 1101, 1000, 32), (33, 250, 520, 64), (64, 128, 2048, 256), (65, 130, 129, 64), (100, 257, 640, 128),
          (129, 300, 777, 1024), (200, 512, 256, 32), (300, 264, 1000, 64), (513, 136, 392, 128)]
EPS = [("NONE", None), ("BIAS", "f32"), ("RELU_BIAS", None), ("GELU_BIAS", "f32"), ("GELU_BIAS", None)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_matmul(gpu, m, n, k, group, dtype):
    for zeros in (True, False):
        a = make(m, n, k, group, dtype, m + n + k, zeros=zeros)
        check(*a, dtype, EPS if zeros else EPS[:2])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_gated(gpu, m, n, k, group, dtype):
    a = make(m, n, k, group, dtype, m + 2 * n + k, gated=True)
    check_gated(*a, dtype, [("SILU", True), ("GELU", False), ("RELU", True)])


# 256 x 256, 192 x 256, 128 x 128 and 64 x 128 tiles: more than one of each, ragged rows, columns and k, an odd
# number of k-tiles, one k-tile, groups longer than k
TILES = [(1030, 8208, 392, 64), (1030, 8208, 520, 128), (2100, 4100, 64, 64), (1000, 4130, 456, 32), (1290, 8300, 131, 128),
         (900, 5000, 130, 32), (700, 1500, 1100, 256), (130, 260, 2000, 64), (66, 1000, 24, 1024), (257, 4099, 333, 64),
         (2900, 4104, 264, 128), (2900, 4104, 264, 64), (2900, 4104, 64, 64), (1340, 8200, 200, 64), (300, 20000, 136, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,group", TILES)
def test_tiles(gpu, m, n, k, group, dtype):
    check(*make(m, n, k, group, dtype, m + n + k), dtype, [("GELU_BIAS", None), ("BIAS", "f32")])
    check_gated(*make(m, n // 2, k, group, dtype, m + n, gated=True), dtype, [("SILU", True), ("RELU", False)])


# k that ends in its first chunk of eight, at its end, just past it and inside a later one; fewer than
# eight; the middle and small tiles with every size of group
ENDS = [(1000, 4130, 9, 64), (1290, 8300, 8, 64), (900, 5000, 135, 64), (257, 4099, 8, 32), (300, 2000, 257, 32), (257, 4099, 15, 128),
        (700, 1500, 127, 32), (2000, 700, 7, 32), (300, 264, 1, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,group", ENDS)
def test_ends_of_k(gpu, m, n, k, group, dtype):
    check(*make(m, n, k, group, dtype, m + n + k), dtype, [("BIAS", "f32")])
    check_gated(*make(m, n // 2, k, group, dtype, m + n, gated=True), dtype, [("SILU", True)])


@pytest.mark.parametrize("m,n,k", [(300, 1000, 260), (1030, 5000, 133), (7, 100, 260)])
def test_nothing_past_a_row(gpu, m, n, k):
    """X inside a tensor of NaN: nothing beside its rows reaches a result."""
    x, W, b, full, mags = make(m, n, k, 64, "bf16", 9)
    buf = torch.full((m * k + 64,), float("nan"), device="cuda", dtype=torch.bfloat16)
    for at in (0, 1, 24):
        y = buf[at:at + m * k].view(m, k)
        y.copy_(x)
        check(y, W, b, full, mags, "bf16", [("BIAS", "f32")], at)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 20, 100, 600, 2100])
@pytest.mark.parametrize("group", [32, 128])
def test_scales_far_apart(gpu, m, group, dtype):
    """Zero scales, scales from the type's smallest to large ones, negative ones, beside each other in
    a row; a NaN and an infinite scale reach their own column alone."""
    n, k = 4200, 512
    g = torch.Generator().manual_seed(m)
    G = k // group
    q = torch.randint(0, 16, (n, k), generator=g).to(torch.uint8)
    z = torch.randint(0, 16, (n, G), generator=g).to(torch.uint8)
    lo, hi = (-24, 12) if dtype == "f16" else (-60, 40)
    s = torch.exp2(torch.randint(lo, hi, (n, G), generator=g).double()) * (1 + torch.randint(0, 8, (n, G), generator=g) / 8)
    s = s * torch.where(torch.rand(n, G, generator=g) < 0.3, -1.0, 1.0) * (torch.rand(n, G, generator=g) > 0.2)
    s = s.to(T[dtype])
    s[7], s[9, 0], s[11, 1] = 0, float("nan"), float("inf")
    x = torch.randn(m, k, generator=g).to(T[dtype])
    W = w4.w4_pack(nibbles(q).cuda(), s.cuda(), z.cuda(), group)
    got = w4.w4_matmul(x.cuda(), W, out_dtype="f32")
    assert got[:, 9].isnan().all() and not torch.isfinite(got[:, 11]).any() and (got[:, 7] == 0).all()
    keep = [i for i in range(n) if i not in (9, 11)]
    s2 = s.double()[keep]
    full = values64(q[keep], s2, z[keep], group).cuda()
    mags = ((q[keep].double() + z[keep].double().repeat_interleave(group, 1)) * s2.abs().repeat_interleave(group, 1)).cuda()
    X = x.double().cuda()
    close(got[:, keep], X @ full.t(), (8 * math.sqrt(k) + 8) * U * (X.abs() @ mags.t()), "f32")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 5, 40, 200, 2100])
def test_exact_sums(gpu, m, dtype):
    """Whole numbers small enough for exact fp32 sums: equal, whatever the order."""
    n, k, group = (70 if m < 1000 else 4200), 500, 64
    g = torch.Generator().manual_seed(m)
    q = torch.randint(0, 16, (n, k), generator=g).to(torch.uint8)
    s = torch.exp2(torch.randint(0, 3, (n, -(-k // group)), generator=g).float()).to(T[dtype])
    z = torch.randint(0, 16, s.shape, generator=g).to(torch.uint8)
    x = torch.randint(-4, 5, (m, k), generator=g).to(T[dtype])
    W = w4.w4_pack(nibbles(q).cuda(), s.cuda(), z.cuda(), group, k)
    want = x.double() @ values64(q, s, z, group).t()   # below 4 15 4 500 < 2^24
    assert torch.equal(w4.w4_matmul(x.cuda(), W, out_dtype="f32").cpu().double(), want)


@pytest.mark.parametrize("m", [1, 40, 200])
def test_rows_stay_apart(gpu, m):
    """NaN and infinities in a token's row or in a group's scale reach their own results only;
    unaligned X and D; nothing is written behind D."""
    x, W, b, full, mags = make(m, 50, 300, 64, "bf16", 2)
    x[m // 2, 7] = float("nan")
    D = w4.w4_matmul(x, W, out_dtype="f32")
    assert D[m // 2].isnan().all()
    keep = [i for i in range(m) if i != m // 2]
    if keep:
        assert torch.isfinite(D[keep]).all()
    buf = torch.full((m * 300 + 9,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x2 = buf[1:1 + m * 300].view(m, 300)
    x2.copy_(x.nan_to_num(0.5))
    out = torch.full((m * 50 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    d = out[3:3 + m * 50].view(m, 50)
    w4.w4_matmul(x2, W, out=d)
    aligned = w4.w4_matmul(x2.clone(), W)
    assert torch.equal(d, aligned) and (out[:3] == 7).all() and (out[3 + m * 50:] == 7).all()


@pytest.mark.parametrize("m,n", [(1, 50), (17, 70), (40, 50), (200, 500), (700, 1500), (2100, 4104)])
def test_infinities_in_a_token(gpu, m, n):
    x, W, b, full, mags = make(m, n, 264, 64, "bf16", 4)
    x[m // 2, 7], x[m // 2, 200] = float("inf"), -float("inf")
    D = w4.w4_matmul(x, W, out_dtype="f32")
    assert not torch.isfinite(D[m // 2]).any()
    keep = [i for i in range(m) if i != m // 2]
    X = x[keep].double()
    close(D[keep], X @ full.t(), (8 * math.sqrt(264) + 8) * U * (X.abs() @ mags.t()), "f32")


def test_no_rows(gpu):
    x, W, b, *_ = make(1, 20, 40, 32, "f16", 1)
    assert w4.w4_matmul(x[:0], W).shape == (0, 20)
    x, W, b, *_ = make(1, 20, 40, 32, "f16", 1, gated=True)
    assert w4.w4_gated(x[:0], W).shape == (0, 20)


@pytest.mark.parametrize("m", [1, 48, 300])
def test_streams_and_graphs(gpu, m):
    x, W, b, *_ = make(m, 264, 520, 128, "bf16", 5)
    xg, Wg, bg, *_ = make(m, 136, 520, 64, "bf16", 6, gated=True)
    ref = (w4.w4_matmul(x, W, b, epilog="BIAS"), w4.w4_gated(xg, Wg, bg))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = (w4.w4_matmul(x, W, b, epilog="BIAS", stream=side), w4.w4_gated(xg, Wg, bg, stream=side))
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    wt = torch.randn(264, 520, device="cuda").bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4_quantize(wt, out=W)
        d = w4.w4_matmul(x, W, b, epilog="BIAS")
        h = w4.w4_gated(xg, Wg, bg)
    for i in range(4):
        d.fill_(7.0)
        h.fill_(7.0)
        wt.copy_(wt.roll(1, 0))
        x.copy_(x.roll(1, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, w4.w4_matmul(x, w4.w4_quantize(wt), b, epilog="BIAS")) and torch.equal(h, ref[1])


def test_offsets_past_4_gib(gpu):
    """D of 4.3 GB: rows from its start, around its middle and at its end, by the bounds above (fewer
    rows alone may run in another tile, whose sums go in another order)."""
    m, n, k = 66000, 16400, 32
    x, W, b, full, mags = make(m, n, k, 32, "bf16", 3)
    D = w4.w4_matmul(x, W, out_dtype="f32")
    for r in (0, 32740, 65500, m - 120):
        X = x[r:r + 120].double()
        close(D[r:r + 120], X @ full.t(), (8 * math.sqrt(k) + 8) * U * (X.abs() @ mags.t()), "f32", r)


def test_refusals(gpu):
    x, W, b, *_ = make(4, 20, 64, 32, "bf16", 1)
    _, Wg, bg, *_ = make(4, 20, 64, 32, "bf16", 1, gated=True)
    z = lambda *s, t=torch.uint8: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    mm = w4.w4_matmul
    for bad in (lambda: mm(x.half(), W), lambda: mm(x[:, :63], W), lambda: mm(x[:, :32].contiguous(), W), lambda: mm(x.cpu(), W),
                lambda: mm(x, Wg), lambda: w4.w4_gated(x, W), lambda: mm(x, W, b), lambda: mm(x, W, epilog="BIAS"),
                lambda: mm(x, W, b, epilog="RELU_AUX_BIAS"), lambda: mm(x, W, out_dtype="f16"), lambda: mm(x, W, b[:19], epilog="BIAS"),
                lambda: mm(x, W, out=z(4, 20, t=torch.float32)), lambda: w4.w4_gated(x, Wg, act="NONE"), lambda: mm(x, x),
                lambda: w4.w4_gated(x, Wg, bg[:39]),
                lambda: w4.w4_quantize(x, 48), lambda: w4.w4_quantize(x, 0), lambda: w4.w4_quantize(x.float(), 32),
                lambda: w4.w4_quantize(x[:3], 32, gated=True), lambda: w4.w4_quantize(x.t(), 32),
                lambda: w4.w4_quantize(x, 32, dtype="f32"), lambda: w4.w4_quantize(x, 32, out=W),
                lambda: w4.w4_pack(z(4, 32), z(4, 1, t=torch.bfloat16), k=65), lambda: w4.w4_pack(z(4, 32), z(4, 2, t=torch.bfloat16)),
                lambda: w4.w4_pack(z(4, 32), z(4, 1, t=torch.float32)), lambda: w4.w4_pack(z(4, 32), z(4, 1, t=torch.bfloat16), z(4, 2)),
                lambda: w4.w4_dequantize(W, "f64"), lambda: w4.w4_dequantize(x),
                lambda: w4.W4Tensor(W.codes[:-1], W.scales, W.zeros, 20, 64, 32),
                lambda: w4.W4Tensor(W.codes, W.scales.float(), W.zeros, 20, 64, 32)):
        with pytest.raises(ValueError):
            bad()
