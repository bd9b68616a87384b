"""Microscaled quantisation and products on the GPU against the 64-bit reference.

Quantisation is exact arithmetic: codes, scales and values have to be equal.
Products: with fp32 accumulation in any order the error of a sum of k terms is at most
k 2^-23 times the sum of the terms' magnitudes (2^-24 per addition, doubled because the
matrix unit's own additions may truncate); the bias adds one rounding, GELU's device form
2^-20 of its argument (one ulp each of exp2 and reciprocal, the argument's error scaled by
at most 30), the store half an ulp of D's type (2^-8 bf16, 2^-11 f16 and its 2^-25 floor)."""
import numpy as np
import pytest
import torch

from gemm_epilogues_epilog_amd import mx
from tests import mx_reference as ref

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rows_with_everything(R, K, dtype, seed):
    """Values over many magnitudes, exact ties, zeros, a zero block, signed zero, subnormals."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-8, 9, (R, K), generator=g).float())
    x[:, ::7] = torch.randint(-16, 17, (R, (K + 6) // 7), generator=g).float() / 4
    x[R // 2] = 0.0
    x[R // 3, : K // 2] = -0.0
    if R > 3:
        x[3] = x[3] * (2.0 ** -20 if dtype == "f16" else 2.0 ** -128 if dtype == "f32" else 2.0 ** -126)
    return x.to(T[dtype])


def from_device(q):
    c, s = q.codes.cpu().numpy().reshape(-1), q.scales.cpu().numpy().reshape(-1)
    return ref.unpack(c, s, q.rows, q.k, q.format)


SHAPES = [(1, 1), (1, 32), (2, 33), (31, 255), (32, 256), (33, 257), (100, 1101), (5, 4096), (65, 40)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,K", SHAPES)
def test_quantize_is_exact(gpu, R, K, dtype, fmt):
    x = rows_with_everything(R, K, dtype, R * 1000 + K)
    c, s = ref.quantize(x.double().numpy(), fmt)
    p, ps = ref.pack(c, s, fmt)
    wide = torch.zeros(R, 2 * K + 3, dtype=T[dtype], device="cuda")
    wide[:, 1:K + 1] = x.cuda()
    strided = torch.zeros(R, K, 2, dtype=T[dtype], device="cuda")
    strided[..., 0] = x.cuda()
    for name, t in (("rows", x.cuda()), ("unaligned rows", wide[:, 1:K + 1]), ("columns", x.cuda().t().contiguous().t()),
                    ("any strides", strided[..., 0])):
        q = mx.mx_quantize(t, fmt, out=filled(R, K, fmt))
        c2, s2 = from_device(q)
        assert np.array_equal(s2, s), name
        assert np.array_equal(c2, c), name
        # padding is written too
        assert np.array_equal(q.codes.cpu().numpy(), p) and np.array_equal(q.scales.cpu().numpy(), ps), name


def filled(R, K, fmt):
    q = mx.MXTensor.empty(R, K, fmt)
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    return q


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantize_infinities_and_nan(gpu, dtype, fmt):
    x = torch.ones(4, 96, dtype=T[dtype])
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2, 70] = -float("inf")
    q = mx.mx_quantize(x.cuda(), fmt)
    _, s = from_device(q)
    one = 127 - ref.EMAX[fmt]
    want = np.full((4, 3), one)
    want[0, 0] = want[1, 1] = want[2, 2] = 255
    assert np.array_equal(s, want)
    v = mx.mx_dequantize(q, "f32").cpu().numpy()
    assert np.array_equal(np.isnan(v), np.repeat(want == 255, 32, axis=1))
    assert (v[~np.isnan(v)] == 1).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quantize_largest_and_smallest(gpu, fmt):
    big = np.array([3.4028234663852886e38, -1e38, 1e37, 2.0 ** 126])
    small = np.array([2.0 ** -149, 2.0 ** -126, -2.0 ** -130, 1.5 * 2.0 ** -127])
    x = np.zeros((2, 64))
    x[0, :4], x[1, :4], x[1, 32] = big, small, 2.0 ** -149
    q = mx.mx_quantize(torch.tensor(x, dtype=torch.float32).cuda(), fmt)
    c, s = ref.quantize(x, fmt)
    c2, s2 = from_device(q)
    assert np.array_equal(s, s2) and np.array_equal(c, c2)
    v = mx.mx_dequantize(q, "f32").cpu().double().numpy()
    assert np.array_equal(v, ref.values(c, s, fmt))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,K", [(1, 1), (33, 257), (64, 512), (7, 40)])
def test_pack_and_dequantize_every_code(gpu, R, K, dtype, fmt):
    rng = np.random.default_rng(R + K)
    c = rng.integers(0, 16 if fmt == "mxfp4" else 256, (R, K)).astype(np.uint8)
    if fmt == "mxfp8":
        c[(c & 127) == 127] = 0
    s = rng.integers(117, 137, (R, -(-K // 32))).astype(np.uint8)
    s[0, 0] = 255
    rowmajor = c if fmt == "mxfp8" else np.pad(c, ((0, 0), (0, K % 2)))
    if fmt == "mxfp4":
        rowmajor = rowmajor[:, ::2] | rowmajor[:, 1::2] << 4
    q = mx.mx_pack(torch.tensor(rowmajor).cuda(), torch.tensor(s).cuda(), fmt, k=K)
    p, ps = ref.pack(c, s, fmt)
    assert np.array_equal(q.codes.cpu().numpy(), p) and np.array_equal(q.scales.cpu().numpy(), ps)
    want = torch.tensor(ref.values(c, s, fmt)).to(T[dtype])
    out = torch.full((R + 1, K + 3), 7.0, dtype=T[dtype], device="cuda")
    for got in (mx.mx_dequantize(q, dtype), mx.mx_dequantize(q, dtype, out=out[:R, :K])):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
    assert (out[R] == 7).all() and (out[:, K:] == 7).all()


# ---- products ---------------------------------------------------------------------------
def operands(m, n, k, x_format, seed, experts=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g)
    w = torch.randn(*((experts, n, k) if experts else (n, k)), generator=g) * k ** -0.5
    X = mx.mx_quantize(x.cuda(), x_format)
    W = mx.mx_quantize(w.cuda(), "mxfp4")
    xv = mx.mx_dequantize(X, "f32").cpu().double().numpy()
    wv = mx.mx_dequantize(W, "f32").cpu().double().numpy()
    b = torch.randn(*((experts, n) if experts else (n,)), generator=g)
    return X, W, xv, wv, b


def bound(xv, wv, want, k, ep, out):
    """Elementwise bound on |got - want| (see the module's text)."""
    mags = np.abs(xv) @ np.abs(wv).T
    err = (k + 2) * 2.0 ** -23 * mags + 2.0 ** -23 * np.abs(want)
    if ep == "GELU_BIAS":
        err = 1.13 * err + 2.0 ** -20 * (np.abs(want) + 1)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[out]
    return err * (1 + half) + half * np.abs(want) + (2.0 ** -25 if out == "f16" else 0) + 1e-37


def check(got, xv, wv, bias, k, ep, out, where=""):
    v = xv @ wv.T
    if ep != "NONE":
        v = v + bias
    want = ref.activate(v, ep)
    # the bias's rounding beside the sum's: both are covered by the sums' magnitudes with it
    e = np.abs(got.double().cpu().numpy() - want)
    b = bound(xv, wv, np.abs(want) + (np.abs(bias) if ep != "NONE" else 0), k, ep, out)
    assert (e <= b).all(), (where, float((e / b).max()), np.argwhere(e > b)[:4].tolist())


MNK = [(1, 1, 1), (1, 33, 300), (2, 64, 64), (15, 100, 512), (16, 257, 256), (17, 32, 1101), (33, 96, 129),
       (64, 130, 2048), (65, 130, 2048), (100, 257, 700), (129, 128, 257), (256, 512, 1024), (300, 777, 640),
       (1, 1024, 11008), (70, 96, 11008), (520, 260, 96)]
# ... and what takes the kernels that those leave out (see the reference's test)
MNK_TILES = [(5, 8200, 300), (40, 4100, 96), (130, 1000, 3300), (777, 130, 11008), (70, 8200, 96), (70, 16400, 96),
             (200, 16400, 96), (1000, 8200, 96), (200, 2050, 3300), (2200, 7300, 520)]


@pytest.mark.parametrize("x_format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,n,k", MNK + MNK_TILES)
def test_product(gpu, m, n, k, x_format):
    X, W, xv, wv, b = operands(m, n, k, x_format, m * 7 + n + k)
    for i, (ep, out) in enumerate([("NONE", "f32"), ("BIAS", "bf16"), ("RELU_BIAS", "f16"), ("GELU_BIAS", "f32")]):
        vec = "f32" if i == 1 else out
        bias = b.to(T[vec]).cuda()
        with mx.MXMatmul(n, k, x_format, ep, out, vec_dtype=vec) as mm:
            guard = torch.full((m + 2, n), 9.0, dtype=T[out], device="cuda")
            got = mm.execute(X, W, None if ep == "NONE" else bias, out=guard[1:m + 1])
            check(got, xv, wv, bias.double().cpu().numpy(), k, ep, out, (ep, out))
            assert (guard[0] == 9).all() and (guard[m + 1] == 9).all()
            again = mm.execute(X, W, None if ep == "NONE" else bias)
            assert torch.equal(got, again)


@pytest.mark.parametrize("m,n,k", [(8192, 512, 512), (4000, 1100, 300)])
@pytest.mark.parametrize("x_format", ["mxfp8", "mxfp4"])
def test_product_on_whole_numbers_is_exact(gpu, m, n, k, x_format):
    """Small whole numbers with power-of-two scales: every sum is exact in fp32."""
    g = torch.Generator().manual_seed(m + k)
    x = torch.randint(-2, 3, (m, k), generator=g).float() * torch.exp2(torch.randint(-2, 3, (m, 1), generator=g).float())
    w = torch.randint(-2, 3, (n, k), generator=g).float()
    X, W = mx.mx_quantize(x.cuda(), x_format), mx.mx_quantize(w.cuda(), "mxfp4")
    assert torch.equal(mx.mx_dequantize(X, "f32").cpu(), x) and torch.equal(mx.mx_dequantize(W, "f32").cpu(), w)
    with mx.MXMatmul(n, k, x_format, out="f32") as mm:
        got = mm.execute(X, W).cpu().double()
    assert torch.equal(got, x.double() @ w.double().t())


@pytest.mark.parametrize("x_format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (5, 33, 300), (64, 96, 256), (100, 512, 1000), (300, 800, 768),
                                   (2048, 4096, 256)])
@pytest.mark.parametrize("ep", ["NONE", "GELU_BIAS"])
def test_product_in_8_bits(gpu, m, n, k, x_format, ep):
    """The 8-bit result is the 32-bit result of the same product, quantised: the sums have
    the same order where the plans agree."""
    X, W, _, _, b = operands(m, n, k, x_format, m + n + k)
    bias = None if ep == "NONE" else b.cuda()
    with mx.MXMatmul(n, k, x_format, ep, "mxfp8") as m8, mx.MXMatmul(n, k, x_format, ep, "f32") as m32:
        out = filled(m, n, "mxfp8")
        m8.execute(X, W, bias, out=out)
        v = m32.execute(X, W, bias).cpu().double().numpy()
        a, c = m8.plan_info(m), m32.plan_info(m)
    got_c, got_s = from_device(out)
    want_c, want_s = ref.quantize(v, "mxfp8")
    if (a["tile_m"], a["tile_n"], a["splits"]) == (c["tile_m"], c["tile_n"], c["splits"]):
        assert np.array_equal(got_s, want_s) and np.array_equal(got_c, want_c)
    else:   # another order of the sums: a value may fall to the neighbouring element
        gv, wv = ref.values(got_c, got_s, "mxfp8"), ref.values(want_c, want_s, "mxfp8")
        top = np.repeat(np.exp2(want_s.astype(float) - 127), 32, axis=1)[:, :n]
        assert (np.abs(gv - wv) <= np.maximum(np.abs(wv) / 8, top * 2.0 ** -8) + 1e-30).all()
    # padding along n reads as zeros, so the result can be the next product's X
    full_c, full_s = ref.unpack(out.codes.cpu().numpy(), out.scales.cpu().numpy(), m, ref.pad(n, 256), "mxfp8")
    assert (full_c[:, n:] == 0).all() and (full_s[:, -(-n // 32):] == 0).all()


def test_product_nan_stays_in_its_row_and_column(gpu):
    for m in (3, 70, 300):
        x, w = torch.ones(m, 320), torch.ones(96, 320)
        x[1, 300], x[2, 5], w[7, 100] = float("nan"), float("inf"), float("inf")
        X, W = mx.mx_quantize(x.cuda(), "mxfp8"), mx.mx_quantize(w.cuda(), "mxfp4")
        with mx.MXMatmul(96, 320, "mxfp8", "RELU_BIAS", "f32") as mm:
            v = mm.execute(X, W, torch.zeros(96, device="cuda")).cpu()
        nan = torch.zeros(m, 96, dtype=torch.bool)
        nan[1], nan[2], nan[:, 7] = True, True, True
        # ReLU keeps a value only where it is > 0: of NaN it gives 0, as the framework's does
        assert (v[nan] == 0).all() and (v[~nan] == 320).all()
        with mx.MXMatmul(96, 320, "mxfp8", "NONE", "bf16") as mm:
            v = mm.execute(X, W).cpu()
        assert torch.equal(torch.isnan(v), nan) and (v[~nan] == 320).all()


def test_product_of_no_rows(gpu):
    X, W = mx.mx_quantize(torch.empty(0, 64, device="cuda"), "mxfp8"), mx.mx_quantize(torch.ones(32, 64, device="cuda"), "mxfp4")
    assert X.codes.numel() == 0
    with mx.MXMatmul(32, 64) as mm:
        assert mm.execute(X, W).shape == (0, 32)
    assert mx.mx_dequantize(X).shape == (0, 64)


# ---- by expert ---------------------------------------------------------------------------
def run_experts(counts, n, k, x_format, ep, out, offsets=None, seed=0):
    E, m = len(counts), sum(counts)
    X, W, xv, wv, b = operands(m, n, k, x_format, seed + m, experts=E)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    o = torch.tensor(off if offsets is None else offsets, dtype=torch.int32, device="cuda")
    with mx.MXMatmul(n, k, x_format, ep, out, experts=E, vec_dtype="f32") as mm:
        D = torch.full((m, n), 9.0, dtype=T[out], device="cuda")
        mm.execute(X, W, None if ep == "NONE" else b.cuda(), offsets=o, out=D)
    return D, xv, wv, b.double().numpy(), o.tolist()


COUNTS_TILES = [([40, 0, 1, 9], 4100, 96), ([100, 17, 0, 0], 520, 96), ([30, 131, 0, 139], 2050, 96),
                ([0, 129, 20, 51], 4100, 96), ([140, 0, 11, 49], 8200, 96), ([300, 0, 300, 0], 16400, 96),
                ([512, 0, 500], 16400, 520)]
COUNTS = [[1], [0, 1], [3, 0, 5, 1], [16, 17, 0, 31, 33], [0, 0, 200, 0], [1] * 40, [70, 1, 300, 0, 129],
          [257, 500, 31, 33, 64, 0, 900], [5] * 70 + [0, 900, 0]]


@pytest.mark.parametrize("x_format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
@pytest.mark.parametrize("n,k", [(96, 300), (300, 512)])
def test_experts(gpu, counts, n, k, x_format):
    for ep, out in (("GELU_BIAS", "f32"), ("BIAS", "bf16"), ("NONE", "f16")):
        D, xv, wv, b, off = run_experts(counts, n, k, x_format, ep, out)
        for e in range(len(counts)):
            if counts[e]:
                r = slice(off[e], off[e + 1])
                check(D[r], xv[r], wv[e], b[e], k, ep, out, (ep, out, e))


@pytest.mark.parametrize("x_format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,n,k", COUNTS_TILES, ids=lambda v: str(max(v)) if isinstance(v, list) else None)
def test_experts_in_every_tile(gpu, counts, n, k, x_format):
    for ep, out in (("RELU_BIAS", "f32"), ("NONE", "bf16")):
        D, xv, wv, b, off = run_experts(counts, n, k, x_format, ep, out)
        for e in range(len(counts)):
            if counts[e]:
                r = slice(off[e], off[e + 1])
                check(D[r], xv[r], wv[e], b[e], k, ep, out, (ep, out, e))


# a last round of at most a quarter of the device's large tiles, which smaller ones take: 260
# tiles of 256 x 256 on 256 compute units, empty experts and ragged ends among them
@pytest.mark.parametrize("x_format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", [[512, 0, 500], [0, 1010]], ids=str)
def test_experts_with_a_short_last_round(gpu, counts, x_format):
    n, k, E = 16400, 520, len(counts)
    m = sum(counts)
    i = mx.MXMatmul(n, k, x_format, "NONE", "f32", experts=E).plan_info(m)
    assert (i["tile_m"], i["tile_n"]) == (256, 256) and i["tiles"] > 256
    for ep, out in (("NONE", "f32"), ("GELU_BIAS", "bf16")):
        D, xv, wv, b, off = run_experts(counts, n, k, x_format, ep, out)
        for e in range(E):
            if counts[e]:
                r = slice(off[e], off[e + 1])
                check(D[r], xv[r], wv[e], b[e], k, ep, out, (ep, out, e))
    # the 8-bit result is the fp32 one's quantisation, its padding columns included
    X, W, _, _, _ = operands(m, n, k, x_format, m, experts=E)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    with mx.MXMatmul(n, k, x_format, "NONE", "f32", experts=E) as mm, \
            mx.MXMatmul(n, k, x_format, "NONE", "mxfp8", experts=E) as m8:
        want = mx.mx_quantize(mm.execute(X, W, offsets=o), "mxfp8")
        got = mx.MXTensor.empty(m, n, "mxfp8")
        got.codes.zero_(), got.scales.zero_()
        m8.execute(X, W, offsets=o, out=got)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


@pytest.mark.parametrize("m", [40, 700])
@pytest.mark.parametrize("offsets", [[5, 20, 20, 30], [-7, 10, 25, 5000], [30, 10, 12, 40], [0, 0, 0, 0],
                                     [2 ** 31 - 1, -2 ** 31, 3, 9]])
def test_experts_offsets_are_held_to_the_rows(gpu, m, offsets):
    D, xv, wv, b, _ = run_experts([m, 0, 0], 64, 300, "mxfp8", "BIAS", "f32", offsets=offsets)
    D = D.cpu()
    covered = torch.zeros(m, dtype=torch.bool)
    for e in range(3):
        lo = min(max(offsets[e], 0), m)
        hi = max(lo, min(offsets[e + 1], m))
        if hi > lo and not covered[lo:hi].any():
            check(D[lo:hi], xv[lo:hi], wv[e], b[e], 300, "BIAS", "f32", (e, lo, hi))
        covered[lo:hi] = True
    assert (D[~covered] == 9).all()


@pytest.mark.parametrize("counts", [[3, 0, 5], [100, 31, 0, 300]], ids=["few", "many"])
def test_experts_in_8_bits(gpu, counts):
    n, k, E, m = 320, 512, len(counts), sum(counts)
    X, W, _, _, b = operands(m, n, k, "mxfp8", 5, experts=E)
    off = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    with mx.MXMatmul(n, k, "mxfp8", "GELU_BIAS", "mxfp8", experts=E) as m8, \
            mx.MXMatmul(n, k, "mxfp8", "GELU_BIAS", "f32", experts=E) as m32:
        q = m8.execute(X, W, b.cuda(), offsets=off)
        v = m32.execute(X, W, b.cuda(), offsets=off).cpu().double().numpy()
    want_c, want_s = ref.quantize(v, "mxfp8")
    got_c, got_s = from_device(q)
    assert np.array_equal(got_s, want_s) and np.array_equal(got_c, want_c)


def test_streams_and_graph(gpu):
    """On another stream, and replayed from a graph with the program's own work between the
    replays: the same bits as the eager call each time."""
    cases = [(1, 256, 1024), (100, 256, 4096), (300, 512, 512)]
    for m, n, k in cases:
        X, W, _, _, b = operands(m, n, k, "mxfp8", 11)
        bias = b.to(torch.bfloat16).cuda()
        mm = mx.MXMatmul(n, k, "mxfp8", "GELU_BIAS", "bf16").plan()
        want = mm.execute(X, W, bias)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = mm.execute(X, W, bias, stream=s)
        s.synchronize()
        assert torch.equal(other, want)
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mm.execute(X, W, bias, out=out)
        for _ in range(4):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(mm.execute(X, W, bias), want)
        mm.free()


def test_binding_refusals(gpu):
    X, W, _, _, b = operands(4, 64, 96, "mxfp8", 1)
    X4 = mx.mx_quantize(torch.ones(4, 96, device="cuda"), "mxfp4")
    bias = b.to(torch.bfloat16).cuda()
    mm = mx.MXMatmul(64, 96, "mxfp8", "BIAS", "bf16").plan()
    for args in ((X4, W, bias), (W, W, bias), (X, X, bias), (X, W, None), (X, W, bias[:8]), (X, W, b.cuda()),
                 (X, W, bias.cpu())):
        with pytest.raises(ValueError):
            mm.execute(*args)
    with pytest.raises(ValueError):
        mm.execute(X, W, bias, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        mm.execute(X, W, bias, out=torch.empty(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        mm.execute(X, W, bias, out=torch.empty(64, 4, dtype=torch.bfloat16, device="cuda").t())
    mm.free()
    WE = mx.mx_quantize(torch.ones(2, 64, 96, device="cuda"), "mxfp4")
    mm = mx.MXMatmul(64, 96, "mxfp8", "NONE", "bf16", experts=2).plan()
    for o in (None, torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda"),
              torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            mm.execute(X, WE, offsets=o)
    with pytest.raises(ValueError):
        mm.execute(X, W, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    mm.free()
    for bad in (torch.ones(4, device="cuda"), torch.ones(4, 8, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            mx.mx_quantize(bad, "mxfp4")
    with pytest.raises(ValueError):
        mx.mx_quantize(torch.ones(4, 8, device="cuda"), "mxfp4", out=X4)
    with pytest.raises(ValueError):
        mx.mx_dequantize(X4, "bf16", out=torch.empty(4, 96, device="cuda"))
    with pytest.raises(ValueError):
        mx.mx_pack(torch.zeros(4, 16, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, dtype=torch.uint8, device="cuda"),
                   "mxfp4", k=40)


def test_operands_past_four_gib(gpu):
    """Offsets that pass 32 bits: quantisation, norm and product of 8.6 GB of rows give the
    last rows what they give them alone. Whole numbers, so every sum is exact."""
    from gemm_epilogues_epilog_amd.norm import rms_norm, rms_norm_backward
    k, n, last = 32768, 40, 96
    m = (1 << 17) + last
    row = torch.arange(k, device="cuda") % 5 - 2
    x = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    x.copy_(row.to(torch.bfloat16))
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-last:] = torch.randint(-2, 3, (last, k), generator=g, device="cuda").to(torch.bfloat16)
    tail = x[-last:].clone()
    X, T_ = mx.mx_quantize(x, "mxfp8"), mx.mx_quantize(tail, "mxfp8")
    assert torch.equal(X.codes[-last * k:], T_.codes) and torch.equal(X.scales[-last * k // 32:], T_.scales)
    assert torch.equal(mx.mx_dequantize(X, "bf16")[-last:], tail)
    W = mx.mx_quantize(torch.randint(-2, 3, (n, k), generator=g, device="cuda").float(), "mxfp4")
    with mx.MXMatmul(n, k, out="f32") as mm:
        D = mm.execute(X, W)
        want = tail.float() @ mx.mx_dequantize(W, "f32").T
        assert torch.equal(D[-last:], want) and torch.equal(D[0], D[1 << 16])
    with mx.MXMatmul(n, k, out="f32", experts=2) as mm:
        W2 = mx.MXTensor(torch.stack([W.codes, W.codes]), torch.stack([W.scales, W.scales]), n, k, "mxfp4", 2)
        off = torch.tensor([0, m - last, m], dtype=torch.int32, device="cuda")
        assert torch.equal(mm.execute(X, W2, offsets=off), D)
    del X, D
    w = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    y, _ = rms_norm(x, w, y_out=x)   # in place
    assert torch.equal(y[-last:], rms_norm(tail, w)[0])
    s = y[-last:].clone()
    dx, dw = rms_norm_backward(y, y, w, dx_out=y)
    assert torch.equal(dx[-last:], rms_norm_backward(s, s, w)[0]) and torch.isfinite(dw.float()).all()


@pytest.mark.parametrize("m,n,k,experts", [(2200, 7300, 520, None), (1012, 16400, 520, 3), (130, 1000, 3300, None)])
def test_graph_of_short_last_rounds_and_split_tiles(gpu, m, n, k, experts):
    """Products of two launches, and one whose parts of k meet through counters, replayed with
    eager work in between: every replay as the eager result."""
    X, W, _, _, b = operands(m, n, k, "mxfp8", 5, experts=experts)
    off = None if experts is None else torch.tensor([0, 512, 512, m], dtype=torch.int32, device="cuda")
    with mx.MXMatmul(n, k, "mxfp8", "GELU_BIAS", "bf16", vec_dtype="f32", experts=experts) as mm:
        i = mm.plan_info(m)
        assert i["splits"] > 1 or (i["tile_m"] == 256 and i["tiles"] > 256)
        want = mm.execute(X, W, b.cuda(), offsets=off).clone()
        out, bias = torch.empty_like(want), b.cuda()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mm.execute(X, W, bias, offsets=off, out=out)
        for _ in range(4):
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(mm.execute(X, W, bias, offsets=off), want)
