"""The norm and its gradient on the GPU against the 64-bit reference.

Bounds. The sum of squares of d values in fp32: relative error at most (log2 d + 8) 2^-24 of
a sum of positive terms added in a tree of short runs (64 lanes, at most 32 terms each);
through the square root half of that, then four more roundings. So |y - want| is at most
40 2^-24 |want|, and the store's half ulp. The gradient's inner sum has terms of both signs:
its error is 40 2^-24 of the sum of their magnitudes. dweight adds `rows` terms in fp32."""
import numpy as np
import pytest
import torch

from gemm_epilogues_epilog_amd import mx, norm
from tests import mx_reference as ref

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}
U = 40 * 2.0 ** -24
SHAPES = [(1, 1), (1, 7), (3, 64), (5, 511), (4, 512), (9, 1024), (333, 1100), (33, 1101), (40, 4096), (2, 8200),
          (3, 16384), (1, 32768), (2, 32767)]


def data(rows, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    make = lambda *s: torch.randn(*s, generator=g).to(T[dtype])   # noqa: E731
    return make(rows, d) * 2, make(rows, d), (1 + 0.3 * torch.randn(d, generator=g)), make(rows, d)


def close(got, want, err, dtype, where=""):
    e = np.abs(got.double().cpu().numpy() - want)
    b = err * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + TINY[dtype]
    assert (e <= b).all(), (where, float((e / b).max()))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(gpu, rows, d, dtype):
    x, res, w, _ = data(rows, d, dtype, rows + d)
    for wt in {dtype, "f32"}:
        wd = w.to(T[wt])
        s = (x.float() + res.float()).to(T[dtype])
        want = ref.rms_norm(s.double().numpy(), wd.double().numpy(), 1e-5)
        y, got_s = norm.rms_norm(x.cuda(), wd.cuda(), res.cuda(), eps=1e-5)
        assert torch.equal(got_s.cpu(), s)
        close(y, want, U * np.abs(want), dtype, wt)
        xc = x.cuda()
        y2, same = norm.rms_norm(xc, wd.cuda(), eps=1e-5)
        assert same is xc
        close(y2, ref.rms_norm(x.double().numpy(), wd.double().numpy(), 1e-5),
              U * np.abs(ref.rms_norm(x.double().numpy(), wd.double().numpy(), 1e-5)), dtype, wt)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_in_8_bits(gpu, rows, d, dtype):
    """q is y in 32 bits, quantised. From fp32 rows the same kernel gives that y itself, so
    the codes have to be equal; from 16-bit rows y comes back rounded, and the values are held
    to an element's spacing around the 64-bit result."""
    x, res, w, _ = data(rows, d, dtype, rows + d)
    q = mx.MXTensor.empty(rows, d, "mxfp8")
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    y, q, s = norm.rms_norm(x.cuda(), w.cuda(), res.cuda(), out="both", mx_out=q)
    c, sc = ref.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), rows, ref.pad(d, 256), "mxfp8")
    assert (c[:, d:] == 0).all() and (sc[:, -(-d // 32):] == 0).all()
    c, sc = c[:, :d], sc[:, : -(-d // 32)]
    if dtype == "f32":
        wc, ws = ref.quantize(y.cpu().double().numpy(), "mxfp8")
        assert np.array_equal(c, wc) and np.array_equal(sc, ws)
    want = ref.rms_norm(s.cpu().double().numpy(), w.double().numpy(), 1e-6)
    top = np.repeat(np.exp2(sc.astype(float) - 127), 32, axis=1)[:, :d]
    # half a step of an element (1/16 of it, or half the smallest), and 448 of up to 512 at the top
    assert (np.abs(ref.values(c, sc, "mxfp8") - want) <= np.maximum(np.abs(want) / 8, top * 2.0 ** -10) * (1 + U)).all()
    q2, s2 = norm.rms_norm(x.cuda(), w.cuda(), res.cuda(), out="mxfp8")
    c2, sc2 = ref.unpack(q2.codes.cpu().numpy(), q2.scales.cpu().numpy(), rows, d, "mxfp8")
    assert np.array_equal(c2, c) and np.array_equal(sc2, sc) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,d", SHAPES + [(1500, 520), (600, 4096)])
def test_backward(gpu, rows, d, dtype):
    s, dres, w, dy = data(rows, d, dtype, rows * 3 + d)
    for wt, dr in ((dtype, None), ("f32", dres)):
        wd = w.to(T[wt])
        S, W, DY = s.double().numpy(), wd.double().numpy(), dy.double().numpy()
        dx, dw = norm.rms_norm_backward(dy.cuda(), s.cuda(), wd.cuda(), None if dr is None else dr.cuda(), eps=1e-5)
        want_dx, want_dw = ref.rms_norm_backward(DY, S, W, 1e-5, None if dr is None else dr.double().numpy())
        r = 1 / np.sqrt(np.mean(S * S, axis=1, keepdims=True) + 1e-5)
        g, h = np.abs(DY * W), np.abs(S * r)
        err = 2 * U * r * (g + h * np.mean(g * h, axis=1, keepdims=True)) + (
            0 if dr is None else 2.0 ** -24 * np.abs(dr.double().numpy()))
        close(dx, want_dx, err, dtype, (wt, "dx"))
        mags = np.sum(np.abs(DY) * h, axis=0)
        close(dw, want_dw, (U + rows * 2.0 ** -24) * mags, wt, (wt, "dw"))
        again = norm.rms_norm_backward(dy.cuda(), s.cuda(), wd.cuda(), None if dr is None else dr.cuda(), eps=1e-5)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_strides_and_in_place(gpu):
    for d in (64, 1101):
        x, res, w, dy = data(37, d, "bf16", d)
        wide = torch.full((37, d + 5), 3.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 2:d + 2] = x.cuda()
        y0, s0 = norm.rms_norm(x.cuda(), w.cuda(), res.cuda())
        r = res.cuda()
        y1, s1 = norm.rms_norm(wide[:, 2:d + 2], w.cuda(), r, sum_out=r)
        assert s1 is r and torch.equal(y0, y1) and torch.equal(s0, r)
        v = wide[:, 2:d + 2]
        y2, s2 = norm.rms_norm(v, w.cuda(), res.cuda(), sum_out=v)
        assert torch.equal(y2, y0) and torch.equal(v, s0) and (wide[:, :2] == 3).all() and (wide[:, d + 2:] == 3).all()
        row = x.cuda()[:1].expand(37, d)   # one row for all
        y3, _ = norm.rms_norm(row, w.cuda(), res.cuda())
        y4, _ = norm.rms_norm(row.contiguous(), w.cuda(), res.cuda())
        assert torch.equal(y3, y4)
        dx0, dw0 = norm.rms_norm_backward(dy.cuda(), s0, w.cuda(), res.cuda())
        g = dy.cuda()
        dx1, dw1 = norm.rms_norm_backward(g, v, w.cuda(), res.cuda(), dx_out=g)
        assert dx1 is g and torch.equal(dx0, g) and torch.equal(dw0, dw1)


def test_no_rows(gpu):
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, s = norm.rms_norm(x, w)
    q, _ = norm.rms_norm(x, w, out="mxfp8")
    assert y.shape == (0, 64) and q.shape == (0, 64)
    dx, dw = norm.rms_norm_backward(x, x, w)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_special_rows(gpu):
    x = torch.ones(5, 96)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 4] = float("inf")
    w = torch.ones(96, device="cuda")
    y, q, _ = norm.rms_norm(x.cuda(), w, out="both", eps=0.0)
    y, v = y.cpu(), mx.mx_dequantize(q, "f32").cpu()
    assert (y[0] == 1).all() and (y[4] == 1).all() and (v[0] == 1).all() and (v[4] == 1).all()
    # a zero row without eps is 0 / 0; a row with a NaN is NaN; inf / inf is NaN and 1 / inf 0
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 4]) and (torch.cat((y[3, :4], y[3, 5:])) == 0).all()
    assert torch.isnan(v[1]).all() and torch.isnan(v[2]).all() and torch.isnan(v[3, :32]).all() and (v[3, 32:] == 0).all()
    y, _ = norm.rms_norm(x.cuda(), w, eps=1e-6)
    assert (y[1] == 0).all()


def test_streams_and_graph(gpu):
    x, res, w, dy = (t.cuda() for t in data(50, 4096, "bf16", 3))
    y, q, s = norm.rms_norm(x, w, res, out="both")
    dx, dw = norm.rms_norm_backward(dy, s, w, res)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2, q2, s2 = norm.rms_norm(x, w, res, out="both", stream=st)
    dx2, dw2 = norm.rms_norm_backward(dy, s2, w, res, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in ((y, y2), (s, s2), (dx, dx2), (dw, dw2)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3, q3, s3 = norm.rms_norm(x, w, res, out="both")
        dx3, dw3 = norm.rms_norm_backward(dy, s3, w, res)
    for _ in range(4):
        for t in (y3, s3, dx3, dw3):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in ((y, y3), (s, s3), (dx, dx3), (dw, dw3)))
        assert torch.equal(mx.mx_dequantize(q3), mx.mx_dequantize(q))


def test_binding_refusals(gpu):
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    h = x.half()
    for kw in (dict(residual=h), dict(residual=x[:2]), dict(residual=x.cpu()), dict(out="f16"), dict(sum_out=x),
               dict(mx_out=mx.MXTensor.empty(4, 64, "mxfp8")), dict(out="mxfp8", y_out=x),
               dict(residual=x, sum_out=x[:1].expand(4, 64)),
               dict(out="mxfp8", mx_out=mx.MXTensor.empty(4, 64, "mxfp4"))):
        with pytest.raises(ValueError):
            norm.rms_norm(x, w, **kw)
    for args in ((x.t(), w), (x, w[:8]), (x, w.half()), (x[0], w), (x.double(), w)):
        with pytest.raises(ValueError):
            norm.rms_norm(*args)
    for args in ((h, x, w), (x[:2], x, w), (x, x, w.double()), (x, x, w, h)):
        with pytest.raises(ValueError):
            norm.rms_norm_backward(*args)


@pytest.mark.parametrize("rows", [4, 5, 33])
@pytest.mark.parametrize("d", [64, 256, 700])
def test_rows_that_share_a_workgroup_in_8_bits(gpu, d, rows):
    """Narrow rows to MXFP8, four to a workgroup, with an odd number of 256-value granules: each
    row's part of the LDS begins on 16 bytes. From fp32 rows the codes are y's, quantised."""
    x, res, w, _ = data(rows, d, "f32", rows + d)
    y, q, _ = norm.rms_norm(x.cuda(), w.cuda(), res.cuda(), out="both")
    c, s = ref.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), rows, d, "mxfp8")
    wc, ws = ref.quantize(y.cpu().double().numpy(), "mxfp8")
    assert np.array_equal(c, wc) and np.array_equal(s, ws)


def test_more_rows_than_a_launch_of_waves_takes(gpu):
    """537 million rows of one value: more lanes than one launch has."""
    rows = 537_000_001
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    res = torch.empty_like(x).normal_(generator=g)
    w = torch.full((1,), 1.5, device="cuda")
    y, s = norm.rms_norm(x, w, res, eps=0.25)
    for r in range(0, rows, 1 << 26):
        part = slice(r, min(rows, r + (1 << 26)))
        f = x[part].float() + res[part].float()
        assert torch.equal(s[part], f.to(torch.bfloat16))
        f = s[part].double()
        want = f / torch.sqrt(f * f + 0.25) * 1.5
        b = want.abs() * (U * (1 + HALF["bf16"]) + HALF["bf16"]) + TINY["bf16"]
        assert ((y[part].double() - want).abs() <= b).all()


def codes_of(y, fmt="mxfp8"):
    """(codes, scales) of y (rows, d) in 64 bits on the device, as the reference's quantize."""
    t = torch.tensor(ref.ELEMENTS[fmt], device=y.device)
    d = y.shape[1]
    p = torch.nn.functional.pad(y.double(), (0, -d % 32)).view(y.shape[0], -1, 32)
    top = p.abs().amax(-1)
    s = torch.where(top == 0, 0, (torch.frexp(top)[1] - 1 - ref.EMAX[fmt] + 127).clamp(0, 254))
    a = (p.abs() * torch.exp2(127.0 - s.double())[..., None]).clamp(max=float(t[-1]))
    hi = torch.searchsorted(t, a).clamp(max=len(t) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = t[hi] - a, a - t[lo]
    c = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo) + 128 * torch.signbit(p)
    return c.view(y.shape[0], -1)[:, :d].to(torch.uint8), s.to(torch.uint8)


def unpacked(q):
    """Row-major codes and scales of an MXFP8 operand, on the device."""
    r, kp = -(-q.rows // 32) * 32, -(-q.k // 256) * 256
    c = q.codes.view(r // 32, kp // 16, 32, 16).transpose(1, 2).reshape(r, kp)
    s = q.scales.view(r // 32, kp // 256, 2, 32, 4).permute(0, 3, 1, 4, 2).reshape(r, kp // 32)
    return c[: q.rows, : q.k], s[: q.rows, : -(-q.k // 32)]


def test_device_forms_of_the_reference(gpu):
    x = torch.randn(70, 300, generator=torch.Generator().manual_seed(2)) * 3
    x[3, 32:64] = 0
    c, s = ref.quantize(x.double().numpy(), "mxfp8")
    c2, s2 = codes_of(x.cuda())
    assert np.array_equal(c2.cpu().numpy(), c) and np.array_equal(s2.cpu().numpy(), s)
    c3, s3 = unpacked(mx.mx_quantize(x.cuda(), "mxfp8"))
    assert torch.equal(c3, c2) and torch.equal(s3, s2)


# enough rows for a row slot to take two, four or eight one after the other, the last slot fewer
@pytest.mark.parametrize("rows,d,unaligned", [(2051, 1101, True), (4099, 2048, False), (8195, 4096, False),
                                              (8200, 520, False), (8201, 519, True), (33001, 300, True),
                                              (16389, 8192, False), (9001, 6000, False), (2049, 12000, False),
                                              (4100, 16001, True), (2050, 32768, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(gpu, rows, d, unaligned, dtype):
    """Row slots that take several rows: the next row's loads in flight, an 8-bit result
    gathered in LDS, a last slot with fewer rows. In place, and with rows at any alignment."""
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    wide = d + (3 if unaligned else 0)
    make = lambda: torch.randn(rows, wide, generator=g, device="cuda").to(T[dtype])[:, :d]   # noqa: E731
    x, res = make(), make()
    w = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    want_s = (x.float() + res.float()).to(T[dtype])
    q = mx.MXTensor.empty(rows, d, "mxfp8")
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    y, q, s = norm.rms_norm(x, w, res, eps=1e-5, out="both", sum_out=res, mx_out=q)
    assert s is res and torch.equal(s, want_s)
    c, sc = unpacked(q)
    for r in range(0, rows, 1024):
        part = slice(r, min(rows, r + 1024))
        f = want_s[part].double()
        want = f / torch.sqrt((f * f).mean(1, keepdim=True) + 1e-5) * w.double()
        b = want.abs() * (U * (1 + HALF[dtype]) + HALF[dtype]) + TINY[dtype]
        assert ((y[part].double() - want).abs() <= b).all(), r
        if dtype == "f32":   # y is what was quantised
            wc, ws = codes_of(y[part])
            assert torch.equal(c[part], wc) and torch.equal(sc[part], ws), r
        else:   # a value near the middle of two elements may fall to either
            top = torch.exp2(sc[part].double() - 127).repeat_interleave(32, 1)[:, :d]
            v = mx.mx_dequantize(q, "f32")[part].double()
            assert ((v - want).abs() <= torch.maximum(want.abs() / 8, top * 2.0 ** -10) * (1 + U)).all(), r
    q2, _ = norm.rms_norm(want_s, w, eps=1e-5, out="mxfp8")
    c2, s2 = unpacked(q2)
    assert torch.equal(c2, c) and torch.equal(s2, sc)


@pytest.mark.parametrize("rows,d", [(2500, 300), (5000, 512), (2051, 64), (3001, 1100), (1100, 2050), (300, 8191),
                                    (600, 16384), (300, 32767)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_of_many_rows(gpu, rows, d, dtype):
    """Row slots that take several rows, several slots to a workgroup."""
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    make = lambda: torch.randn(rows, d, generator=g, device="cuda").to(T[dtype])   # noqa: E731
    s, dy, dres = make() * 2, make(), make()
    w = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    dx, dw = norm.rms_norm_backward(dy, s, w, dres, eps=1e-5)
    S, G, R, W = s.double(), dy.double(), dres.double(), w.double()
    r = 1 / torch.sqrt((S * S).mean(1, keepdim=True) + 1e-5)
    gw, h = G * W, S * r
    want = r * (gw - h * (gw * h).mean(1, keepdim=True)) + R
    err = 2 * U * r * (gw.abs() + h.abs() * (gw * h).abs().mean(1, keepdim=True)) + 2.0 ** -24 * R.abs()
    assert ((dx.double() - want).abs() <= err * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + TINY[dtype]).all()
    mags = (G * h).abs().sum(0)
    assert ((dw.double() - (G * h).sum(0)).abs() <= (U + rows * 2.0 ** -24) * mags * (1 + HALF["f32"]) + TINY["f32"]).all()
