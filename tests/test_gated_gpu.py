"""The gated feed-forward block on the GPU against the formulas in 64 bits.

Bounds. u = 2^-24. A sum of k products in fp32: every addition is off by at most u of a partial
sum, which is at most S, the sum of the products' magnitudes; the errors are independent in
sign, so k of them stay within 8 sqrt(k) u S (Hoeffding: 8 standard deviations, 1e-13 of the
elements). The activation's exponential is off by a few u and by 2 |g| u through its argument.
The gradients go through dZ rounded to the matrices' type: each term of a sum is then off by
half a step of dZ, independently, so the sum by 8 times the root of the sum of their squares.
Results are rounded once more, by half a step."""
import math

import numpy as np
import pytest
import torch

from gemm_epilogues_epilog_amd import gated

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}
U = 2.0 ** -24
ACTS = ["SILU", "GELU", "RELU"]
C = 2 * math.sqrt(2 / math.pi)


def act64(g, act):
    """a(g) and its slope."""
    if act == "RELU":
        return g.clamp(min=0), (g > 0).double()
    u, du = (g, torch.ones_like(g)) if act == "SILU" else (C * (g + 0.044715 * g ** 3), C * (1 + 3 * 0.044715 * g ** 2))
    p = torch.sigmoid(u)
    return g * p, p + g * p * (1 - p) * du


def make(m, n, k, dtype, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(T[dtype]).cuda()   # noqa: E731
    return r(m, k), r(2 * n, k, scale=k ** -0.5), (r(2 * n, scale=0.5) if bias else None)


def sum_error(a, b, extra=0.0):
    """Of a @ b in fp32, plus a bias."""
    k = a.shape[1]
    return (8 * math.sqrt(k) + 4) * U * (a.abs() @ b.abs() + extra)


def close(got, want, err, dtype, where=""):
    e = (got.double() - want).abs()
    bound = err * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + TINY[dtype]
    assert torch.isfinite(got.double()).all(), where
    assert (e <= bound).all(), (where, float((e / bound).max()))


def check_forward(x, w, b, act, dtype, got_h, got_z, where=""):
    n = w.shape[0] // 2
    X, W = x.double(), w.double()
    B = b.double() if b is not None else torch.zeros(2 * n, dtype=torch.float64, device="cuda")
    Z = X @ W.t() + B
    ez = sum_error(X, W.t(), B.abs())
    if got_z is not None:
        close(got_z, Z, ez, dtype, (where, "z"))
    G, V = Z[:, :n], Z[:, n:]
    a, _ = act64(G, act)
    err = 1.13 * ez[:, :n] * (V.abs() + ez[:, n:]) + a.abs() * ez[:, n:] + (10 + 4 * G.abs()) * U * (a * V).abs()
    close(got_h, a * V, err, dtype, (where, "h"))


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 3, 5), (1, 1376, 512), (7, 33, 129), (17, 64, 64), (33, 100, 96), (64, 250, 250),
          (65, 513, 7), (130, 128, 320), (200, 136, 200), (257, 264, 136), (300, 1101, 743)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward(gpu, m, n, k, dtype):
    for i, act in enumerate(ACTS):
        x, w, b = make(m, n, k, dtype, m + n + k, bias=i != 1)
        h, z = gated.gated_forward(x, w, b, act=act, save=True)
        check_forward(x, w, b, act, dtype, h, z, act)
        h2, none = gated.gated_forward(x, w, b, act=act)
        assert none is None and torch.equal(h, h2)
    if b is not None and dtype != "f32":   # a bias in 32 bits
        h, z = gated.gated_forward(x, w, b.float(), act=act, save=True)
        check_forward(x, w, b, act, dtype, h, z, "f32 bias")


# the 256 x 256 tiles: persistent (k a multiple of 128, from 256 on) and one workgroup a tile; a
# three-stage ring (k of 24 tiles or more); ragged rows and columns; more tiles than compute units
LARGE = [(2048, 2176, 256), (1999, 2168, 384), (2048, 2176, 320), (1801, 2200, 200), (130, 264, 1600), (2300, 4100, 264)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_forward_tiles(gpu, m, n, k, dtype):
    for act, bias in (("SILU", False), ("GELU", True), ("RELU", True)):
        x, w, b = make(m, n, k, dtype, m + n + k, bias=bias)
        h, z = gated.gated_forward(x, w, b, act=act, save=True)
        check_forward(x, w, b, act, dtype, h, z, act)
        if b is not None:
            b = b.float()
            h, z = gated.gated_forward(x, w, b, act=act, save=True)
            check_forward(x, w, b, act, dtype, h, z, act)
        assert torch.equal(gated.gated_forward(x, w, b, act=act)[0], h)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,d", [(2048, 4352, 256), (1999, 4344, 384), (2048, 4352, 320), (1801, 4400, 200), (130, 264, 1600),
                                   (2048, 8192, 256), (1152, 4096, 512), (1150, 4088, 200)])
def test_backward_tiles(gpu, m, n, d, dtype):
    for act in ACTS:
        x, w, _ = make(m, n, 64, dtype, m + n + d, bias=False)
        g = torch.Generator().manual_seed(d)
        h, z = gated.gated_forward(x, w, act=act, save=True)
        wd = (torch.randn(d, n, generator=g) * n ** -0.5).to(T[dtype]).cuda()
        dy = (torch.randn(m, d, generator=g) * 0.3).to(T[dtype]).cuda()
        out = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, act=act, bias_grad="f32")
        check_backward(dy, x, w, z, wd, h, act, dtype, out, act)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,d,n", [(1, 1, 1), (1, 512, 1376), (3, 33, 129), (40, 264, 1000), (130, 500, 96), (257, 128, 3000)])
def test_down(gpu, m, d, n, dtype):
    g = torch.Generator().manual_seed(m + d)
    h = torch.randn(m, n, generator=g).to(T[dtype]).cuda()
    w = (torch.randn(d, n, generator=g) * n ** -0.5).to(T[dtype]).cuda()
    close(gated.gated_down(h, w), h.double() @ w.double().t(), sum_error(h.double(), w.double().t()), dtype)


def check_backward(dy, x, w, z, wd, h, act, dtype, g, where=""):
    n = w.shape[0] // 2
    half = HALF[dtype] if dtype != "f32" else U
    D = dy.double()
    eh = torch.zeros(1, dtype=torch.float64, device="cuda")
    dh = D
    if wd is not None:
        dh = D @ wd.double()
        eh = sum_error(D, wd.double())
    G, V = z.double()[:, :n], z.double()[:, n:]
    a, da = act64(G, act)
    dz = torch.cat((dh * V * da, dh * a), 1)
    # fp32 errors of dZ: those of dH, and a few units (2 |g| through the exponential's argument)
    slack = (16 + 4 * G.abs()) * U
    lead = 1 + G.abs() * 1.2   # the slope is a sum of two terms of this size at most
    ez = torch.cat(((eh * da.abs() + slack * dh.abs() * lead) * V.abs(), eh * a.abs() + slack * (dh * a).abs()), 1)
    r = half * dz.abs() + ez   # of each term, rounded
    if g.dx is not None:
        W = w.double()
        close(g.dx, dz @ W, 8 * torch.sqrt((r * r) @ (W * W)) + sum_error(dz, W), dtype, (where, "dx"))
    if g.dw is not None:
        X = x.double()
        close(g.dw, dz.t() @ X, 8 * torch.sqrt((r * r).t() @ (X * X)) + sum_error(dz.t(), X), dtype, (where, "dw"))
    if g.dw_down is not None:
        H = h.double()
        close(g.dw_down, D.t() @ H, sum_error(D.t(), H), dtype, (where, "dw_down"))
    if g.dbias is not None:
        t = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[g.dbias.dtype]
        e = 8 * torch.sqrt((r * r).sum(0)) + (8 * math.sqrt(dz.shape[0]) + 4) * U * dz.abs().sum(0)
        close(g.dbias, dz.sum(0), e, t, (where, "dbias"))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k,d", [(1, 1, 1, 1), (1, 64, 64, 64), (2, 3, 5, 7), (7, 33, 129, 64), (77, 1000, 520, 520),
                                     (64, 250, 250, 251), (129, 136, 264, 72), (300, 264, 128, 128), (257, 1101, 743, 96)])
def test_backward(gpu, m, n, k, d, dtype):
    for i, act in enumerate(ACTS):
        x, w, b = make(m, n, k, dtype, m * 3 + n + k)
        gen = torch.Generator().manual_seed(d)
        h, z = gated.gated_forward(x, w, b, act=act, save=True)
        wd = (torch.randn(d, n, generator=gen) * n ** -0.5).to(T[dtype]).cuda()
        dy = (torch.randn(m, d, generator=gen) * 0.3).to(T[dtype]).cuda()
        g = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, act=act, bias_grad="f32" if i else dtype)
        check_backward(dy, x, w, z, wd, h, act, dtype, g, act)
        again = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, act=act, bias_grad="f32" if i else dtype)
        for p, q in zip(g, again):
            assert torch.equal(p, q)
        dh = (torch.randn(m, n, generator=gen) * 0.3).to(T[dtype]).cuda()
        g = gated.gated_backward(dh, x, w, z, act=act)
        assert g.dw_down is None and g.dbias is None
        check_backward(dh, x, w, z, None, None, act, dtype, g, act + " dh")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k,d", [(40, 100, 1, 3), (70, 1, 200, 5), (3, 64, 3, 100), (200, 7, 7, 130), (150, 130, 5, 2), (300, 3, 8, 4),
                                     (9, 4, 4, 4), (34, 8, 9, 8)])
def test_rows_of_a_few_bytes(gpu, m, n, k, d, dtype):
    """Rows of fewer than 16 bytes, of any operand, and just as many."""
    x, w, b = make(m, n, k, dtype, m + n + k + d)
    gen = torch.Generator().manual_seed(d)
    h, z = gated.gated_forward(x, w, b, act="GELU", save=True)
    check_forward(x, w, b, "GELU", dtype, h, z)
    wd = (torch.randn(d, n, generator=gen) * n ** -0.5).to(T[dtype]).cuda()
    dy = (torch.randn(m, d, generator=gen) * 0.3).to(T[dtype]).cuda()
    close(gated.gated_down(h, wd), h.double() @ wd.double().t(), sum_error(h.double(), wd.double().t()), dtype)
    g = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, act="GELU", bias_grad="f32")
    check_backward(dy, x, w, z, wd, h, "GELU", dtype, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k,d", [(40, 33, 50, 21), (150, 136, 136, 72), (300, 70, 129, 65)])
def test_nothing_past_an_operand(gpu, m, n, k, d, dtype):
    """Every operand between NaN, at offsets of its own: nothing beside them reaches a result, and
    nothing beside a result is written."""
    def inside(t, at):
        buf = torch.full((t.numel() + 96,), float("nan"), device="cuda", dtype=t.dtype)
        v = buf[at:at + t.numel()].view(t.shape)
        v.copy_(t)
        return v, buf
    x, w, b = make(m, n, k, dtype, m + n + k + d)
    wd = (torch.randn(d, n, device="cuda") * n ** -0.5).to(T[dtype])
    dy = (torch.randn(m, d, device="cuda") * 0.3).to(T[dtype])
    for at in (0, 1, 16):
        X, W, B, WD, DY = (inside(t, at)[0] for t in (x, w, b, wd, dy))
        H, hb = inside(torch.zeros(m, n, device="cuda", dtype=T[dtype]), at)
        Z, zb = inside(torch.zeros(m, 2 * n, device="cuda", dtype=T[dtype]), at)
        gated.gated_forward(X, W, B, act="SILU", out=H, z_out=Z)
        check_forward(x, w, b, "SILU", dtype, H, Z)
        assert all(buf[:at].isnan().all() and buf[at + v.numel():].isnan().all() for v, buf in ((H, hb), (Z, zb)))
        check_backward(dy, x, w, Z, wd, H, "SILU", dtype,
                       gated.gated_backward(DY, X, W, Z, w_down=WD, h=H, act="SILU", bias_grad="f32"))


def test_gradient_against_differences(gpu):
    """Loss sum(c * y) of the whole block in fp32, moved along random directions: the central
    difference of the forward pass in 64 bits against the product of gradient and direction."""
    m, n, k, d = 5, 24, 16, 12
    for act in ("SILU", "GELU"):
        x, w, b = make(m, n, k, "f32", 3)
        g = torch.Generator().manual_seed(4)
        wd = torch.randn(d, n, generator=g).cuda() * 0.3
        c = torch.randn(m, d, generator=g).cuda()

        def loss(x, w, b, wd):
            z = x @ w.t() + b
            return ((act64(z[:, :n], act)[0] * z[:, n:]) @ wd.t() * c.double()).sum()

        h, z = gated.gated_forward(x, w, b, act=act, save=True)
        grads = gated.gated_backward(c, x, w, z, w_down=wd, h=h, act=act, bias_grad="f32")
        args = [t.double() for t in (x, w, b, wd)]
        for i, got in enumerate((grads.dx, grads.dw, grads.dbias, grads.dw_down)):
            step = torch.randn(args[i].shape, generator=g).cuda().double()
            up = [a + 1e-5 * step if j == i else a for j, a in enumerate(args)]
            down = [a - 1e-5 * step if j == i else a for j, a in enumerate(args)]
            want = (loss(*up) - loss(*down)) / 2e-5
            assert abs(float((got.double() * step).sum() - want)) <= 1e-5 * float((got.double() * step).abs().sum()) + 1e-6


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_no_rows(gpu, dtype):
    x, w, b = make(0, 24, 16, dtype, 1)
    h, z = gated.gated_forward(x, w, b, save=True)
    assert h.shape == (0, 24) and z.shape == (0, 48)
    wd = torch.ones(8, 24, dtype=T[dtype], device="cuda")
    assert gated.gated_down(h, wd).shape == (0, 8)
    g = gated.gated_backward(torch.empty(0, 8, dtype=T[dtype], device="cuda"), x, w, z, w_down=wd, h=h, bias_grad="f32")
    assert g.dx.shape == (0, 16)
    for t, s in ((g.dw, (48, 16)), (g.dw_down, (8, 24)), (g.dbias, (48,))):
        assert t.shape == s and (t == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(5, 40, 48), (5, 41, 47), (150, 136, 136)])
def test_special_values(gpu, m, n, k, dtype):
    """Large and infinite sums: a row with NaN is NaN and leaves the others alone; SILU and GELU of a
    very negative gate give zero, of a very positive one the gate itself."""
    x, w, _ = make(m, n, k, dtype, 9, bias=False)
    x[1, 3] = float("nan")
    x[3] = 0
    bias = torch.zeros(2 * n, device="cuda")
    bias[0], bias[1], bias[2], bias[n:] = -1000.0, 1000.0, float("inf"), 2.0
    for act in ACTS:
        h, z = gated.gated_forward(x, w, bias, act=act, save=True)
        assert h[1, 3:].isnan().all() or act == "RELU"
        keep = [i for i in range(m) if i != 1]
        assert not h[keep][:, [0, 1] + list(range(3, n))].isnan().any()
        assert h[3, 0] == 0 and h[3, 1] == 2000 and h[3, 2] == float("inf") and (h[3, 3:] == 0).all()
        dy = torch.ones(m, n, dtype=T[dtype], device="cuda")
        g = gated.gated_backward(dy, x, w, z[:, :], act=act, bias_grad="f32", need_dx=False, need_dw=False)
        assert g.dx is None and g.dw is None and g.dbias[n + 3:].isnan().any() == (act != "RELU")


def test_large_gates_have_slopes(gpu):
    """Slopes far out: 0 and 1, without 0 times infinity."""
    g = torch.tensor([-1e4, -100.0, -20.0, 20.0, 100.0, 1e4, 3e37, -3e37], device="cuda")
    for act in ACTS:
        z = torch.cat((g, torch.ones_like(g)))[None]
        one = torch.ones(1, 8, device="cuda")
        out = gated.gated_backward(one, one[:, :1], torch.ones(16, 1, device="cuda"), z, act=act, bias_grad="f32")
        d = out.dbias[:8]
        assert (d[3:7] - 1).abs().max() < 1e-6 and d[[0, 1, 2, 7]].abs().max() < 1e-6


def test_streams_outputs_and_graphs(gpu):
    x, w, b = make(40, 264, 136, "bf16", 5)
    wd = (torch.randn(64, 264, device="cuda") * 0.1).bfloat16()
    dy = torch.randn(40, 64, device="cuda").bfloat16()
    h0, z0 = gated.gated_forward(x, w, b, save=True)
    y0 = gated.gated_down(h0, wd)
    g0 = gated.gated_backward(dy, x, w, z0, w_down=wd, h=h0, bias_grad="bf16")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h, z = torch.empty_like(h0), torch.empty_like(z0)
    gated.gated_forward(x, w, b, out=h, z_out=z, stream=side)
    y = gated.gated_down(h, wd, stream=side)
    g = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, bias_grad="bf16", stream=side)
    side.synchronize()
    for p, q in zip((h, z, y, *g), (h0, z0, y0, *g0)):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gated.gated_forward(x, w, b, out=h, z_out=z)
        y = gated.gated_down(h, wd)
        g = gated.gated_backward(dy, x, w, z, w_down=wd, h=h, bias_grad="bf16")
    for i in range(4):
        for t in (h, z, y, *g):
            t.fill_(7.0)
        x.copy_(x.roll(1, 0))
        dy.copy_(dy.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        h1, z1 = gated.gated_forward(x, w, b, save=True)
        want = (h1, z1, gated.gated_down(h1, wd), *gated.gated_backward(dy, x, w, z1, w_down=wd, h=h1, bias_grad="bf16"))
        for p, q in zip((h, z, y, *g), want):
            assert torch.equal(p, q)


def test_refusals(gpu):
    x, w, b = make(4, 8, 16, "bf16", 1)
    h, z = gated.gated_forward(x, w, b, save=True)
    wd = torch.ones(8, 8, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(4, 8, dtype=torch.bfloat16, device="cuda")
    f = gated.gated_forward
    for bad in (lambda: f(x.cpu(), w, b), lambda: f(x, w.cpu(), b), lambda: f(x.float(), w, b), lambda: f(x, w[:, :15], b),
                lambda: f(x, w[:15], b), lambda: f(x[:, ::2], w, b), lambda: f(x, w, b[:15]), lambda: f(x, w, b.half()),
                lambda: f(x, w, b, act="TANH"), lambda: f(x, w, b, out=h.float()), lambda: f(x, w, b, z_out=z[:, :15]),
                lambda: f(x.double(), w.double()), lambda: f(x[0], w), lambda: gated.gated_down(h, wd[:, :7]),
                lambda: gated.gated_down(h, wd[0]), lambda: gated.gated_backward(dy, x, w, z[:, :8]),
                lambda: gated.gated_backward(dy[:3], x, w, z), lambda: gated.gated_backward(dy, x, w, z, h=h),
                lambda: gated.gated_backward(dy, x, w, z, w_down=wd, h=h[:, :4]),
                lambda: gated.gated_backward(dy, x, w, z, bias_grad="f16"),
                lambda: gated.gated_backward(dy, x, w, z, act="NONE")):
        with pytest.raises(ValueError):
            bad()


def test_offsets_past_4_gib(gpu):
    """Rows and columns whose byte offsets pass 2^32: the last rows against the same rows alone."""
    m, n, k = 70000, 16400, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(2 * n, k, generator=g, device="cuda").bfloat16()
    h, z = gated.gated_forward(x, w, save=True)          # Z is 4.6 GB
    for r in (0, 65530, m - 130):
        h1, z1 = gated.gated_forward(x[r:r + 130].contiguous(), w, save=True)
        check_forward(x[r:r + 130], w, None, "SILU", "bf16", h[r:r + 130], z[r:r + 130])
        assert torch.equal(h1, h[r:r + 130]) and torch.equal(z1, z[r:r + 130])
    del h
    dh = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16)
    dh[-1] = 1
    gr = gated.gated_backward(dh, x, w, z, bias_grad="f32")   # only the last row counts
    one = gated.gated_backward(dh[-1:].contiguous(), x[-1:].contiguous(), w, z[-1:].contiguous(), bias_grad="f32")
    assert torch.equal(gr.dw, one.dw) and torch.equal(gr.dbias, one.dbias)
    assert (gr.dx[:-1] == 0).all()
    check_backward(dh[-1:], x[-1:], w, z[-1:], None, None, "SILU", "bf16", one._replace(dw=None, dx=gr.dx[-1:]))
