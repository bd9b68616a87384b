"""The 64-bit reference of the microscaled operators against hand-worked values, and the
host side of the operators: sizes, refusals and the plan's rules. No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import gemm_epilogues_epilog_amd as ge
from gemm_epilogues_epilog_amd import mx, norm
from tests import mx_reference as ref


def test_elements():
    assert ref.E4M3[-1] == 448 and ref.E4M3[8] == 2.0 ** -6 and ref.E4M3[1] == 2.0 ** -9
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3)


@pytest.mark.parametrize("fmt,x,codes,scale", [
    # largest 4: exponent 2, scale 1
    ("mxfp4", [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.5], [6, 0, 2, 2, 4, 4, 6, 9], 127),
    # largest 7.9: scale 1, saturates at 6; 5 is halfway between 4 and 6: even code 6 (4)
    ("mxfp4", [7.9, 5, -5.01], [7, 6, 15], 127),
    # largest 1: scale 1/4
    ("mxfp4", [1, 0.125], [6, 1], 125),
    ("mxfp8", [256, 1, 0.0009765625], [120, 56, 0], 127),
    ("mxfp8", [511, -464], [126, 254], 127),
    ("mxfp4", [0, 0], [0, 0], 0),
    ("mxfp4", [np.inf, 1], [0, 0], 255),
    ("mxfp8", [np.nan, 1], [0, 0], 255),
])
def test_quantize_by_hand(fmt, x, codes, scale):
    c, s = ref.quantize(np.array([x]), fmt)
    assert c[0].tolist() == codes and s[0].tolist() == [scale]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("R,K", [(1, 1), (33, 257), (64, 512), (5, 40)])
def test_layout_round_trip(fmt, R, K):
    rng = np.random.default_rng(R * K)
    c = rng.integers(0, 16 if fmt == "mxfp4" else 256, (R, K)).astype(np.uint8)
    s = rng.integers(0, 256, (R, -(-K // 32))).astype(np.uint8)
    p, ps = ref.pack(c, s, fmt)
    assert p.size == mx.mx_code_bytes(fmt, R, K) == ge.load().gemm_epilog_mx_code_bytes(ge.MX_FORMATS[fmt], R, K)
    assert ps.size == mx.mx_scale_bytes(R, K) == ge.load().gemm_epilog_mx_scale_bytes(R, K)
    c2, s2 = ref.unpack(p, ps, R, K, fmt)
    assert np.array_equal(c, c2) and np.array_equal(s, s2)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    s, w, dy = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7))
    f = lambda s, w: float(np.sum(ref.rms_norm(s, w, 1e-3) * dy))   # noqa: E731
    dx, dw = ref.rms_norm_backward(dy, s, w, 1e-3)
    h = 1e-6
    for i in range(3):
        for j in range(7):
            d = np.zeros_like(s)
            d[i, j] = h
            # central differences: error h^2 f''' / 6 and 2^-53 |f| / h, far below 1e-8
            assert abs((f(s + d, w) - f(s - d, w)) / (2 * h) - dx[i, j]) < 1e-8
    for j in range(7):
        d = np.zeros_like(w)
        d[j] = h
        assert abs((f(s, w + d) - f(s, w - d)) / (2 * h) - dw[j]) < 1e-8


# ---- host rules -----------------------------------------------------------------------
INVALID, UNSUPPORTED, NULL, MISALIGNED, SCRATCH = 1, 2, 3, 4, 7
P = 4096   # stands for a device pointer; the checks never follow it


@pytest.mark.parametrize("args,status", [
    ((-1, 8, 1, P, 8, 1, 0, P, P), INVALID),
    ((8, 0, 1, P, 8, 1, 0, P, P), INVALID),
    ((8, (1 << 20) + 1, 1, P, 8, 1, 0, P, P), INVALID),
    ((1 << 31, 8, 1, P, 8, 1, 0, P, P), INVALID),
    (((1 << 31) - 1, 1 << 20, 1, P, 8, 1, 0, P, P), INVALID),   # more tiles than a launch holds
    ((8, 8, 3, P, 8, 1, 0, P, P), INVALID),                     # type
    ((8, 8, 1, P, 8, 1, 2, P, P), INVALID),                     # format
    ((8, 8, 1, P, -8, 1, 0, P, P), INVALID),
    ((8, 8, 1, P, 8, -1, 0, P, P), INVALID),
    ((8, 8, 1, None, 8, 1, 0, P, P), NULL),
    ((8, 8, 1, P, 8, 1, 0, None, P), NULL),
    ((8, 8, 1, P, 8, 1, 0, P, None), NULL),
    ((8, 8, 1, P + 1, 8, 1, 0, P, P), MISALIGNED),
    ((8, 8, 1, P, 8, 1, 0, P + 8, P), MISALIGNED),
    ((8, 8, 1, P, 8, 1, 0, P, P + 4), MISALIGNED),
    ((0, 8, 1, None, 8, 1, 0, None, None), 0),                  # nothing to do
])
def test_quantize_refusals(args, status):
    assert ge.load().gemm_epilog_mx_quantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((8, 8, 0, P, P, 1, P, 7), INVALID),        # rows overlap
    ((8, 8, 2, P, P, 1, P, 8), INVALID),
    ((8, 8, 0, P, P, 4, P, 8), INVALID),
    ((8, 8, 0, None, P, 1, P, 8), NULL),
    ((8, 8, 0, P, P, 1, None, 8), NULL),
    ((8, 8, 0, P + 4, P, 1, P, 8), MISALIGNED),
    ((8, 8, 0, P, P, 0, P + 2, 8), MISALIGNED),
    ((0, 8, 0, None, None, 1, None, 8), 0),
])
def test_dequantize_refusals(args, status):
    assert ge.load().gemm_epilog_mx_dequantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((8, 8, 3, P, P, P, P), INVALID),
    ((8, 0, 0, P, P, P, P), INVALID),
    ((8, 8, 0, None, P, P, P), NULL),
    ((8, 8, 0, P, P, P, None), NULL),
    ((8, 8, 0, P + 1, P + 1, P + 8, P), MISALIGNED),   # sources may lie anywhere
    ((0, 8, 0, None, None, None, None), 0),
])
def test_pack_refusals(args, status):
    assert ge.load().gemm_epilog_mx_pack(*args, None) == status


def types(x=1, d=2, vec=2):
    return ge.ge_mx_types_t(x, d, vec)


@pytest.mark.parametrize("args,status", [
    ((0, 8, 0, types(), 1), INVALID),
    ((8, 0, 0, types(), 1), INVALID),
    (((1 << 20) + 1, 8, 0, types(), 1), INVALID),
    ((8, 8, -1, types(), 1), INVALID),
    ((8, 8, 4097, types(), 1), INVALID),
    ((8, 8, 0, types(x=2), 1), INVALID),
    ((8, 8, 0, types(d=4), 1), INVALID),
    ((8, 8, 0, types(vec=3), 1), INVALID),
    ((8, 8, 0, types(d=2, vec=1), 1), UNSUPPORTED),     # bias neither D's type nor fp32
    ((8, 8, 0, types(), 3), UNSUPPORTED),               # RELU_AUX_BIAS
    ((8, 8, 0, types(), 4), UNSUPPORTED),
    ((8, 8, 0, types(), 100), UNSUPPORTED),
    ((8, 8, 0, types(), 9), INVALID),
])
def test_plan_refusals(args, status):
    L = ge.load()
    h = ctypes.c_void_p()
    assert L.gemm_epilog_mx_plan(*args, ctypes.byref(h)) == status and h.value is None
    info = ge.ge_mx_plan_info_t()
    assert L.gemm_epilog_mx_plan_info(*args, 8, 256, ctypes.byref(info)) == status


def test_plan_null_and_info_refusals():
    L = ge.load()
    assert L.gemm_epilog_mx_plan(8, 8, 0, types(), 1, None) == NULL
    assert L.gemm_epilog_mx_plan_info(8, 8, 0, types(), 1, 8, 256, None) == NULL
    info = ge.ge_mx_plan_info_t()
    for m, cus in ((-1, 256), (1 << 31, 256), (8, 0), (8, 4097)):
        assert L.gemm_epilog_mx_plan_info(8, 8, 0, types(), 1, m, cus, ctypes.byref(info)) == INVALID
    assert L.gemm_epilog_mx_execute(None, 8, P, P, P, P, P, None, P, None, None) == NULL
    assert L.gemm_epilog_mx_free(None) == 0


@pytest.mark.parametrize("experts", [None, 1, 7, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (4096, 11008), (11008, 4096), (100000, 300)])
@pytest.mark.parametrize("m", [0, 1, 16, 17, 64, 65, 100, 1000, 8192, 100000])
def test_plan_info_covers_the_output(m, n, k, experts):
    for out in ("bf16", "mxfp8"):
        i = mx.MXMatmul(n, k, out=out, experts=experts).plan_info(m)
        cols = ref.pad(n, 256) if out == "mxfp8" else n
        cover = -(-cols // i["tile_n"])
        if m == 0:
            assert i["workgroups"] == 0
            continue
        assert 1 <= i["splits"] <= max(1, ref.pad(k, 256) // 128)
        if i["stages"]:
            assert 1 <= i["workgroups"] <= i["tiles"] * i["splits"]
        else:   # workgroups per expert and columns: one, or several that share its rows
            assert i["workgroups"] % i["tiles"] == 0
        if experts is None:
            rows = -(-m // i["tile_m"]) if i["stages"] else 1
            assert i["tiles"] == rows * cover
            # every part of every split tile has its workgroup and its slot of the workspace
            if i["splits"] > 1:
                assert i["workgroups"] == i["tiles"] * i["splits"]
                assert i["workgroups"] * i["tile_m"] * i["tile_n"] * 4 <= i["workspace_bytes"]
        elif i["stages"]:
            # any split of m rows over the experts fits: the worst spreads a row group each
            assert i["tiles"] >= cover * max(-(-m // i["tile_m"]), min(m, experts))
        else:
            assert i["tiles"] == cover * experts


def test_tested_products_reach_every_kernel():
    """The shapes that the device tests multiply, and their result types, take every
    configuration with every kind of operand on 256 compute units."""
    from tests import test_mx_gpu as gpu
    single = {(256, 256, False), (128, 256, False), (128, 128, False), (128, 64, False), (64, 64, False),
              (64, 64, True), (16, 32, False), (16, 16, False)}
    grouped = {(t, n, False) for t, n, _ in single}
    for fmt in ("mxfp8", "mxfp4"):
        for out in ("f32", "bf16"):
            seen = set()
            for m, n, k in gpu.MNK + gpu.MNK_TILES:
                i = mx.MXMatmul(n, k, fmt, "NONE", out).plan_info(m, compute_units=256)
                seen.add((i["tile_m"], i["tile_n"], i["splits"] > 1))
            assert single <= seen, (fmt, out, sorted(single - seen))
            cases = [(c, n, k) for c in gpu.COUNTS for n, k in ((96, 300), (300, 512))] + gpu.COUNTS_TILES
            seen = set()
            for counts, n, k in cases:
                i = mx.MXMatmul(n, k, fmt, "NONE", out, experts=len(counts)).plan_info(sum(counts), compute_units=256)
                seen.add((i["tile_m"], i["tile_n"], i["splits"] > 1))
            assert grouped <= seen, (fmt, out, sorted(grouped - seen))


@pytest.mark.parametrize("args,status", [
    # rows, d, dt, x, ldx, res, ldr, w, wdt, eps, sum, lds, y, ldy, codes, scales
    ((-1, 8, 1, P, 8, None, 0, P, 1, 1e-6, None, 0, P, 8, None, None), INVALID),
    ((4, 0, 1, P, 8, None, 0, P, 1, 1e-6, None, 0, P, 8, None, None), INVALID),
    ((4, 8, 3, P, 8, None, 0, P, 1, 1e-6, None, 0, P, 8, None, None), INVALID),
    ((4, 8, 1, P, 8, None, 0, P, 1, -1.0, None, 0, P, 8, None, None), INVALID),
    ((4, 8, 1, P, 8, None, 0, P, 1, float("nan"), None, 0, P, 8, None, None), INVALID),
    ((4, 8, 1, P, 8, None, 0, P, 1, float("inf"), None, 0, P, 8, None, None), INVALID),
    ((4, 8, 1, P, -1, None, 0, P, 1, 1e-6, None, 0, P, 8, None, None), INVALID),
    ((4, 8, 1, P, 8, None, 0, P, 1, 1e-6, None, 0, P, 7, None, None), INVALID),      # rows of y overlap
    ((4, 8, 1, P, 8, P, 8, P, 1, 1e-6, P, 7, P, 8, None, None), INVALID),
    ((4, 32769, 1, P, 40000, None, 0, P, 1, 1e-6, None, 0, P, 40000, None, None), UNSUPPORTED),
    ((4, 8, 1, P, 8, None, 0, P, 2, 1e-6, None, 0, P, 8, None, None), UNSUPPORTED),  # weight bf16 for f16 rows
    ((4, 8, 1, None, 8, None, 0, P, 1, 1e-6, None, 0, P, 8, None, None), NULL),
    ((4, 8, 1, P, 8, None, 0, None, 1, 1e-6, None, 0, P, 8, None, None), NULL),
    ((4, 8, 1, P, 8, None, 0, P, 1, 1e-6, None, 0, None, 8, None, None), NULL),      # no output
    ((4, 8, 1, P, 8, P, 8, P, 1, 1e-6, None, 0, P, 8, None, None), NULL),            # residual without sum
    ((4, 8, 1, P, 8, None, 0, P, 1, 1e-6, None, 0, P, 8, P, None), NULL),            # codes without scales
    ((4, 8, 1, P + 1, 8, None, 0, P, 1, 1e-6, None, 0, P, 8, None, None), MISALIGNED),
    ((4, 8, 1, P, 8, None, 0, P, 1, 1e-6, None, 0, None, 8, P + 2, P), MISALIGNED),
    ((0, 8, 1, None, 8, None, 0, None, 1, 1e-6, None, 0, None, 8, None, None), 0),
])
def test_norm_refusals(args, status):
    assert ge.load().gemm_epilog_rms_norm(*args, None) == status


@pytest.mark.parametrize("args,status", [
    # rows, d, dt, dy, lddy, s, lds, w, wdt, eps, dres, lddr, dx, lddx, dw, ws, ws_bytes
    ((4, 8, 1, P, 8, P, 8, P, 1, 1e-6, None, 0, P, 7, P, P, 1 << 20), INVALID),
    ((4, 8, 1, P, -8, P, 8, P, 1, 1e-6, None, 0, P, 8, P, P, 1 << 20), INVALID),
    ((4, 40000, 1, P, 40000, P, 40000, P, 1, 1e-6, None, 0, P, 40000, P, P, 1 << 30), UNSUPPORTED),
    ((4, 8, 1, None, 8, P, 8, P, 1, 1e-6, None, 0, P, 8, P, P, 1 << 20), NULL),
    ((4, 8, 1, P, 8, P, 8, P, 1, 1e-6, None, 0, P, 8, None, P, 1 << 20), NULL),
    ((4, 8, 1, P, 8, P, 8, P, 1, 1e-6, None, 0, P, 8, P, None, 1 << 20), NULL),
    ((4, 8, 1, P, 8, P, 8, P, 1, 1e-6, None, 0, P, 8, P, P, 16), SCRATCH),
    ((4, 8, 0, P, 8, P, 8, P, 0, 1e-6, None, 0, P, 8, P + 2, P, 1 << 20), MISALIGNED),
])
def test_norm_backward_refusals(args, status):
    assert ge.load().gemm_epilog_rms_norm_backward(*args, None) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mx_quantize(x, "mxfp4")
    with pytest.raises(ValueError, match="device tensor"):
        norm.rms_norm(x, torch.ones(64))
    with pytest.raises(ValueError, match="device tensor"):
        norm.rms_norm_backward(x, x, torch.ones(64))
    with pytest.raises(ValueError, match="unknown format"):
        mx.MXTensor(x, x, 4, 64, "fp4")
    with pytest.raises(ValueError, match="contiguous uint8"):
        mx.MXTensor(torch.zeros(8, dtype=torch.uint8), torch.zeros(8, dtype=torch.uint8), 4, 64, "mxfp4")
    for kw in (dict(x_format="f16"), dict(epilog="SWISH"), dict(out="u8"), dict(vec_dtype="f64"), dict(experts=0)):
        with pytest.raises(ValueError):
            mx.MXMatmul(64, 64, **kw)


def test_accuracy_shapes_reach_every_configuration_and_split():
    """The shapes of the accuracy tests take every tile, whole and with k shared between
    workgroups, on 256 compute units, by format of X and type of result."""
    from tests import test_mx_accuracy_gpu as gpu
    whole = {(16, 16, False), (16, 32, False), (64, 64, False), (128, 64, False), (128, 128, False), (128, 256, False),
             (256, 256, False)}
    for fmt in ("mxfp8", "mxfp4"):
        split = {(64, 64, True), (128, 128, True)} | ({(128, 64, True)} if fmt == "mxfp8" else set())
        for out in ("f32", "bf16", "f16", "mxfp8"):
            seen = {gpu.takes(mx.MXMatmul(n, k, fmt, "NONE", out), m)
                    for m, n, k in (gpu.EVERY_8 if out == "mxfp8" else gpu.EVERY)}
            need = (whole | split) - ({(16, 16, False)} if out == "mxfp8" else set())   # 8 bits take whole blocks of 32
            assert need <= seen, (fmt, out, sorted(need - seen))
