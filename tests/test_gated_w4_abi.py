"""Arguments that the C ABI of the gated block and of the 4-bit weights refuses, on the host before
any HIP call (no GPU): status codes, and the sizes that callers allocate by."""
import ctypes

import pytest

import gemm_epilogues_epilog_amd as ge

F32, F16, BF16 = 0, 1, 2
P = 1 << 20   # a pointer that nothing follows: every check comes before any use


@pytest.fixture(scope="module")
def lib():
    return ge.load()


def forward(lib, m=4, n=8, k=8, dt=BF16, act=0, x=P, w=P, bias=None, vec=BF16, h=P, z=None):
    return lib.gemm_epilog_gated_forward(m, n, k, dt, act, x, w, bias, vec, h, z, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(m=1 << 31), 1), (dict(n=0), 1), (dict(n=(1 << 20) + 1), 1), (dict(k=0), 1),
    (dict(k=(1 << 20) + 1), 1), (dict(dt=3), 1), (dict(dt=-1), 1), (dict(act=3), 1), (dict(act=-1), 1), (dict(vec=7), 1),
    (dict(vec=F16), 2), (dict(dt=F32, vec=BF16), 2), (dict(m=(1 << 31) - 1, n=1 << 20), 2),
    (dict(x=None), 3), (dict(w=None), 3), (dict(h=None), 3),
    (dict(x=P + 1), 4), (dict(w=P + 1), 4), (dict(h=P + 1), 4), (dict(z=P + 1), 4), (dict(bias=P + 1), 4),
    (dict(bias=P + 2, vec=F32), 4), (dict(dt=F32, vec=F32, x=P + 2), 4),
])
def test_forward_refuses(lib, kw, status):
    assert forward(lib, **kw) == status


@pytest.mark.parametrize("args,status", [
    ((-1, 8, 8, BF16, P, P, P), 1), ((4, 0, 8, BF16, P, P, P), 1), ((4, 8, 1 << 21, BF16, P, P, P), 1), ((4, 8, 8, 9, P, P, P), 1),
    ((4, 8, 8, BF16, None, P, P), 3), ((4, 8, 8, BF16, P, None, P), 3), ((4, 8, 8, BF16, P, P, None), 3),
    ((4, 8, 8, BF16, P + 1, P, P), 4), ((4, 8, 8, F32, P, P, P + 2), 4), (((1 << 31) - 1, 1 << 20, 8, BF16, P, P, P), 2),
])
def test_down_refuses(lib, args, status):
    assert lib.gemm_epilog_gated_down(*args, None) == status


def backward(lib, m=4, n=8, k=8, d=8, dt=BF16, act=0, dy=P, x=P, w=P, z=P, h=P, wd=P, dx=P, dw=P, dwd=P, db=P, vec=BF16,
             ws=P, size=1 << 40):
    return lib.gemm_epilog_gated_backward(m, n, k, d, dt, act, dy, x, w, z, h, wd, dx, dw, dwd, db, vec, ws, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(d=0), 1), (dict(d=(1 << 20) + 1), 1), (dict(dt=5), 1),
    (dict(act=9), 1), (dict(vec=-1), 1), (dict(vec=F16), 2), (dict(m=(1 << 24) + 1), 2),
    (dict(wd=None, dwd=None, d=16), 1), (dict(wd=None), 3), (dict(dy=None), 3), (dict(z=None), 3), (dict(x=None), 3),
    (dict(w=None), 3), (dict(h=None), 3), (dict(ws=None), 3), (dict(ws=P + 128), 4), (dict(dy=P + 1), 4), (dict(dx=P + 1), 4),
    (dict(dwd=P + 1), 4), (dict(db=P + 2, vec=F32), 4), (dict(size=100), 7),
])
def test_backward_refuses(lib, kw, status):
    assert backward(lib, **kw) == status


def test_backward_workspace(lib):
    size = lib.gemm_epilog_gated_workspace_bytes
    assert size(0, 8, 8, 8, BF16) == 0 and size(4, 0, 8, 8, BF16) == 0 and size((1 << 24) + 1, 8, 8, 8, BF16) == 0
    assert size(4, 8, 8, 8, 7) == 0
    for m, n, k, d, dt in ((1, 1, 1, 1, F32), (2048, 11008, 4096, 4096, BF16), (77, 1000, 520, 520, F16)):
        need = size(m, n, k, d, dt)
        assert need >= m * 2 * n * (4 if dt == F32 else 2)   # dZ
        assert backward(lib, m=m, n=n, k=k, d=d, dt=dt, vec=dt, size=need - 1) == 7


@pytest.mark.parametrize("rows,k,group,halves", [(0, 8, 32, 1), (8, 0, 32, 1), (8, 8, 0, 1), (8, 8, 16, 1), (8, 8, 96, 1),
                                                 (8, 8, 200, 1), (8, 8, 32, 0), (8, 8, 32, 3), (7, 8, 32, 2),
                                                 ((1 << 20) + 1, 8, 32, 1), (8, (1 << 20) + 1, 32, 1)])
def test_w4_sizes_outside_the_set(lib, rows, k, group, halves):
    assert lib.gemm_epilog_w4_scale_count(rows, k, group, halves) == 0
    assert lib.gemm_epilog_w4_quantize(rows, k, BF16, P, k, group, halves, 0, BF16, P, P, P, None) == 1
    assert lib.gemm_epilog_w4_pack(rows, k, group, halves, P, P, None, P, P, P, None) == 1
    assert lib.gemm_epilog_w4_dequantize(rows, k, group, halves, BF16, P, P, P, BF16, P, 1 << 21, None) == 1


def test_w4_sizes(lib):
    assert lib.gemm_epilog_w4_code_bytes(16, 128, 1) == 1024 and lib.gemm_epilog_w4_code_bytes(17, 129, 1) == 4096
    assert lib.gemm_epilog_w4_code_bytes(34, 128, 2) == 4096   # two halves of 17 rows
    assert lib.gemm_epilog_w4_scale_count(17, 129, 64, 1) == 32 * 3
    assert lib.gemm_epilog_w4_scale_count(1 << 20, 1 << 20, 32, 1) == (1 << 20) * (1 << 15)


def quantize(lib, src_dt=BF16, src=P, ld=64, dt=BF16, c=P, s=P, z=P):
    return lib.gemm_epilog_w4_quantize(8, 64, src_dt, src, ld, 32, 1, 0, dt, c, s, z, None)


@pytest.mark.parametrize("kw,status", [(dict(src_dt=4), 1), (dict(dt=3), 1), (dict(dt=F32), 2), (dict(ld=-1), 1), (dict(src=None), 3),
                                       (dict(c=None), 3), (dict(s=None), 3), (dict(z=None), 3), (dict(c=P + 8), 4),
                                       (dict(z=P + 1), 4), (dict(src=P + 1), 4), (dict(src=P + 2, src_dt=F32), 4)])
def test_quantize_refuses(lib, kw, status):
    assert quantize(lib, **kw) == status


def test_pack_and_dequantize_refuse(lib):
    pack = lambda sc=P, ss=P: lib.gemm_epilog_w4_pack(8, 64, 32, 1, sc, ss, None, P, P, P, None)   # noqa: E731
    assert pack(sc=None) == 3 and pack(ss=None) == 3 and pack(ss=P + 1) == 4
    de = lambda dt=BF16, o=BF16, d=P, ld=64: lib.gemm_epilog_w4_dequantize(8, 64, 32, 1, dt, P, P, P, o, d, ld, None)   # noqa: E731
    assert de(dt=F32) == 2 and de(o=9) == 1 and de(ld=63) == 1 and de(d=None) == 3 and de(d=P + 1) == 4


def matmul(lib, m=4, n=8, k=64, group=32, dt=BF16, out=BF16, ep=5, x=P, c=P, s=P, z=P, bias=P, vec=BF16, D=P):
    return lib.gemm_epilog_w4_matmul(m, n, k, group, dt, out, ep, x, c, s, z, bias, vec, D, None)


def gated(lib, m=4, n=8, k=64, group=32, dt=BF16, act=0, x=P, c=P, s=P, z=P, bias=P, vec=BF16, D=P):
    return lib.gemm_epilog_w4_gated(m, n, k, group, dt, act, x, c, s, z, bias, vec, D, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(m=1 << 31), 1), (dict(n=0), 1), (dict(n=(1 << 20) + 1), 1), (dict(k=0), 1), (dict(group=33), 1),
    (dict(dt=4), 1), (dict(dt=F32, vec=F32), 2), (dict(vec=F16), 2), (dict(x=None), 3), (dict(c=None), 3), (dict(s=None), 3),
    (dict(z=None), 3), (dict(D=None), 3), (dict(x=P + 1), 4), (dict(D=P + 1), 4), (dict(s=P + 2), 4), (dict(bias=P + 1), 4),
])
def test_products_refuse(lib, kw, status):
    assert matmul(lib, **kw) == status
    assert gated(lib, **kw) == status


def test_products_refuse_more(lib):
    assert matmul(lib, ep=3) == 2 and matmul(lib, ep=99) == 2 and matmul(lib, bias=None) == 3
    assert matmul(lib, out=F16) == 2 and matmul(lib, out=8) == 1 and matmul(lib, out=F32, D=P + 2) == 4
    assert gated(lib, act=3) == 1 and gated(lib, n=1 << 62) == 1


def test_exports_match_argument_counts():
    """Every new entry point has a signature, so that ctypes converts 64-bit sizes and pointers."""
    L = ge.load()
    for name in ge.EXPORTS:
        if "_gated_" in name or "_w4_" in name:
            assert getattr(L, name).argtypes and getattr(L, name).restype in (ctypes.c_int, ctypes.c_size_t)
