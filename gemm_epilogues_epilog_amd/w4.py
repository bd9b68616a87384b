"""4-bit weights with group scales and their products (C ABI: gemm_epilog_w4_* in
include/gemm_epilog.h, which states the formulas and the layout).

W = w4_quantize(w, group=128)                         # (rows, k) f32 / f16 / bf16, once per weight
W = w4_pack(codes, scales, zeros, group=128)          # or from a checkpoint's row-major arrays
v = w4_dequantize(W)                                  # the values it stands for
D = w4_matmul(x, W, bias, epilog="GELU_BIAS")         # act(x W^T + bias), any number of tokens
h = w4_gated(x, W, bias, act="SILU")                  # act(G) * U of a weight made with gated=True

Argument marshalling only: every step runs in the library's kernels, on the current torch
stream unless another is given.
"""
from typing import Optional

import torch

from . import DTYPES, EPILOG, load
from .gated import _bias, _gate, _out, _rows2
from .mx import _NAME, _TORCH, _check, _empty, _stream, on_device

_HALF = (torch.float16, torch.bfloat16)
_MAX_DIM = 1 << 20   # of a half's rows, of k and of a group
_EPILOGS = ("NONE", "BIAS", "RELU_BIAS", "GELU_BIAS")


def _group_ok(group: int) -> int:
    group = int(group)
    if group not in (32, 64) and (group < 128 or group % 128):
        raise ValueError("group must be 32, 64 or a multiple of 128")
    return group


class W4Tensor:
    """A (rows, k) weight in 4 bits: uint8 codes, 16-bit scales and uint8 zeros in the library's
    layout. gated: rows is 2 n, the gate's rows and then the up projection's."""

    __slots__ = ("rows", "k", "group", "gated", "dtype", "device", "ptrs", "_parts", "_buf")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, rows: int, k: int,
                 group: int = 128, gated: bool = False):
        self.rows, self.k, self.group, self.gated = int(rows), int(k), _group_ok(group), bool(gated)
        cb, sc = self.sizes(self.rows, self.k, self.group, self.gated)
        for name, t, types, size in (("codes", codes, (torch.uint8,), cb), ("scales", scales, _HALF, sc),
                                     ("zeros", zeros, (torch.uint8,), sc)):
            if t.dtype not in types or not t.is_contiguous() or t.numel() != size or t.device != codes.device:
                raise ValueError(f"{name} must be {size} contiguous {types[0]} values on {codes.device}")
        self._parts, self._buf = (codes, scales, zeros), codes
        self.ptrs = codes.data_ptr(), scales.data_ptr(), zeros.data_ptr()
        self.dtype, self.device = scales.dtype, codes.device

    @staticmethod
    def sizes(rows: int, k: int, group: int, gated: bool):
        """(code bytes, scales) of a weight, padding included."""
        halves = 2 if gated else 1
        if not (1 <= rows <= _MAX_DIM * halves and rows % halves == 0 and 1 <= k <= _MAX_DIM and group <= _MAX_DIM):
            raise ValueError(f"a weight of {rows} x {k} with groups of {group} is not supported")
        rg = halves * -(-(rows // halves) // 16)
        return rg * -(-k // 128) * 1024, rg * -(-k // group) * 16

    @classmethod
    def empty(cls, rows: int, k: int, group: int = 128, gated: bool = False, dtype=torch.bfloat16, device="cuda",
              stream=None):
        """A weight to be written: codes, scales and zeros in one allocation."""
        group = _group_ok(group)
        if dtype not in _HALF:
            raise ValueError("the scales are f16 or bf16")
        cb, sc = cls.sizes(rows, k, group, gated)
        q = cls.__new__(cls)
        q.rows, q.k, q.group, q.gated, q.dtype = int(rows), int(k), group, bool(gated), dtype
        q._buf, q._parts = _empty(cb + 3 * sc, torch.uint8, device, stream), None
        at = q._buf.data_ptr()
        q.device, q.ptrs = q._buf.device, (at, at + cb, at + cb + 2 * sc)
        return q

    def _views(self):
        if self._parts is None:
            cb, sc = self.sizes(self.rows, self.k, self.group, self.gated)
            self._parts = self._buf[:cb], self._buf[cb:cb + 2 * sc].view(self.dtype), self._buf[cb + 2 * sc:]
        return self._parts

    @property
    def codes(self) -> torch.Tensor:
        return self._views()[0]

    @property
    def scales(self) -> torch.Tensor:
        return self._views()[1]

    @property
    def zeros(self) -> torch.Tensor:
        return self._views()[2]

    @property
    def shape(self):
        return (self.rows, self.k)


def _weight(q, device=None) -> W4Tensor:
    if not isinstance(q, W4Tensor):
        raise ValueError("the weight must be a W4Tensor")
    on_device(q._buf, "the weight", device)
    return q


def _target(out, rows, k, group, gated, dtype, device, stream) -> W4Tensor:
    if out is None:
        return W4Tensor.empty(rows, k, group, gated, dtype, device, stream)
    if not isinstance(out, W4Tensor) or out.shape != (rows, k) or out.group != group or out.gated != gated or \
            out.dtype != dtype or out.device != device:
        raise ValueError("out does not match")
    return out


def w4_quantize(w: torch.Tensor, group: int = 128, symmetric: bool = False, gated: bool = False,
                dtype: Optional[str] = None, out: Optional[W4Tensor] = None, stream=None) -> W4Tensor:
    """w (rows, k), contiguous rows. dtype: the scales' ("f16" or "bf16"), by default w's."""
    on_device(w, "w")
    if w.dtype not in _NAME or w.dim() != 2 or (w.shape[1] > 1 and w.stride(1) != 1):
        raise ValueError("w must be a 2-dimensional f32, f16 or bf16 tensor with contiguous rows")
    if dtype is None and w.dtype == torch.float32:
        raise ValueError("an f32 weight needs dtype='f16' or 'bf16'")
    t = w.dtype if dtype is None else _TORCH.get(dtype)
    if t not in _HALF:
        raise ValueError("the scales are f16 or bf16")
    rows, k = w.shape
    group = _group_ok(group)
    q = _target(out, rows, k, group, bool(gated), t, w.device, stream)
    _check(load().gemm_epilog_w4_quantize(rows, k, DTYPES[_NAME[w.dtype]], w.data_ptr(), w.stride(0) if rows > 1 else k,
                                          group, 2 if gated else 1, int(bool(symmetric)), DTYPES[_NAME[t]], *q.ptrs,
                                          _stream(stream, w.device)), "gemm_epilog_w4_quantize")
    return q


def w4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None, group: int = 128,
            k: Optional[int] = None, gated: bool = False, out: Optional[W4Tensor] = None, stream=None) -> W4Tensor:
    """Row-major codes (rows, ceil(k / 2)) uint8, scales (rows, groups) f16 or bf16, zeros (rows,
    groups) uint8 or None for 8. k defaults to twice the codes' width."""
    on_device(codes, "codes")
    group = _group_ok(group)
    if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous 2-dimensional uint8 tensor")
    rows, width = codes.shape
    k = 2 * width if k is None else int(k)
    if k < 1 or width != (k + 1) // 2:
        raise ValueError("codes do not fit k")
    groups = -(-k // group)
    for name, t, types in (("scales", scales, _HALF), ("zeros", zeros, (torch.uint8,))):
        if t is None and name == "zeros":
            continue
        on_device(t, name, codes.device)
        if t.dtype not in types or tuple(t.shape) != (rows, groups) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous ({rows}, {groups}) tensor of {types}")
    q = _target(out, rows, k, group, bool(gated), scales.dtype, codes.device, stream)
    _check(load().gemm_epilog_w4_pack(rows, k, group, 2 if gated else 1, codes.data_ptr(), scales.data_ptr(),
                                      None if zeros is None else zeros.data_ptr(), *q.ptrs,
                                      _stream(stream, codes.device)), "gemm_epilog_w4_pack")
    return q


def w4_dequantize(q: W4Tensor, dtype: Optional[str] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(q - z) s, (rows, k), in the scales' type unless dtype names another."""
    _weight(q)
    t = q.dtype if dtype is None else _TORCH.get(dtype)
    if t is None:
        raise ValueError(f"unknown type {dtype!r}")
    v = _out(out, "out", (q.rows, q.k), t, q.device, stream, q._buf)
    _check(load().gemm_epilog_w4_dequantize(q.rows, q.k, q.group, 2 if q.gated else 1, DTYPES[_NAME[q.dtype]], *q.ptrs,
                                            DTYPES[_NAME[t]], v.data_ptr(), q.k, _stream(stream, q.device)),
           "gemm_epilog_w4_dequantize")
    return v


def _operands(x, W, gated: bool):
    m, k = _rows2(x, "x")
    _weight(W, x.device)
    if W.gated != gated:
        raise ValueError("w4_gated takes a weight made with gated=True, w4_matmul one without")
    if W.k != k or W.dtype != x.dtype:
        raise ValueError(f"x must be (m, {W.k}) {W.dtype}, got {tuple(x.shape)} {x.dtype}")
    return m, k


def w4_matmul(x: torch.Tensor, W: W4Tensor, bias: Optional[torch.Tensor] = None, epilog: str = "NONE",
              out_dtype: Optional[str] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(x W^T + bias), (m, rows), in x's type or "f32". epilog: NONE, BIAS, RELU_BIAS, GELU_BIAS."""
    m, k = _operands(x, W, False)
    if epilog not in _EPILOGS:
        raise ValueError(f"epilog must be one of {_EPILOGS}")
    if (bias is None) != (epilog == "NONE"):
        raise ValueError(f"{epilog} {'needs a' if bias is None else 'takes no'} bias")
    n, dev, name = W.rows, x.device, _NAME[x.dtype]
    if out_dtype not in (None, name, "f32"):
        raise ValueError(f"out_dtype must be {name!r} or 'f32'")
    bp, vec = _bias(bias, n, x.dtype, dev)
    o = out_dtype or name
    D = _out(out, "out", (m, n), _TORCH[o], dev, stream, x, W._buf, bias)
    _check(load().gemm_epilog_w4_matmul(m, n, k, W.group, DTYPES[name], DTYPES[o], EPILOG[epilog], x.data_ptr(),
                                        *W.ptrs, bp, vec, D.data_ptr(), _stream(stream, dev)), "gemm_epilog_w4_matmul")
    return D


def w4_gated(x: torch.Tensor, W: W4Tensor, bias: Optional[torch.Tensor] = None, act: str = "SILU",
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(G) * U with [G | U] = x W^T + bias, (m, rows / 2)."""
    m, k = _operands(x, W, True)
    a, n, dev = _gate(act), W.rows // 2, x.device
    bp, vec = _bias(bias, 2 * n, x.dtype, dev)
    h = _out(out, "out", (m, n), x.dtype, dev, stream, x, W._buf, bias)
    _check(load().gemm_epilog_w4_gated(m, n, k, W.group, DTYPES[_NAME[x.dtype]], a, x.data_ptr(), *W.ptrs, bp, vec,
                                       h.data_ptr(), _stream(stream, dev)), "gemm_epilog_w4_gated")
    return h
