"""Microscaled operands and products over torch device tensors (C ABI: gemm_epilog_mx_*
in include/gemm_epilog.h, which states the formats and the layout).

q = mx_quantize(x, "mxfp4")            # (rows, k) or (experts, rows, k) to 4 or 8 bits
v = mx_dequantize(q, "bf16")           # the values it stands for
w = mx_pack(codes, scales, "mxfp4")    # row-major codes and scales of a checkpoint

mm = MXMatmul(n, k, x_format="mxfp8", epilog="GELU_BIAS", out="mxfp8"); mm.plan()
D = mm.execute(X, W, bias)             # act(X W^T + bias), any number of rows
With experts=E the rows of X are sorted by expert and `offsets` (E + 1, int32, on the
device) holds where each expert's rows begin.

Argument marshalling only: every step runs in the library's kernels, on the current torch
stream unless another is given.
"""
import contextlib
import ctypes
from typing import Optional

import torch

from . import (DTYPES, EPILOG, MX_FORMATS, MX_OUT, GemmEpilogError, ge_mx_plan_info_t, ge_mx_types_t, load)

# torch.cuda.current_stream(device).cuda_stream without the Stream object in between, which
# costs more than a small launch
_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream

_NAME = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
_TORCH = {v: k for k, v in _NAME.items()}


def _pad(v: int, to: int) -> int:
    return (v + to - 1) // to * to


def mx_code_bytes(fmt: str, rows: int, k: int) -> int:
    """Bytes of the codes of one (rows, k) operand, padding included."""
    return _pad(rows, 32) * _pad(k, 256) // (2 if fmt == "mxfp4" else 1)


def mx_scale_bytes(rows: int, k: int) -> int:
    return _pad(rows, 32) * _pad(k, 256) // 32


def _check(st: int, where: str) -> None:
    if st != 0:
        raise GemmEpilogError(st, where)


def _stream(stream, device) -> int:
    """The hipStream_t to launch on: the given one, or torch's current stream of the
    tensors' device."""
    if stream is None:
        return _current_stream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _allocating_on(stream):
    """Outputs and workspaces are allocated for the stream that writes them: memory that
    torch frees on another stream could still be in use there."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        return torch.cuda.stream(torch.cuda.ExternalStream(stream)) if stream else torch.cuda.stream(
            torch.cuda.default_stream())
    return torch.cuda.stream(stream)


def _format(fmt: str) -> int:
    if fmt not in MX_FORMATS:
        raise ValueError(f"unknown format {fmt!r}: one of {sorted(MX_FORMATS)}")
    return MX_FORMATS[fmt]


def on_device(t, name: str, device=None):
    """A device tensor, on `device` if given; the library launches on the device that is
    current, so that has to be the tensor's."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None:
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
    elif t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")


def _empty(shape, dtype, device, stream):
    if stream is None:   # (sizes one by one cost a third less than as a tuple)
        if isinstance(shape, int):
            return torch.empty(shape, dtype=dtype, device=device)
        return torch.empty(*shape, dtype=dtype, device=device)
    with _allocating_on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class MXTensor:
    """A (rows, k) microscaled operand, or `experts` of them one after the other: uint8
    codes and scales in the library's layout."""

    __slots__ = ("rows", "k", "format", "experts", "device", "code_ptr", "scale_ptr", "_codes", "_scales", "_buffer")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, k: int, format: str,
                 experts: Optional[int] = None):
        _format(format)
        if rows < 0 or k < 1 or (experts is not None and experts < 1):
            raise ValueError("rows must not be negative, k and experts positive")
        e = 1 if experts is None else experts
        for name, t, size in (("codes", codes, e * mx_code_bytes(format, rows, k)),
                              ("scales", scales, e * mx_scale_bytes(rows, k))):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != size:
                raise ValueError(f"{name} must be {size} contiguous uint8 values")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on the same device")
        self.rows, self.k, self.format, self.experts = rows, k, format, experts
        self._codes, self._scales, self._buffer, self.device = codes, scales, None, codes.device
        self.code_ptr, self.scale_ptr = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def empty(cls, rows: int, k: int, format: str, experts: Optional[int] = None, device="cuda", stream=None):
        """An operand to be written, codes and scales in one allocation."""
        _format(format)
        q = cls.__new__(cls)
        e = 1 if experts is None else experts
        cb = e * mx_code_bytes(format, rows, k)
        q.rows, q.k, q.format, q.experts = rows, k, format, experts
        q._buffer = b = _empty(cb + e * mx_scale_bytes(rows, k), torch.uint8, device, stream)
        q._codes = q._scales = None
        q.device = b.device
        q.code_ptr = b.data_ptr()
        q.scale_ptr = q.code_ptr + cb
        return q

    def _view(self, lo: int, hi: int):
        v = self._buffer[lo:hi]
        return v if self.experts is None else v.view(self.experts, -1)

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = self._view(0, self.scale_ptr - self.code_ptr)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._view(self.scale_ptr - self.code_ptr, self._buffer.numel())
        return self._scales

    @property
    def shape(self):
        return (self.rows, self.k) if self.experts is None else (self.experts, self.rows, self.k)


def _parts(q: MXTensor):
    """(codes pointer, scales pointer) of each expert."""
    c, s = q.code_ptr, q.scale_ptr
    if q.experts is None:
        return ((c, s),)
    cb, sb = mx_code_bytes(q.format, q.rows, q.k), mx_scale_bytes(q.rows, q.k)
    return [(c + e * cb, s + e * sb) for e in range(q.experts)]


def mx_quantize(x: torch.Tensor, format: str, out: Optional[MXTensor] = None, stream=None) -> MXTensor:
    """x (rows, k) or (experts, rows, k), f32 / f16 / bf16, any strides; the blocks run
    along k."""
    on_device(x, "x")
    fmt = _format(format)
    if x.dtype not in _NAME or x.dim() not in (2, 3):
        raise ValueError("x must be a 2- or 3-dimensional f32, f16 or bf16 tensor")
    rows, k = x.shape[-2:]
    experts = x.shape[0] if x.dim() == 3 else None
    if k < 1 or experts == 0:
        raise ValueError("k and experts must be positive")
    if out is None:
        out = MXTensor.empty(rows, k, format, experts, x.device, stream)
    elif out.shape != tuple(x.shape) or out.format != format or out.device != x.device:
        raise ValueError("out does not match x")
    L, s, dt = load(), _stream(stream, x.device), DTYPES[_NAME[x.dtype]]
    rs, cs = x.stride(-2), x.stride(-1)
    if k == 1:
        cs = 1
    step = x.stride(0) * x.element_size() if experts else 0
    for e, (c, sc) in enumerate(_parts(out)):
        _check(L.gemm_epilog_mx_quantize(rows, k, dt, x.data_ptr() + e * step, rs, cs, fmt, c, sc, s),
               "gemm_epilog_mx_quantize")
    return out


def mx_dequantize(q: MXTensor, dtype: str = "bf16", out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values q stands for, (rows, k) or (experts, rows, k)."""
    if not isinstance(q, MXTensor) or q.device.type != "cuda" or q.device.index != torch._C._cuda_getDevice():
        raise ValueError("q must be an MXTensor on the current device")
    if dtype not in _TORCH:
        raise ValueError(f"unknown type {dtype!r}")
    if out is None:
        out = _empty(q.shape, _TORCH[dtype], q.device, stream)
    else:
        on_device(out, "out", q.device)
        if tuple(out.shape) != q.shape or out.dtype != _TORCH[dtype] or (q.k > 1 and out.stride(-1) != 1) or \
                (q.rows > 1 and out.stride(-2) < q.k) or \
                (q.experts is not None and q.experts > 1 and out.stride(0) < (q.rows - 1) * out.stride(-2) + q.k):
            raise ValueError(f"out must be a {q.shape} {dtype} tensor whose rows are contiguous and apart")
    L, s, fmt = load(), _stream(stream, q.device), MX_FORMATS[q.format]
    if q.experts is None:
        _check(L.gemm_epilog_mx_dequantize(q.rows, q.k, fmt, q.code_ptr, q.scale_ptr, DTYPES[dtype], out.data_ptr(),
                                           out.stride(0) if q.rows > 1 else q.k, s), "gemm_epilog_mx_dequantize")
        return out
    step = out.stride(0) * out.element_size()
    ld = out.stride(-2) if q.rows > 1 else q.k
    for e, (c, sc) in enumerate(_parts(q)):
        _check(L.gemm_epilog_mx_dequantize(q.rows, q.k, fmt, c, sc, DTYPES[dtype], out.data_ptr() + e * step, ld, s),
               "gemm_epilog_mx_dequantize")
    return out


def mx_pack(codes: torch.Tensor, scales: torch.Tensor, format: str, k: Optional[int] = None, stream=None) -> MXTensor:
    """Row-major codes ([experts,] rows, k / 2 or k bytes) and scales ([experts,] rows, k / 32
    bytes) in the library's layout. k defaults to what the codes hold (give it where the
    last byte of an odd MXFP4 row holds one value)."""
    on_device(codes, "codes")
    on_device(scales, "scales", codes.device)
    fmt = _format(format)
    for name, t in (("codes", codes), ("scales", scales)):
        if t.dtype != torch.uint8 or t.dim() not in (2, 3) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2- or 3-dimensional uint8 tensor")
    rows, width = codes.shape[-2:]
    if k is None:
        k = width * 2 if format == "mxfp4" else width
    if k < 1 or width != ((k + 1) // 2 if format == "mxfp4" else k) or \
            tuple(scales.shape) != (*codes.shape[:-1], (k + 31) // 32):
        raise ValueError("codes and scales do not fit k")
    q = MXTensor.empty(rows, k, format, codes.shape[0] if codes.dim() == 3 else None, codes.device, stream)
    L, s = load(), _stream(stream, codes.device)
    for e, (c, sc) in enumerate(_parts(q)):
        _check(L.gemm_epilog_mx_pack(rows, k, fmt, codes.data_ptr() + e * rows * width,
                                     scales.data_ptr() + e * rows * ((k + 31) // 32), c, sc, s), "gemm_epilog_mx_pack")
    return q


class MXMatmul:
    """D = act(X W^T + bias), X microscaled (m, k), W MXFP4 (n, k): plan once per (n, k),
    execute for any m and any weights.

    mm = MXMatmul(n, k, "mxfp8", "GELU_BIAS", "bf16"); mm.plan(); D = mm.execute(X, W, bias); mm.free()
    or `with MXMatmul(...) as mm:`. epilog: NONE, BIAS, RELU_BIAS, GELU_BIAS. out: f32, f16,
    bf16, or mxfp8 (execute then returns an MXTensor, the next product's X). vec_dtype: the
    bias's type, by default out's (f32 for mxfp8). experts=E: grouped products.
    """

    def __init__(self, n: int, k: int, x_format: str = "mxfp8", epilog: str = "NONE", out: str = "bf16",
                 vec_dtype: Optional[str] = None, experts: Optional[int] = None):
        _format(x_format)
        if epilog not in EPILOG:
            raise ValueError(f"unknown epilogue {epilog!r}")
        if out not in MX_OUT:
            raise ValueError(f"unknown output {out!r}: one of {sorted(MX_OUT)}")
        self.n, self.k, self.x_format, self.epilog, self.out = int(n), int(k), x_format, epilog, out
        self.vec_dtype = vec_dtype or ("f32" if out == "mxfp8" else out)
        if self.vec_dtype not in DTYPES:
            raise ValueError(f"unknown type {vec_dtype!r}")
        if experts is not None and experts < 1:
            raise ValueError("experts must be positive")
        self.experts = experts
        self.handle = None
        self.device = None

    def _types(self):
        return ge_mx_types_t(MX_FORMATS[self.x_format], MX_OUT[self.out], DTYPES[self.vec_dtype])

    def plan(self):
        if self.handle is None:
            h = ctypes.c_void_p()
            _check(load().gemm_epilog_mx_plan(self.n, self.k, self.experts or 0, self._types(), EPILOG[self.epilog],
                                              ctypes.byref(h)), "gemm_epilog_mx_plan")
            self.handle = h.value
            self.device = torch.device("cuda", torch.cuda.current_device())
        return self

    def plan_info(self, m: int, compute_units: int = 256) -> dict:
        """What an execute of m rows launches (computed on the host, no device needed)."""
        info = ge_mx_plan_info_t()
        _check(load().gemm_epilog_mx_plan_info(self.n, self.k, self.experts or 0, self._types(), EPILOG[self.epilog],
                                               int(m), int(compute_units), ctypes.byref(info)),
               "gemm_epilog_mx_plan_info")
        return {name: getattr(info, name) for name, _ in ge_mx_plan_info_t._fields_}

    def execute(self, X: MXTensor, W: MXTensor, bias: Optional[torch.Tensor] = None,
                offsets: Optional[torch.Tensor] = None, out=None, stream=None):
        if self.handle is None:
            self.plan()
        n, k, experts, dev = self.n, self.k, self.experts, self.device
        if not isinstance(X, MXTensor) or X.format != self.x_format or X.k != k or X.experts is not None:
            raise ValueError(f"X must be a (rows, {k}) {self.x_format} MXTensor")
        if not isinstance(W, MXTensor) or W.format != "mxfp4" or W.k != k or W.rows != n or W.experts != experts:
            raise ValueError(f"W must be a {(n, k) if experts is None else (experts, n, k)} mxfp4 MXTensor")
        if X.device != dev or W.device != dev:
            raise ValueError(f"X and W must be on the plan's device {dev}")
        if dev.index != torch._C._cuda_getDevice():   # (where the library launches)
            raise ValueError(f"the plan's device {dev} is not the current device")
        bp = op = sp = None
        if self.epilog != "NONE":
            if bias is None:
                raise ValueError(f"{self.epilog} needs a bias")
            if bias.dtype != _TORCH[self.vec_dtype] or bias.device != dev or not bias.is_contiguous() or \
                    bias.numel() != n * (experts or 1):
                raise ValueError(f"bias must be {n * (experts or 1)} contiguous {self.vec_dtype} values on {dev}")
            bp = bias.data_ptr()
        if experts is not None:
            if offsets is None or offsets.dtype != torch.int32 or offsets.device != dev or \
                    not offsets.is_contiguous() or offsets.numel() != experts + 1:
                raise ValueError(f"offsets must be {experts + 1} contiguous int32 values on {dev}")
            op = offsets.data_ptr()
        elif offsets is not None:
            raise ValueError("offsets belong to a plan with experts")
        m = X.rows
        if self.out == "mxfp8":
            if out is None:
                out = MXTensor.empty(m, n, "mxfp8", None, dev, stream)
            elif not isinstance(out, MXTensor) or out.shape != (m, n) or out.format != "mxfp8" or out.device != dev:
                raise ValueError(f"out must be a ({m}, {n}) mxfp8 MXTensor on {dev}")
            dp, sp = out.code_ptr, out.scale_ptr
        else:
            t = _TORCH[self.out]
            if out is None:
                out = _empty((m, n), t, dev, stream)
            elif out.dtype != t or out.device != dev or not out.is_contiguous() or tuple(out.shape) != (m, n):
                raise ValueError(f"out must be a contiguous ({m}, {n}) {self.out} tensor on {dev}")
            dp = out.data_ptr()
        _check(load().gemm_epilog_mx_execute(self.handle, m, X.code_ptr, X.scale_ptr, W.code_ptr, W.scale_ptr, bp, op,
                                             dp, sp, _stream(stream, dev)), "gemm_epilog_mx_execute")
        return out

    def free(self):
        if self.handle is not None:
            load().gemm_epilog_mx_free(self.handle)
            self.handle = None

    def __enter__(self):
        return self.plan()

    def __exit__(self, *exc):
        self.free()
        return False

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
