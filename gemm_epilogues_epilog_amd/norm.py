"""Residual addition with root-mean-square norm, and its gradient (C ABI:
gemm_epilog_rms_norm, gemm_epilog_rms_norm_backward in include/gemm_epilog.h).

y, s = rms_norm(x, weight, residual)                    # s = x + residual, y = norm(s) weight
q, s = rms_norm(x, weight, residual, out="mxfp8")       # y in 8 bits, the X of MXMatmul
y, q, s = rms_norm(x, weight, residual, out="both")     # y as x's type for a router, q for the experts
dx, dweight = rms_norm_backward(dy, s, weight, dresidual)
"""
from typing import Optional

import torch

from . import DTYPES, load
from .mx import _NAME, MXTensor, _allocating_on, _check, _stream, on_device


def _rows(t: torch.Tensor, name: str, shape, dtype, device):
    """Row stride of a (rows, d) operand whose rows are contiguous."""
    on_device(t, name, device)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor")
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _weight(w: torch.Tensor, d: int, dtype, device) -> int:
    on_device(w, "weight", device)
    if w.dtype not in (dtype, torch.float32) or w.numel() != d or not w.is_contiguous():
        raise ValueError(f"weight must be {d} contiguous values of x's type or f32")
    return DTYPES[_NAME[w.dtype]]


def _empty(rows: int, d: int, dtype, device, stream):
    with _allocating_on(stream):
        return torch.empty((rows, d), dtype=dtype, device=device)


def _apart(t: torch.Tensor, name: str, rows: int, d: int):
    if rows > 1 and t.stride(0) < d:
        raise ValueError(f"the rows of {name} must not overlap")


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             out: Optional[str] = None, sum_out: Optional[torch.Tensor] = None, y_out: Optional[torch.Tensor] = None,
             mx_out: Optional[MXTensor] = None, stream=None):
    """x (rows, d), f32 / f16 / bf16. out: x's type (or its name), "mxfp8", or "both".
    Returns (y, s), (q, s), or (y, q, s); s is x itself without a residual. sum_out may be x
    or residual (in place)."""
    on_device(x, "x")
    if x.dtype not in _NAME or x.dim() != 2:
        raise ValueError("x must be a (rows, d) f32, f16 or bf16 tensor")
    rows, d = x.shape
    name, dev = _NAME[x.dtype], x.device
    if out not in (None, name, "mxfp8", "both"):
        raise ValueError(f"out must be {name!r}, 'mxfp8' or 'both'")
    if d < 1:
        raise ValueError("d must be positive")
    ldx = _rows(x, "x", x.shape, x.dtype, dev)
    wdt = _weight(weight, d, x.dtype, dev)
    rp = sp = yp = cp = scp = None
    ldr = lds = ldy = d
    s = x
    if residual is not None:
        ldr = _rows(residual, "residual", x.shape, x.dtype, dev)
        rp = residual.data_ptr()
        s = sum_out if sum_out is not None else _empty(rows, d, x.dtype, dev, stream)
        lds = _rows(s, "sum_out", x.shape, x.dtype, dev)
        _apart(s, "sum_out", rows, d)
        sp = s.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out belongs to a residual")
    y = q = None
    if out != "mxfp8":
        y = y_out if y_out is not None else _empty(rows, d, x.dtype, dev, stream)
        ldy = _rows(y, "y_out", x.shape, x.dtype, dev)
        _apart(y, "y_out", rows, d)
        yp = y.data_ptr()
    elif y_out is not None:
        raise ValueError("y_out needs out to be x's type or 'both'")
    if out in ("mxfp8", "both"):
        q = mx_out
        if q is None:
            with _allocating_on(stream):
                q = MXTensor.empty(rows, d, "mxfp8", device=dev)
        if q.shape != (rows, d) or q.format != "mxfp8" or q.device != dev:
            raise ValueError(f"mx_out must be a ({rows}, {d}) mxfp8 MXTensor on {dev}")
        cp, scp = q.codes.data_ptr(), q.scales.data_ptr()
    elif mx_out is not None:
        raise ValueError("mx_out needs out to be 'mxfp8' or 'both'")
    _check(load().gemm_epilog_rms_norm(rows, d, DTYPES[name], x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), wdt, eps,
                                       sp, lds, yp, ldy, cp, scp, _stream(stream, dev)), "gemm_epilog_rms_norm")
    return (y, q, s) if out == "both" else (q, s) if out == "mxfp8" else (y, s)


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor,
                      dresidual: Optional[torch.Tensor] = None, eps: float = 1e-6, dx_out: Optional[torch.Tensor] = None,
                      stream=None):
    """(dx, dweight) from the stored s. dresidual: the gradient that reaches s past the
    norm. dx is the gradient of x and of residual alike; dx_out may be dy or dresidual."""
    on_device(s, "s")
    if s.dtype not in _NAME or s.dim() != 2 or s.shape[1] < 1:
        raise ValueError("s must be a (rows, d) f32, f16 or bf16 tensor")
    rows, d = s.shape
    dev = s.device
    lds = _rows(s, "s", s.shape, s.dtype, dev)
    lddy = _rows(dy, "dy", s.shape, s.dtype, dev)
    wdt = _weight(weight, d, s.dtype, dev)
    drp, lddr = None, d
    if dresidual is not None:
        lddr = _rows(dresidual, "dresidual", s.shape, s.dtype, dev)
        drp = dresidual.data_ptr()
    dx = dx_out if dx_out is not None else _empty(rows, d, s.dtype, dev, stream)
    lddx = _rows(dx, "dx_out", s.shape, s.dtype, dev)
    _apart(dx, "dx_out", rows, d)
    L = load()
    size = L.gemm_epilog_rms_norm_workspace_bytes(rows, d)
    with _allocating_on(stream):
        dw = torch.empty(d, dtype=weight.dtype, device=dev)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(L.gemm_epilog_rms_norm_backward(rows, d, DTYPES[_NAME[s.dtype]], dy.data_ptr(), lddy, s.data_ptr(), lds,
                                           weight.data_ptr(), wdt, eps, drp, lddr, dx.data_ptr(), lddx, dw.data_ptr(),
                                           ws.data_ptr(), size, _stream(stream, dev)), "gemm_epilog_rms_norm_backward")
    return dx, dw
