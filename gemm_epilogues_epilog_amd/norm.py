"""Residual addition with root-mean-square norm, and its gradient (C ABI:
gemm_epilog_rms_norm, gemm_epilog_rms_norm_backward in include/gemm_epilog.h).

y, s = rms_norm(x, weight, residual)                    # s = x + residual, y = norm(s) weight
q, s = rms_norm(x, weight, residual, out="mxfp8")       # y in 8 bits, the X of MXMatmul
y, q, s = rms_norm(x, weight, residual, out="both")     # y in x's type as well, for what is not quantised
dx, dweight = rms_norm_backward(dy, s, weight, dresidual)
"""
from typing import Optional

import torch

from . import DTYPES, load
from .mx import _NAME, MXTensor, _check, _empty, _stream, on_device


def _rows(t: torch.Tensor, name: str, rows: int, d: int, dtype, device) -> int:
    """Row stride of a (rows, d) operand whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype or t.shape != (rows, d):
        raise ValueError(f"{name} must be a ({rows}, {d}) {dtype} tensor on {device}")
    if t.is_contiguous():
        return d
    if d > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if rows > 1 else d


def _like(x: torch.Tensor, stream) -> torch.Tensor:
    """A contiguous tensor of x's shape and type."""
    if stream is None and x.is_contiguous():
        return torch.empty_like(x)
    return _empty(x.shape, x.dtype, x.device, stream)


def _out_rows(t: torch.Tensor, name: str, rows: int, d: int, dtype, device) -> int:
    ld = _rows(t, name, rows, d, dtype, device)
    if ld < d:
        raise ValueError(f"the rows of {name} must not overlap")
    return ld


def _weight(w: torch.Tensor, d: int, dtype, device) -> int:
    if not isinstance(w, torch.Tensor) or w.device != device or (w.dtype != dtype and w.dtype != torch.float32) or \
            w.numel() != d or not w.is_contiguous():
        raise ValueError(f"weight must be {d} contiguous values of x's type or f32 on {device}")
    return DTYPES[_NAME[w.dtype]]


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
    t = x.dtype
    ldx = _rows(x, "x", rows, d, t, dev)
    wdt = _weight(weight, d, t, dev)
    rp = sp = yp = cp = scp = None
    ldr = lds = ldy = d
    s = x
    if residual is not None:
        ldr = _rows(residual, "residual", rows, d, t, dev)
        rp = residual.data_ptr()
        if sum_out is None:
            s = _like(x, stream)
        else:
            s = sum_out
            lds = _out_rows(s, "sum_out", rows, d, t, dev)
        sp = s.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out belongs to a residual")
    y = q = None
    if out != "mxfp8":
        if y_out is None:
            y = _like(x, stream)
        else:
            y = y_out
            ldy = _out_rows(y, "y_out", rows, d, t, dev)
        yp = y.data_ptr()
    elif y_out is not None:
        raise ValueError("y_out needs out to be x's type or 'both'")
    if out == "mxfp8" or out == "both":
        q = mx_out
        if q is None:
            q = MXTensor.empty(rows, d, "mxfp8", None, dev, stream)
        elif q.shape != (rows, d) or q.format != "mxfp8" or q.device != dev:
            raise ValueError(f"mx_out must be a ({rows}, {d}) mxfp8 MXTensor on {dev}")
        cp, scp = q.code_ptr, q.scale_ptr
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
    dev, t = s.device, s.dtype
    lds = _rows(s, "s", rows, d, t, dev)
    lddy = _rows(dy, "dy", rows, d, t, dev)
    wdt = _weight(weight, d, t, dev)
    drp, lddr, lddx = None, d, d
    if dresidual is not None:
        lddr = _rows(dresidual, "dresidual", rows, d, t, dev)
        drp = dresidual.data_ptr()
    if dx_out is None:
        dx = _like(s, stream)
    else:
        dx = dx_out
        lddx = _out_rows(dx, "dx_out", rows, d, t, dev)
    L = load()
    size = L.gemm_epilog_rms_norm_workspace_bytes(rows, d)
    dw = torch.empty_like(weight) if stream is None else _empty(weight.shape, weight.dtype, dev, stream)
    ws = _empty(size, torch.uint8, dev, stream)
    _check(L.gemm_epilog_rms_norm_backward(rows, d, DTYPES[_NAME[t]], dy.data_ptr(), lddy, s.data_ptr(), lds,
                                           weight.data_ptr(), wdt, eps, drp, lddr, dx.data_ptr(), lddx, dw.data_ptr(),
                                           ws.data_ptr(), size, _stream(stream, dev)), "gemm_epilog_rms_norm_backward")
    return dx, dw
