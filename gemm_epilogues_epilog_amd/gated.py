"""The gated feed-forward block and its gradients (C ABI: gemm_epilog_gated_* in
include/gemm_epilog.h, which states the formulas).

h, z = gated_forward(x, w, bias, act="SILU", save=True)   # h = act(G) * U, z = [G | U] = x w^T + bias
y = gated_down(h, w_down)                                  # h w_down^T
g = gated_backward(dy, x, w, z, w_down=w_down, h=h)        # g.dx, g.dw, g.dw_down, g.dbias

Tokens along the rows; w (2 n, k) holds the gate's rows, then the up projection's. f32, f16
and bf16, any sizes; argument marshalling only.
"""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import DTYPES, GATES, load
from .mx import _NAME, _TORCH, _check, _empty, _stream, on_device


class GatedGrads(NamedTuple):
    """Gradients; None where they were not asked for."""
    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]
    dw_down: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


def _dense(t, name: str, shape, dtype, device) -> int:
    """The pointer of a contiguous tensor of this shape and type."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype or t.shape != shape or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")
    return t.data_ptr()


def _out(t, name: str, shape, dtype, device, stream, *others):
    """A new result, or the caller's, which has to lie apart from the operands."""
    if t is None:
        return _empty(shape, dtype, device, stream)
    at = _dense(t, name, shape, dtype, device)
    for o in others:
        if o is not None and at < o.data_ptr() + o.numel() * o.element_size() and \
                o.data_ptr() < at + t.numel() * t.element_size():
            raise ValueError(f"{name} must not overlap an operand or another result")
    return t


def _rows2(x, name: str):
    on_device(x, name)
    if x.dtype not in _NAME or x.dim() != 2 or x.shape[1] < 1 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-dimensional f32, f16 or bf16 tensor")
    return x.shape


def _gate(act: str) -> int:
    if act not in GATES:
        raise ValueError(f"unknown activation {act!r}: one of {sorted(GATES)}")
    return GATES[act]


def _halves(w, k: int, dtype, device) -> int:
    """n of a (2 n, k) weight."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] < 2 or w.shape[0] % 2:
        raise ValueError(f"w must be a (2 n, {k}) tensor: the gate's rows, then the up projection's")
    _dense(w, "w", (w.shape[0], k), dtype, device)
    return w.shape[0] // 2


def _bias(bias, n: int, dtype, device):
    """(pointer, type) of n bias values of dtype or f32."""
    if bias is None:
        return None, DTYPES["f32"]
    if not isinstance(bias, torch.Tensor) or bias.device != device or bias.dtype not in (dtype, torch.float32) or \
            bias.numel() != n or not bias.is_contiguous():
        raise ValueError(f"bias must be {n} contiguous values of {dtype} or f32 on {device}")
    return bias.data_ptr(), DTYPES[_NAME[bias.dtype]]


def gated_forward(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "SILU",
                  save: bool = False, out: Optional[torch.Tensor] = None, z_out: Optional[torch.Tensor] = None,
                  stream=None):
    """(h, z): h (m, n); z (m, 2 n) for the backward pass with save=True (or z_out), else None."""
    m, k = _rows2(x, "x")
    dev, t = x.device, x.dtype
    a = _gate(act)
    n = _halves(w, k, t, dev)
    bp, vec = _bias(bias, 2 * n, t, dev)
    h = _out(out, "out", (m, n), t, dev, stream, x, w, bias)
    z = _out(z_out, "z_out", (m, 2 * n), t, dev, stream, x, w, bias, h) if save or z_out is not None else None
    _check(load().gemm_epilog_gated_forward(m, n, k, DTYPES[_NAME[t]], a, x.data_ptr(), w.data_ptr(), bp, vec,
                                            h.data_ptr(), None if z is None else z.data_ptr(), _stream(stream, dev)),
           "gemm_epilog_gated_forward")
    return h, z


def gated_down(h: torch.Tensor, w_down: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y (m, d) = h w_down^T, h (m, n), w_down (d, n)."""
    m, n = _rows2(h, "h")
    dev, t = h.device, h.dtype
    if not isinstance(w_down, torch.Tensor) or w_down.dim() != 2 or w_down.shape[0] < 1:
        raise ValueError(f"w_down must be a (d, {n}) tensor")
    d = w_down.shape[0]
    _dense(w_down, "w_down", (d, n), t, dev)
    y = _out(out, "out", (m, d), t, dev, stream, h, w_down)
    _check(load().gemm_epilog_gated_down(m, d, n, DTYPES[_NAME[t]], h.data_ptr(), w_down.data_ptr(), y.data_ptr(),
                                         _stream(stream, dev)), "gemm_epilog_gated_down")
    return y


def gated_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, z: torch.Tensor,
                   w_down: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None, act: str = "SILU",
                   bias_grad: Optional[str] = None, need_dx: bool = True, need_dw: bool = True,
                   stream=None) -> GatedGrads:
    """From dy (m, d), the gradient of y = h w_down^T; without w_down, dy (m, n) is the gradient
    of h. dw_down comes back where w_down and h are given, dbias where bias_grad names its type
    (x's or "f32"). A tile of dx is NaN where a wait ran out (gated_lost_waits)."""
    m, k = _rows2(x, "x")
    dev, t = x.device, x.dtype
    a = _gate(act)
    n = _halves(w, k, t, dev)
    zp = _dense(z, "z", (m, 2 * n), t, dev)
    d, wp, hp = n, None, None
    if w_down is not None:
        if not isinstance(w_down, torch.Tensor) or w_down.dim() != 2 or w_down.shape[0] < 1:
            raise ValueError(f"w_down must be a (d, {n}) tensor")
        d = w_down.shape[0]
        wp = _dense(w_down, "w_down", (d, n), t, dev)
    if h is not None:
        if w_down is None:
            raise ValueError("h serves the gradient of w_down")
        hp = _dense(h, "h", (m, n), t, dev)
    dyp = _dense(dy, "dy", (m, d), t, dev)
    if bias_grad is not None and (bias_grad not in _TORCH or _TORCH[bias_grad] not in (t, torch.float32)):
        raise ValueError(f"bias_grad must be {_NAME[t]!r} or 'f32'")
    dt = DTYPES[_NAME[t]]
    dx = _empty((m, k), t, dev, stream) if need_dx else None
    dw = _empty((2 * n, k), t, dev, stream) if need_dw else None
    dwd = _empty((d, n), t, dev, stream) if h is not None else None
    db = _empty(2 * n, _TORCH[bias_grad], dev, stream) if bias_grad is not None else None
    L = load()
    size = L.gemm_epilog_gated_workspace_bytes(m, n, k, d, dt)
    ws = _empty(size, torch.uint8, dev, stream)
    ptr = lambda v: None if v is None else v.data_ptr()   # noqa: E731
    _check(L.gemm_epilog_gated_backward(m, n, k, d, dt, a, dyp, x.data_ptr(), w.data_ptr(), zp, hp, wp, ptr(dx), ptr(dw),
                                        ptr(dwd), ptr(db), DTYPES[bias_grad or "f32"], ws.data_ptr(), size,
                                        _stream(stream, dev)), "gemm_epilog_gated_backward")
    return GatedGrads(dx, dw, dwd, db)


def gated_lost_waits(stream=None) -> int:
    """Synchronise the stream and return how many waits of gated_backward ran out on the current
    device since the last call (their tiles of dx hold NaN)."""
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    n = ctypes.c_uint32(0)
    _check(load().gemm_epilog_gated_lost_waits(stream, ctypes.byref(n)), "gemm_epilog_gated_lost_waits")
    return int(n.value)
