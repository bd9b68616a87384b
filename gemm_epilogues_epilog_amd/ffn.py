"""Feed-forward blocks through the library's norm, quantisation and products: serving with
microscaled weights, dense or by expert, and the gated block, in training and in serving with
integer 4-bit weights.

Tokens lie along the rows: x and residual (tokens, d), one bias per column. Sums and norms are
fp32. In the microscaled blocks weights are quantised to MXFP4 once, activations to MXFP8 on
the way.

MXFeedForward, per call:
  q, s = rms_norm(x, weight, residual)    s = x + residual, q its norm in MXFP8
  h    = gelu(q W1^T + b1)                (tokens, hidden), MXFP8
  y    = h W2^T + b2                      (tokens, d)
MXExperts, per call:
  y, s = rms_norm(x, weight, residual)
  top_k experts of each token by the router's logits y R^T, their weights a softmax of them
  the tokens' rows sorted by expert, one MXFP8 operand
  h    = gelu(X W1[e]^T + b1[e]), z = h W2[e]^T + b2[e]   the experts' rows in one launch each
  out  = sum over a token's experts of weight times its row of z
GatedFeedForward (fp32, fp16, bf16) and W4FeedForward (fp16, bf16), per call:
  t, s = rms_norm(x, weight, residual)
  h    = act(t Wg^T + bg) * (t Wu^T + bu)          (tokens, hidden), W1 = [Wg; Wu]
  y    = h W2^T                                     (tokens, d)
and GatedFeedForward.backward all gradients of that from those of y and s.
The caller adds the result to s in the next block's norm, as its residual.
"""
from typing import Dict, NamedTuple, Optional, Tuple

import torch

from . import GATES, Matmul
from .gated import gated_backward, gated_down, gated_forward
from .mx import _NAME, MXMatmul, MXTensor, mx_quantize
from .norm import rms_norm, rms_norm_backward
from .w4 import W4Tensor, w4_gated, w4_matmul, w4_quantize

_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def _weight4(w, shape) -> MXTensor:
    """A weight in MXFP4: as given, or quantised once."""
    if isinstance(w, MXTensor):
        if w.shape != shape or w.format != "mxfp4":
            raise ValueError(f"the weight must be a {shape} mxfp4 MXTensor, got {w.shape} {w.format}")
        return w
    if tuple(w.shape) != shape:
        raise ValueError(f"the weight must be {shape}, got {tuple(w.shape)}")
    return mx_quantize(w, "mxfp4")


def _bias(b, shape, dtype) -> torch.Tensor:
    if tuple(b.shape) != shape or b.dtype != dtype:
        raise ValueError(f"the bias must be {shape} of {dtype}, got {tuple(b.shape)} of {b.dtype}")
    return b.contiguous()


class MXFeedForward:
    """Plans for one (d, hidden) and any number of tokens. W1 (hidden, d) and W2 (d, hidden)
    are tensors or MXFP4 MXTensors, the biases and the norm's weight of type dtype. Calls
    enqueue on the current torch stream; one stream at a time, as for the plans."""

    def __init__(self, norm_weight, W1, b1, W2, b2, d: int, hidden: int, dtype: str = "bf16", eps: float = 1e-6):
        if dtype not in _TORCH:
            raise ValueError("the block runs in fp16 or bf16")
        t = _TORCH[dtype]
        self.norm_weight, self.eps, self.dtype = norm_weight, eps, t
        self.W1, self.W2 = _weight4(W1, (hidden, d)), _weight4(W2, (d, hidden))
        self.b1, self.b2 = _bias(b1, (hidden,), t), _bias(b2, (d,), t)
        self.up = MXMatmul(hidden, d, "mxfp8", "GELU_BIAS", "mxfp8", vec_dtype=dtype).plan()
        self.down = MXMatmul(d, hidden, "mxfp8", "BIAS", dtype).plan()

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(y, s)."""
        q, s = rms_norm(x, self.norm_weight, residual, self.eps, out="mxfp8")
        return self.down.execute(self.up.execute(q, self.W1, self.b1), self.W2, self.b2), s

    def free(self):
        self.up.free()
        self.down.free()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()
        return False


class MXExperts:
    """Plans for one (tokens, d, hidden, experts). W1 (experts, hidden, d), W2 (experts, d,
    hidden), b1 (experts, hidden), b2 (experts, d), router (experts, d); d and experts
    multiples of 8 (the router's product). The rows an expert gets are known on the
    device only, so nothing waits for the host."""

    def __init__(self, norm_weight, router, W1, b1, W2, b2, tokens: int, d: int, hidden: int, experts: int,
                 top_k: int = 2, dtype: str = "bf16", eps: float = 1e-6):
        if dtype not in _TORCH:
            raise ValueError("the block runs in fp16 or bf16")
        if tokens < 1 or not 1 <= top_k <= experts:
            raise ValueError("tokens must be positive and top_k between 1 and experts")
        for name, v in (("d", d), ("experts", experts)):
            if v < 8 or v % 8:
                raise ValueError(f"{name} = {v} must be a positive multiple of 8")
        t = _TORCH[dtype]
        if tuple(router.shape) != (experts, d) or router.dtype != t:
            raise ValueError(f"router must be ({experts}, {d}) of {t}")
        self.tokens, self.d, self.experts, self.top_k, self.dtype = tokens, d, experts, top_k, t
        self.norm_weight, self.eps, self.router = norm_weight, eps, router.contiguous()
        self.W1, self.W2 = _weight4(W1, (experts, hidden, d)), _weight4(W2, (experts, d, hidden))
        self.b1, self.b2 = _bias(b1, (experts, hidden), t), _bias(b2, (experts, d), t)
        self.logits = Matmul(tokens, experts, d, dtype, "NONE", trans_b=True).plan()
        self.up = MXMatmul(hidden, d, "mxfp8", "GELU_BIAS", "mxfp8", vec_dtype=dtype, experts=experts).plan()
        self.down = MXMatmul(d, hidden, "mxfp8", "BIAS", dtype, experts=experts).plan()
        self._edges = torch.arange(experts + 1, device=router.device)

    def route(self, y: torch.Tensor):
        """(weights (tokens, top_k) fp32, order, offsets): the routed rows sorted by expert
        are rows order // top_k of y; expert e has rows offsets[e] .. offsets[e + 1] - 1."""
        best, chosen = torch.topk(self.logits.execute(y, self.router).float(), self.top_k, dim=1)
        by_expert, order = torch.sort(chosen.flatten(), stable=True)
        return torch.softmax(best, 1), order, torch.searchsorted(by_expert, self._edges).int()

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(out, s)."""
        if tuple(x.shape) != (self.tokens, self.d):
            raise ValueError(f"x must be ({self.tokens}, {self.d}), got {tuple(x.shape)}")
        y, s = rms_norm(x, self.norm_weight, residual, self.eps)
        weights, order, offsets = self.route(y)
        X = mx_quantize(y[order // self.top_k], "mxfp8")
        z = self.down.execute(self.up.execute(X, self.W1, self.b1, offsets), self.W2, self.b2, offsets)
        rows = torch.empty_like(z)
        rows[order] = z   # back in the tokens' order, top_k rows each
        out = (rows.view(self.tokens, self.top_k, self.d).float() * weights[..., None]).sum(1)
        return out.to(self.dtype), s

    def free(self):
        for p in (self.logits, self.up, self.down):
            p.free()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()
        return False


class Saved(NamedTuple):
    """What GatedFeedForward.forward leaves for its backward."""
    t: torch.Tensor   # the norm's result
    s: torch.Tensor   # x + residual
    z: torch.Tensor   # [G | U]
    h: torch.Tensor


def _matching(name: str, w, shape, dtype) -> torch.Tensor:
    if tuple(w.shape) != shape or w.dtype != dtype:
        raise ValueError(f"{name} must be {shape} of {dtype}, got {tuple(w.shape)} of {w.dtype}")
    return w


def _act(act: str) -> str:
    if act not in GATES:
        raise ValueError(f"unknown activation {act!r}: one of {sorted(GATES)}")
    return act


class GatedFeedForward:
    """The gated block in training: W1 (2 hidden, d), the gate's rows and then the up projection's,
    W2 (d, hidden), b1 (2 hidden) or None; weights are read where they are, so an optimizer may
    update them in place between calls. Any number of tokens; work goes to the current torch
    stream."""

    def __init__(self, norm_weight, W1, W2, b1=None, act: str = "SILU", eps: float = 1e-6):
        if W1.dim() != 2 or W1.shape[0] < 2 or W1.shape[0] % 2 or W1.dtype not in _NAME:
            raise ValueError("W1 must be a (2 hidden, d) f32, f16 or bf16 tensor")
        self.hidden, self.d, self.dtype = W1.shape[0] // 2, W1.shape[1], W1.dtype
        self.W1, self.W2 = W1, _matching("W2", W2, (self.d, self.hidden), W1.dtype)
        self.b1 = None if b1 is None else _matching("b1", b1, (2 * self.hidden,), b1.dtype)
        if b1 is not None and b1.dtype not in (W1.dtype, torch.float32):
            raise ValueError(f"b1 must be of {W1.dtype} or f32")
        self.norm_weight, self.act, self.eps = norm_weight, _act(act), eps

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, Saved]:
        """(y, s, saved)."""
        t, s = rms_norm(x, self.norm_weight, residual, self.eps)
        h, z = gated_forward(t, self.W1, self.b1, self.act, save=True)
        return gated_down(h, self.W2), s, Saved(t, s, z, h)

    def backward(self, dy: torch.Tensor, saved: Saved, ds: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
        """Gradients: "dx" (of x and of residual alike), "dnorm", "dW1", "dW2", and "db1" with a bias.
        ds: the gradient that reaches s past the block."""
        g = gated_backward(dy, saved.t, self.W1, saved.z, w_down=self.W2, h=saved.h, act=self.act,
                           bias_grad=None if self.b1 is None else _NAME[self.b1.dtype])
        dx, dnorm = rms_norm_backward(g.dx, saved.s, self.norm_weight, ds, self.eps)
        out = {"dx": dx, "dnorm": dnorm, "dW1": g.dw, "dW2": g.dw_down}
        if g.dbias is not None:
            out["db1"] = g.dbias
        return out


class W4FeedForward:
    """The gated block in serving, its weights in 4 bits with group scales: W1 (2 hidden, d) and W2
    (d, hidden) as tensors, quantised here once, or as W4Tensors (W1's made with gated=True). b1
    (2 hidden) and b2 (d) or None, of the weights' type. Any number of tokens."""

    def __init__(self, norm_weight, W1, W2, b1=None, b2=None, act: str = "SILU", group: int = 128, eps: float = 1e-6):
        W1 = W1 if isinstance(W1, W4Tensor) else w4_quantize(W1, group, gated=True)
        W2 = W2 if isinstance(W2, W4Tensor) else w4_quantize(W2, group)
        self.hidden, self.d, self.dtype = W1.rows // 2, W1.k, W1.dtype
        if not W1.gated or W2.gated or W2.shape != (self.d, self.hidden) or W2.dtype != self.dtype:
            raise ValueError(f"W1 must be a gated (2 hidden, d) weight and W2 ({self.d}, {self.hidden}) of {self.dtype}")
        self.W1, self.W2 = W1, W2
        self.b1 = None if b1 is None else _bias(b1, (2 * self.hidden,), self.dtype)
        self.b2 = None if b2 is None else _bias(b2, (self.d,), self.dtype)
        self.norm_weight, self.act, self.eps = norm_weight, _act(act), eps

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(y, s)."""
        t, s = rms_norm(x, self.norm_weight, residual, self.eps)
        h = w4_gated(t, self.W1, self.b1, self.act)
        return w4_matmul(h, self.W2, self.b2, "NONE" if self.b2 is None else "BIAS"), s
