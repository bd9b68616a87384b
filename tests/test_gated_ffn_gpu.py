"""The gated feed-forward blocks on the GPU: their operators run together, against the same block
in 64 bits.

Tolerance, relative to a row's norm. In training every intermediate (t, z, h, dZ and the norm's
gradient) is rounded to the type once, off by at most half a step each, and the errors of a
product's terms are independent: each stage adds at most half a step times the slopes between,
which are below 1.2, and no chain has more than six of them: 8 half steps, plus the same again
for sums that partly cancel. Serving with 4-bit weights adds a rounding of each weight by at most
half its group's scale; the weights are compared after quantising, so only 16-bit rounding is left."""
import math

import pytest
import torch

from gemm_epilogues_epilog_amd import w4
from gemm_epilogues_epilog_amd.ffn import GatedFeedForward, W4FeedForward

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -20, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # (f32: a few hundred units of sums)


def block64(x, r, nw, W1, W2, b1, act, eps):
    s = x if r is None else x + r
    t = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * nw
    z = t @ W1.t() + (0 if b1 is None else b1)
    n = W1.shape[0] // 2
    g = z[:, :n]
    a = g * torch.sigmoid(g) if act == "SILU" else g.clamp(min=0) if act == "RELU" else \
        0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return (a * z[:, n:]) @ W2.t(), s


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,d,hidden,act,bias", [(1, 128, 256, "SILU", False), (7, 130, 301, "GELU", True),
                                                      (150, 256, 520, "SILU", True), (300, 264, 136, "GELU", False)])
def test_training_block(gpu, tokens, d, hidden, act, bias, dtype):
    g = torch.Generator().manual_seed(tokens + d)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(T[dtype]).cuda()   # noqa: E731
    x, res, nw = r(tokens, d), r(tokens, d), (1 + r(d, scale=0.2))
    W1, W2 = r(2 * hidden, d, scale=d ** -0.5), r(d, hidden, scale=hidden ** -0.5)
    b1 = r(2 * hidden, scale=0.3) if bias else None
    dy, ds = r(tokens, d), r(tokens, d)
    block = GatedFeedForward(nw, W1, W2, b1, act)
    y, s, saved = block.forward(x, res)
    grads = block.backward(dy, saved, ds)
    # the block in 64 bits, its gradients by differentiating the formulas; the sum s is a stored
    # value, so its rounding is taken as given
    leaves = {"dx": s.double(), "dnorm": nw.double(), "dW1": W1.double(), "dW2": W2.double()}
    if bias:
        leaves["db1"] = b1.double()
    for v in leaves.values():
        v.requires_grad_(True)
    want, s64 = block64(leaves["dx"], None, leaves["dnorm"], leaves["dW1"], leaves["dW2"], leaves.get("db1"), act, 1e-6)
    ((want * dy.double()).sum() + (s64 * ds.double()).sum()).backward()
    assert torch.equal(s, (x.float() + res.float()).to(T[dtype]))
    assert off(y, want.detach()) < 16 * HALF[dtype]
    assert set(grads) == set(leaves)
    for name, v in leaves.items():
        assert grads[name].shape == v.shape and off(grads[name], v.grad) < 16 * HALF[dtype], name
    again = block.backward(dy, block.forward(x, res)[2], ds)
    for name in grads:
        assert torch.equal(again[name], grads[name])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 30, 200])
@pytest.mark.parametrize("d,hidden,group,act,bias", [(256, 640, 128, "SILU", False), (260, 500, 32, "GELU", True)])
def test_serving_block(gpu, tokens, d, hidden, group, act, bias, dtype):
    g = torch.Generator().manual_seed(tokens + d)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(T[dtype]).cuda()   # noqa: E731
    x, res, nw = r(tokens, d), r(tokens, d), (1 + r(d, scale=0.2))
    W1, W2 = r(2 * hidden, d, scale=d ** -0.5), r(d, hidden, scale=hidden ** -0.5)
    b1, b2 = (r(2 * hidden, scale=0.3), r(d, scale=0.3)) if bias else (None, None)
    block = W4FeedForward(nw, W1, W2, b1, b2, act, group)
    y, s = block.forward(x, res)
    D = lambda q: w4.w4_dequantize(q, "f32").double()   # noqa: E731
    want, _ = block64(s.double(), None, nw.double(), D(block.W1), D(block.W2), None if b1 is None else b1.double(), act, 1e-6)
    if bias:
        want = want + b2.double()
    assert off(y, want) < 16 * HALF[dtype]
    same = W4FeedForward(nw, w4.w4_quantize(W1, group, gated=True), w4.w4_quantize(W2, group), b1, b2, act)
    assert torch.equal(same.forward(x, res)[0], y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, _ = block.forward(x, res)
    for _ in range(3):
        x.copy_(x.roll(1, 1))
        yg.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, block.forward(x, res)[0])


def test_refusals(gpu):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    for bad in (dict(W1=z(95, 64)), dict(W1=z(96, 64, dtype=torch.float64)), dict(W2=z(48, 64)), dict(W2=z(64, 48).float()),
                dict(b1=z(48)), dict(b1=z(96).half()), dict(act="TANH")):
        with pytest.raises(ValueError):
            GatedFeedForward(**{**dict(norm_weight=z(64), W1=z(96, 64), W2=z(64, 48)), **bad})
    for bad in (dict(W1=z(95, 64)), dict(W2=z(48, 64)), dict(b1=z(48)), dict(b2=z(64).float()), dict(act="NONE"),
                dict(group=48), dict(W1=w4.w4_quantize(z(96, 64), 32)), dict(W2=w4.w4_quantize(z(64, 48), 32, gated=True))):
        with pytest.raises(ValueError):
            W4FeedForward(**{**dict(norm_weight=z(64), W1=z(96, 64), W2=z(64, 48)), **bad})
    with pytest.raises(ValueError):
        GatedFeedForward(z(64), z(96, 64), z(64, 48)).forward(z(4, 63))
