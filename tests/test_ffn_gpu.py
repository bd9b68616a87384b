"""The feed-forward blocks on the GPU against the same block in 64 bits without
quantisation, and against their operators one by one.

Tolerance of the whole block, from the element types: an MXFP4 weight is off by 0.11 of
itself in the root mean square (half a step of 1/4 .. 1/2 spread evenly, and the values
above 6 held to 6), an MXFP8 activation by 0.03; the errors of a product's terms are
independent, so each product adds 0.115 relative to its result, two of them 0.16 together, and
GELU's slope is at most 1.13: 0.2. Rounding to 16 bits is nothing beside it. A token sent to a
wrong expert or a wrong row puts that row off by about 1.4. Bound: 0.3 for every row of 256
values or more."""
import numpy as np
import pytest
import torch

from gemm_epilogues_epilog_amd import mx
from gemm_epilogues_epilog_amd.ffn import MXExperts, MXFeedForward
from gemm_epilogues_epilog_amd.norm import rms_norm

pytestmark = pytest.mark.gpu

T = {"f16": torch.float16, "bf16": torch.bfloat16}


def rand(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(T[dtype])


def gelu(v):
    return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))


def norm64(x, r, w):
    s = (x + r).double().numpy()   # rounded to x's type, as the operator's sum
    return s, s / np.sqrt((s * s).mean(1, keepdims=True) + 1e-6) * w.double().numpy()


def off(got, want):
    return np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,d,hidden", [(1, 256, 1000), (5, 512, 300), (70, 300, 768), (600, 512, 1024)])
def test_feed_forward(gpu, tokens, d, hidden, dtype):
    g = torch.Generator().manual_seed(tokens + d)
    x, r = (rand(g, tokens, d, dtype=dtype) for _ in range(2))
    w = rand(g, d, dtype=dtype)
    W1, b1 = rand(g, hidden, d, dtype=dtype, scale=d ** -0.5), rand(g, hidden, dtype=dtype, scale=0.2)
    W2, b2 = rand(g, d, hidden, dtype=dtype, scale=hidden ** -0.5), rand(g, d, dtype=dtype, scale=0.2)
    s64, y64 = norm64(x, r, w)
    D = lambda t: t.double().numpy()
    want = gelu(y64 @ D(W1).T + D(b1)) @ D(W2).T + D(b2)
    with MXFeedForward(*(t.cuda() for t in (w, W1, b1, W2, b2)), d, hidden, dtype) as block:
        y, s = block.forward(x.cuda(), r.cuda())
        assert np.array_equal(s.double().cpu().numpy(), s64)
        assert (off(y.double().cpu().numpy(), want) < 0.3).all()
        again, _ = block.forward(x.cuda(), r.cuda())
        assert torch.equal(y, again)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,d,hidden,experts,top_k",
                         [(1, 256, 320, 8, 2), (7, 256, 1000, 16, 1), (90, 264, 768, 8, 3), (1000, 512, 512, 8, 2)])
def test_experts(gpu, tokens, d, hidden, experts, top_k, dtype):
    g = torch.Generator().manual_seed(tokens + d)
    x, r = (rand(g, tokens, d, dtype=dtype) for _ in range(2))
    w, R = rand(g, d, dtype=dtype), rand(g, experts, d, dtype=dtype, scale=d ** -0.5)
    W1, b1 = rand(g, experts, hidden, d, dtype=dtype, scale=d ** -0.5), rand(g, experts, hidden, dtype=dtype, scale=0.2)
    W2, b2 = rand(g, experts, d, hidden, dtype=dtype, scale=hidden ** -0.5), rand(g, experts, d, dtype=dtype, scale=0.2)
    with MXExperts(*(t.cuda() for t in (w, R, W1, b1, W2, b2)), tokens, d, hidden, experts, top_k, dtype) as block:
        out, s = block.forward(x.cuda(), r.cuda())
        s64, y64 = norm64(x, r, w)
        assert np.array_equal(s.double().cpu().numpy(), s64)
        # the routing, from the operator's y: near ties of 16-bit logits may fall either way
        y, _ = rms_norm(x.cuda(), w.cuda(), r.cuda())
        p, order, offsets = (t.cpu() for t in block.route(y))
        assert sorted(order.tolist()) == list(range(tokens * top_k))
        assert offsets[0] == 0 and offsets[-1] == tokens * top_k and (offsets.diff() >= 0).all()
        assert torch.allclose(p.sum(1), torch.ones(tokens), atol=1e-5)
        chosen = np.empty(tokens * top_k, dtype=np.int64)
        chosen[order.numpy()] = np.repeat(np.arange(experts), offsets.diff().numpy())
        chosen = chosen.reshape(tokens, top_k)
        logits = y.double().cpu().numpy() @ R.double().numpy().T
        step = 2.0 ** (-8 if dtype == "bf16" else -11) * np.abs(logits).max()
        top = np.sort(logits, 1)[:, ::-1][:, :top_k]
        assert (np.abs(np.sort(np.take_along_axis(logits, chosen, 1), 1)[:, ::-1] - top) <= 2 * step).all()
        D = lambda t: t.double().numpy()
        want = np.zeros((tokens, d))
        for t in range(tokens):
            for j in range(top_k):
                e = chosen[t, j]
                h = gelu(D(W1[e]) @ y64[t] + D(b1[e]))
                want[t] += float(p[t, j]) * (D(W2[e]) @ h + D(b2[e]))
        assert (off(out.double().cpu().numpy(), want) < 0.3).all()


def test_refusals(gpu):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    dense = lambda **k: MXFeedForward(**{**dict(norm_weight=z(64), W1=z(96, 64), b1=z(96), W2=z(64, 96), b2=z(64), d=64,
                                                hidden=96), **k})
    dense().free()
    dense(W1=mx.mx_quantize(z(96, 64), "mxfp4")).free()
    for bad in (dict(W1=z(64, 96)), dict(W2=mx.mx_quantize(z(64, 96), "mxfp8")), dict(b1=z(95)),
                dict(b2=z(64, dtype=torch.float32)), dict(dtype="f32")):
        with pytest.raises(ValueError):
            dense(**bad)
    grouped = lambda **k: MXExperts(**{**dict(norm_weight=z(64), router=z(8, 64), W1=z(8, 96, 64), b1=z(8, 96),
                                              W2=z(8, 64, 96), b2=z(8, 64), tokens=4, d=64, hidden=96, experts=8), **k})
    block = grouped()
    with pytest.raises(ValueError):
        block.forward(z(5, 64))
    block.free()
    for bad in (dict(tokens=0), dict(top_k=9), dict(top_k=0), dict(router=z(8, 63)), dict(W1=z(7, 96, 64)),
                dict(b2=z(8, 63)), dict(d=60), dict(experts=6)):
        with pytest.raises(ValueError):
            grouped(**bad)
