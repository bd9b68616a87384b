"""The microscaled operators and the norm from their definitions, in 64 bits on the CPU:
the layout address by address, the rounding by searching the list of elements."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(f * 2.0 ** -9) if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
                 for e in range(16) for f in range(8)][:127])
ELEMENTS = {"mxfp4": E2M1, "mxfp8": E4M3}
EMAX = {"mxfp4": 2, "mxfp8": 8}


def pad(v, to):
    return -(-v // to) * to


def code_at(r, k, kdim, fmt):
    """Address of the byte that holds (r, k)."""
    per = 32 if fmt == "mxfp4" else 16
    byte = (k % 32) // 2 if fmt == "mxfp4" else k % 16
    return ((r // 32) * (pad(kdim, 256) // per) + k // per) * 512 + (r % 32) * 16 + byte


def scale_at(r, k, kdim):
    return ((r // 32) * (pad(kdim, 256) // 256) + k // 256) * 256 + (k // 32 % 2) * 128 + (r % 32) * 4 + k // 64 % 4


def quantize(x, fmt):
    """(codes, scales) of x (R, K), row-major with one code per value; codes of a block
    without a finite scale are left 0."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    B = -(-K // 32)
    p = np.zeros((R, B * 32))
    p[:, :K] = x
    p = p.reshape(R, B, 32)
    top = np.max(np.abs(p), axis=-1)
    bad = ~np.isfinite(top)
    safe = np.where(bad | (top == 0), 1.0, top)
    _, e = np.frexp(safe)
    s = np.clip(e - 1 - EMAX[fmt] + 127, 0, 254)
    s = np.where(top == 0, 0, s)
    t = ELEMENTS[fmt]
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(p) / np.exp2(s - 127.0)[..., None], t[-1])
    a = np.where(bad[..., None], 0.0, a)
    hi = np.minimum(np.searchsorted(t, a), len(t) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = t[hi] - a, a - t[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = c + np.where(np.signbit(p) & ~bad[..., None], len(E2M1) if fmt == "mxfp4" else 128, 0)
    return c.reshape(R, -1)[:, :K].astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def values(codes, scales, fmt):
    """What row-major codes and scales stand for."""
    t = ELEMENTS[fmt]
    t = np.concatenate([t, -t]) if fmt == "mxfp4" else np.concatenate([t, [np.nan], -t, [np.nan]])
    f = np.exp2(scales.astype(np.float64) - 127)
    f[scales == 255] = np.nan
    return t[codes] * np.repeat(f, 32, axis=1)[:, : codes.shape[1]]


def pack(codes, scales, fmt):
    R, K = codes.shape
    out = np.zeros(pad(R, 32) * pad(K, 256) // (2 if fmt == "mxfp4" else 1), np.uint8)
    so = np.zeros(pad(R, 32) * pad(K, 256) // 32, np.uint8)
    r, k = np.meshgrid(np.arange(R), np.arange(K), indexing="ij")
    if fmt == "mxfp4":
        for odd in (0, 1):
            m = k % 2 == odd
            out[code_at(r[m], k[m], K, fmt)] |= (codes[m] << (4 * odd)).astype(np.uint8)
    else:
        out[code_at(r, k, K, fmt)] = codes
    r, b = np.meshgrid(np.arange(R), np.arange(scales.shape[1]) * 32, indexing="ij")
    so[scale_at(r, b, K)] = scales
    return out, so


def unpack(packed, pscales, R, K, fmt):
    r, k = np.meshgrid(np.arange(R), np.arange(K), indexing="ij")
    c = packed[code_at(r, k, K, fmt)]
    if fmt == "mxfp4":
        c = (c >> (4 * (k % 2)).astype(np.uint8)) & 15
    r, b = np.meshgrid(np.arange(R), np.arange(-(-K // 32)) * 32, indexing="ij")
    return c, pscales[scale_at(r, b, K)]


def gelu(v):
    return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def activate(v, ep):
    if ep == "RELU_BIAS":
        return np.where(v > 0, v, 0.0)
    return gelu(v) if ep == "GELU_BIAS" else v


def rms_norm(s, w, eps):
    s, w = np.asarray(s, np.float64), np.asarray(w, np.float64)
    return s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * w


def rms_norm_backward(dy, s, w, eps, dres=None):
    dy, s, w = (np.asarray(v, np.float64) for v in (dy, s, w))
    r = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    g, h = dy * w, s * r
    dx = r * (g - h * np.mean(g * h, axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, np.sum(dy * h, axis=0)
