"""CPU oracle of the FP8 linear layer's operators (include/linear/
xpose_linear.h), in float64 numpy from their formulas: block quantisation to
e4m3, the product of quantised matrices, layer norm with its backward pass,
and clipping by a global norm.  It shares no code with the kernels."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
SMALLEST_SCALE = np.float32(2.0 ** -126)


def e4m3_decode(bits):
    """The values that e4m3 bytes stand for, in float64."""
    b = np.asarray(bits).astype(np.int64)
    exp, frac = (b >> 3) & 15, b & 7
    mag = np.where(exp == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (exp - 10.0))
    mag = np.where((b & 127) == 127, np.nan, mag)
    return np.where(b >> 7, -mag, mag)


def e4m3_encode(x):
    """float32 values to e4m3 bytes, to nearest even; over 448 (past the
    rounding) and NaN give NaN."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    mag = np.abs(x)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(mag)
        step = np.ldexp(1.0, np.maximum(e, -5) - 4)  # 4 bits from 2^-6 on
        r = np.rint(mag / step) * step
        _, e = np.frexp(r)  # rounding may have carried
        biased = np.maximum(e - 1 + 7, 0)
        small = r < 2.0 ** -6
        frac = np.where(small, r * 2.0 ** 9, r * np.ldexp(1.0, 10 - biased) - 8)
        bits = np.where(small, frac, biased * 8 + frac)
        bits = np.where(~(r <= E4M3_MAX), 127, bits)
    return (bits.astype(np.int64) | (np.signbit(x) << 7)).astype(np.uint8)


def _padded(x, rows, cols):
    out = np.zeros((rows, cols), x.dtype)
    out[:x.shape[0], :x.shape[1]] = x
    return out


def quantize(x, block_rows=1, pow2=False):
    """(bytes, scales) of a float32 matrix."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    p = _padded(x, rb * block_rows, cb * BLOCK)
    blocks = np.abs(p).reshape(rb, block_rows, cb, BLOCK)
    with np.errstate(all="ignore"):
        amax = blocks.max(axis=(1, 3))  # a NaN stays
        scale = np.maximum(amax / np.float32(E4M3_MAX), SMALLEST_SCALE)
        if pow2:
            m, e = np.frexp(scale.astype(np.float64))
            up = np.ldexp(1.0, np.where(m == 0.5, e - 1, e))
            scale = np.where(np.isfinite(scale), up, scale).astype(np.float32)
        each = np.repeat(np.repeat(scale, block_rows, 0), BLOCK, 1)[:rows, :cols]
        q = e4m3_encode(x / each)
    return q, np.ascontiguousarray(scale.T)


def dequantize(q, scale, block_rows=1):
    rows, cols = q.shape
    each = np.repeat(np.repeat(scale.T.astype(np.float64), block_rows, 0), BLOCK, 1)
    return e4m3_decode(q) * each[:rows, :cols]


def gemm(qa, scale_a, qb, scale_b, block_rows=1):
    """(a b^T, |a| |b|^T)."""
    a, b = dequantize(qa, scale_a), dequantize(qb, scale_b, block_rows)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def layer_norm(x, weight, bias, eps):
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(axis=1) + eps)
    return d * rstd[:, None] * weight + bias, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * weight
    s1 = g.mean(axis=1, keepdims=True)
    s2 = (g * xhat).mean(axis=1, keepdims=True)
    return (g - s1 - xhat * s2) * rstd[:, None], (dy * xhat).sum(0), dy.sum(0)


def clip(grads, max_norm, eps):
    """(norm, factor)."""
    norm = math.sqrt(math.fsum(math.fsum((np.asarray(g, np.float64).ravel() ** 2).tolist())
                               for g in grads))
    return norm, min(1.0, max_norm / (norm + eps))
