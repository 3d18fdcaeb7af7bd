"""CPU oracle of a residual block's operators (include/linear/xpose_block.h),
in float64 numpy from their formulas: root-mean-square norm with its backward
pass, low-rank adapters with their gradients, and the dropout mask.  It shares
no code with the kernels."""
from __future__ import annotations

import numpy as np


def rms_norm(h, weight, eps):
    """(y, rstd)."""
    h = np.asarray(h, np.float64)
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * weight, rstd


def rms_norm_backward(dy, h, rstd, weight, dresidual=0.0):
    """(dx, dweight)."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    xhat = h * rstd[:, None]
    g = dy * weight
    dx = (g - xhat * (g * xhat).mean(axis=1, keepdims=True)) * rstd[:, None]
    return dx + dresidual, (dy * xhat).sum(axis=0)


def adapters(x, a, b, ids, scale, base):
    """(out, hidden); scale: one number for each adapter."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    out, hidden = np.array(base, np.float64), np.zeros((x.shape[0], a.shape[1]))
    for row, l in enumerate(ids):
        if 0 <= l < len(a):
            hidden[row] = a[l] @ x[row]
            out[row] += scale[l] * (b[l] @ hidden[row])
    return out, hidden


def adapters_backward(dout, x, a, b, ids, scale, hidden, base):
    """(dx, da, db, dh)."""
    dout, x, a, b = (np.asarray(v, np.float64) for v in (dout, x, a, b))
    dx, da, db = np.array(base, np.float64), np.zeros(a.shape), np.zeros(b.shape)
    dh = np.zeros((len(ids), a.shape[1]))
    for row, l in enumerate(ids):
        if 0 <= l < len(a):
            dh[row] = scale[l] * (dout[row] @ b[l])
            dx[row] += dh[row] @ a[l]
            da[l] += np.outer(dh[row], x[row])
            db[l] += scale[l] * np.outer(dout[row], hidden[row])
    return dx, da, db, dh


def philox(counter, key):
    """Philox4x32-10 of four counter words and two key words, as four words:
    Python's integers, one block."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(np.floor(65536 * p + 0.5))


def dropout_mask(rows, cols, p, seed, offset, row0=0):
    """Whether each element stays, for rows row0 and on."""
    low = 0xFFFFFFFF
    keep = np.zeros((rows, cols), bool)
    for row in range(rows):
        for block in range(-(-cols // 8)):
            words = philox((block, row0 + row, offset & low, offset >> 32 & low), (seed & low, seed >> 32 & low))
            bits = [words[e // 2] >> 16 * (e % 2) & 0xFFFF for e in range(8)]
            here = min(8, cols - 8 * block)
            keep[row, 8 * block:8 * block + here] = np.array(bits[:here]) >= threshold(p)
    return keep
