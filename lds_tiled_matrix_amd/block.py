"""What stands around a linear layer in a residual stream: root-mean-square
norm with the residual's addition and its backward pass, low-rank adapters of
many requests beside the layer's shared product with their gradients, and
dropout from a counter-based generator.

Binding of ``include/linear/xpose_block.h``, which has the formulas.  Streams,
devices, errors, quantised matrices and autograd are as in ``linear.py``: torch
supplies memory and streams, ``stream`` is one to run on instead of the current
one, nothing is recorded for autograd, and what a call writes to a tensor given
as ``out`` or ``residual_out`` counts as a change in place.
"""
from __future__ import annotations

import ctypes
import operator

from .linear import _lib, _torch_side

# Every entry point of include/linear/xpose_block.h, in its order.
BLOCK_EXPORTS = ("xpose_rms_norm", "xpose_rms_norm_quantize",
                 "xpose_rms_norm_backward", "xpose_rms_norm_backward_workspace",
                 "xpose_adapters", "xpose_adapters_workspace",
                 "xpose_adapters_backward", "xpose_adapters_backward_workspace",
                 "xpose_dropout")


def _signatures():
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    f32, f64, u64 = ctypes.c_float, ctypes.c_double, ctypes.c_uint64
    i64_p = ctypes.POINTER(i64)
    norm = [i64, i64, p, i64, i32, p, i64, p, i64, p, i32, f32]
    sizes, weights = [i64] * 5, [p, i64, i64, p, i64, i64, i32, p, p, f32]
    return {
        "xpose_rms_norm": norm + [p, i64, p, p],
        "xpose_rms_norm_quantize": norm + [i32, p, i64, p, i64, p, p],
        "xpose_rms_norm_backward": [i64, i64, p, i64, p, i64, i32, p, p, i64, p, i32, p, i64, p, p, i64, p],
        "xpose_rms_norm_backward_workspace": [i64, i64, i64_p],
        "xpose_adapters": sizes + [p, i64, p, i64] + weights + [p, i64, p, i64, i32, p, p, i64, p],
        "xpose_adapters_workspace": [i64, i64, i64, i64, i32, i32, i64_p],
        "xpose_adapters_backward": sizes + [p, i64, p, i64] + weights + [p, p, i64, p, i64, i32, p, p, p, i64, p],
        "xpose_adapters_backward_workspace": [i64, i64, i64, i64, i64, i32, i64_p],
        "xpose_dropout": [i64, i64, p, i64, i32, f64, u64, p, u64, p, i64, p, i64, p],
    }


def _bind(lib):
    for name, args in _signatures().items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


_bind(_lib)


# ----- root-mean-square norm ---------------------------------------------------

def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-5, stats: bool = False, out=None, residual_out=None,
             stream=None):
    """Root-mean-square norm over the last dimension of a matrix, of x or, with
    ``residual``, of h = x + residual rounded to x's dtype: y, (y, h), and with
    ``stats`` also rstd, the last.  ``weight`` (None: ones) is float32 or of a
    16-bit type; y and h have x's dtype; ``out`` and ``residual_out`` (where h
    goes) may each be x or residual."""
    got = _torch_side().rms_norm(x, weight, residual, eps, stats, out, residual_out, stream)
    return tuple(got) if len(got) > 1 else got[0]


def rms_norm_quantize(x, weight=None, *, residual=None, eps: float = 1e-5, pow2: bool = False, stats: bool = False,
                      residual_out=None, stream=None):
    """The same straight to a quantised matrix: (q, scale), then h with
    ``residual`` and rstd with ``stats``.  The normalised values are quantised
    from float32, with a scale for each row and 128 columns."""
    return tuple(_torch_side().rms_norm_quantize(x, weight, residual, eps, pow2, stats, residual_out, stream))


def rms_norm_backward(dy, h, rstd, weight=None, *, dresidual=None, stream=None):
    """(dx, dweight) for the output's gradient dy; h and rstd are what
    ``rms_norm(..., stats=True)`` gave (h: x where there was no residual).
    ``dresidual`` is the gradient that h has from the rest of the stream, and
    is added to dx, which is then x's and the residual's alike.  dx has h's
    dtype; dweight is float32, the same bit for bit on every run."""
    return _torch_side().rms_norm_backward(dy, h, rstd, weight, dresidual, stream)


# ----- low-rank adapters ---------------------------------------------------------

def adapters(x, a, b, ids, *, base=None, scale=1.0, scale_x=None, hidden: bool = False, out=None, stream=None):
    """base + scale (x A.T) B.T with the A and B of each row's adapter: row i
    has ``a[ids[i]]`` and ``b[ids[i]]``, and rows whose id is not one of them
    (-1) have none and get base.

    ``x``: (m, k) of the adapters' dtype, or e4m3 with its scales ``scale_x``;
    ``a``: (count, rank, k), ``b``: (count, n, rank), float32, float16 or
    bfloat16; ``ids``: m values of int32, in any order; ``base`` (None: zeros):
    (m, n) of the adapters' dtype or float32, which the result has too;
    ``scale``: a number, or a float32 tensor of one for each adapter.  ``out``
    may be base itself (x where that is base); rows without an adapter are left
    as they are then.
    With ``hidden`` (out, hidden), the latter x A.T in float32, which
    ``adapters_backward`` needs."""
    got = _torch_side().adapters(x, a, b, ids, base, scale, scale_x, hidden, out, stream)
    return tuple(got) if hidden else got[0]


def adapters_backward(dout, x, a, b, ids, hidden, *, base=None, scale=1.0, wanted=(True, True, True), out=None,
                      stream=None):
    """(dx, da, db) for the gradient dout of ``adapters(x, a, b, ids,
    hidden=True)``.  ``base`` (None: zeros) is what dx is added to, such as the
    shared product's gradient of x, and sets its dtype; ``out``, where dx goes,
    may be base itself (dout or x where that is base).  da and db are float32,
    shaped as a and b, zeros for adapters of no row.  ``wanted`` says which of
    the three are: the others are None and not computed; the workspace that the
    call takes from torch's allocator is the same."""
    return tuple(_torch_side().adapters_backward(dout, x, a, b, ids, hidden, base, scale, list(wanted), out, stream))


# ----- dropout ---------------------------------------------------------------------

def dropout(x, p: float, seed, *, offset: int = 0, residual=None, out=None, stream=None):
    """residual + x / (1 - p) where an element stays, residual (None: zeros)
    where it is dropped.  Whether it stays is a function of ``seed``,
    ``offset`` and the element's row and column alone, so nothing is stored: the
    gradient of x is ``dropout(dy, p, seed, offset=offset)``.

    ``seed``: a number, or an int64 tensor of one value that the GPU reads, for
    graphs whose replays are to differ.  ``offset`` tells the dropouts of one
    seed apart; both count modulo 2^64.  p counts in steps of 2^-16.  ``out``
    may be x or residual."""
    if hasattr(seed, "__index__") and not hasattr(seed, "data_ptr"):
        seed = operator.index(seed) & ((1 << 64) - 1)
    return _torch_side().dropout(x, p, seed, operator.index(offset) & ((1 << 64) - 1), residual, out, stream)
