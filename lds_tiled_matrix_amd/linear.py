"""The operators of a normalised linear layer in 8-bit floating point:
matrix product with block scales, block quantisation, layer norm with its
backward pass, and the clipping of gradients by their global norm.

Binding of ``include/linear/xpose_linear.h``, which has the formulas.  torch
supplies device memory (outputs, workspaces) and streams; the work runs only
in the library's gfx950 kernels.

A quantised matrix is a pair ``(q, scale)``: ``q`` a (rows, cols) tensor of
``torch.float8_e4m3fn`` whose rows start at multiples of 16 bytes, ``scale``
a float32 tensor with ceil(cols / 128) rows, one for each 128 columns of
``q``, and one column for each row of ``q`` (``block_rows`` 1) or for each
128 rows (``block_rows`` 128).  An element stands for q * scale.

Every function takes ``stream``, a torch stream to run on instead of the
current one: nothing waits for the current one then, so the arguments have to
be ready there, and what the call allocates comes from that stream's memory.
Tensors must be on the current device.  Arguments that do not fit together
raise ValueError, wrong dtypes TypeError, and what the library refuses
(alignment, overlaps) XposeError, all before anything is launched.

Nothing is recorded for autograd: results do not require gradients, whatever
the arguments do, and ``layer_norm_backward`` and the products of transposed
operands are called by hand (or from a torch.autograd.Function).  What a call
writes to a tensor given as ``out`` counts as a change in place.
"""
from __future__ import annotations

import ctypes

import lds_tiled_matrix_amd as _base

LINEAR_POW2 = 1

# Every entry point of include/linear/xpose_linear.h, in its order.
LINEAR_EXPORTS = ("xpose_fp8_gemm", "xpose_fp8_gemm_plan",
                  "xpose_fp8_quantize", "xpose_layer_norm",
                  "xpose_layer_norm_quantize", "xpose_layer_norm_backward",
                  "xpose_layer_norm_backward_workspace",
                  "xpose_clip_grad_norm", "xpose_clip_grad_norm_workspace")


class XposeFp8GemmInfo(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("workgroups", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class XposeClipTensor(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def _signatures():
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    f32, f64 = ctypes.c_float, ctypes.c_double
    i64_p, clip_p = ctypes.POINTER(i64), ctypes.POINTER(XposeClipTensor)
    norm = [i64, i64, p, i64, i32, p, p, i32, f32]
    return {
        "xpose_fp8_gemm": [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32,
                           p, i64, i32, i32, p, i64, p],
        "xpose_fp8_gemm_plan": [i64, i64, i64, i32, i32, i32,
                                ctypes.POINTER(XposeFp8GemmInfo)],
        "xpose_fp8_quantize": [i64, i64, p, i64, i32, i32, i32, p, i64, p, i64,
                               p, i64, p, i64, p],
        "xpose_layer_norm": norm + [p, i64, p, p, p],
        "xpose_layer_norm_quantize": norm + [i32, p, i64, p, i64, p, p, p],
        "xpose_layer_norm_backward": [i64, i64, p, i64, p, i64, i32, p, p, p,
                                      i32, p, i64, p, p, p, i64, p],
        "xpose_layer_norm_backward_workspace": [i64, i64, i64_p],
        "xpose_clip_grad_norm": [i64, clip_p, f64, f64, p, p, i64, p],
        "xpose_clip_grad_norm_workspace": [i64, clip_p, i64_p],
    }


def _bind(lib):
    for name, args in _signatures().items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


_lib = _base._lib
_bind(_lib)
_check = _base._check


_native = None


def _torch_side():
    """_linear.so, the torch side of these functions (csrc/linear_torch.cpp),
    loaded by the first call that needs it: the rest of the package does
    without it."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (_linear.so takes its libraries from it)
        try:
            from . import _linear
        except ImportError as e:
            raise ImportError(f"{_base._HERE}/_linear.so is not built or does not fit this torch ({e}); "
                              "run `python lds_tiled_matrix_amd/build.py`") from e
        _native = _linear
    return _native


# ----- matrix product ----------------------------------------------------------

def fp8_gemm_plan(m: int, n: int, k: int, *, block_rows: int = 1,
                  out_dtype=None, pow2: bool = False) -> dict:
    """The kernel and workspace of a product of these sizes (host only)."""
    info = XposeFp8GemmInfo()
    code = _base.XPOSE_BF16 if out_dtype is None else _base.dtype_code(out_dtype)
    _check(_lib.xpose_fp8_gemm_plan(m, n, k, block_rows, code,
                                    LINEAR_POW2 if pow2 else 0,
                                    ctypes.byref(info)), "xpose_fp8_gemm_plan")
    return info.as_dict()


def fp8_gemm(a, scale_a, b, scale_b, *, out=None, out_dtype=None,
             pow2: bool = False, stream=None):
    """a @ b.T of two quantised matrices, a (m, k) with a scale for each row
    and 128 columns, b (n, k) with the same or with one for each 128 x 128
    tile (told by ``scale_b``'s shape).  Returns an (m, n) tensor of
    ``out_dtype`` (bfloat16 unless ``out`` or it say otherwise).  float32
    results sum their products in full; 16-bit ones run at twice the rate,
    with sums a little short of float32 (see the header).

    ``pow2``: every scale is a power of two (made with ``pow2=True``), which
    the matrix cores then apply themselves."""
    return _torch_side().fp8_gemm(a, scale_a, b, scale_b, out, out_dtype, pow2, stream)


# ----- quantisation --------------------------------------------------------------

def fp8_quantize(x, *, block_rows: int = 1, pow2: bool = False,
                 transposed: bool = False, stream=None):
    """(q, scale) of a float32, float16 or bfloat16 matrix; with
    ``transposed`` (q, scale, qt, scale_t), the latter two of x.T, from one
    pass over x.  ``block_rows`` 1: a scale for each row and 128 columns (in
    each direction); 128: one for each 128 x 128 tile."""
    return tuple(_torch_side().fp8_quantize(x, block_rows, pow2, transposed, stream))


# ----- layer norm ------------------------------------------------------------------

def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5,
               stats: bool = False, out=None, stream=None):
    """Layer norm over the last dimension of a matrix: y, or with ``stats``
    (y, mean, rstd), what ``layer_norm_backward`` needs.  ``weight`` and
    ``bias`` (None: ones, zeros) are both float32 or both of a 16-bit type;
    y has x's dtype; ``out`` may be x."""
    y = _torch_side().layer_norm(x, weight, bias, eps, stats, out, stream)
    return tuple(y) if stats else y[0]


def layer_norm_quantize(x, weight=None, bias=None, *, eps: float = 1e-5,
                        pow2: bool = False, stats: bool = False, stream=None):
    """Layer norm straight to a quantised matrix: (q, scale), or with
    ``stats`` (q, scale, mean, rstd).  The normalised values are quantised
    from float32, with a scale for each row and 128 columns."""
    return tuple(_torch_side().layer_norm_quantize(x, weight, bias, eps, pow2, stats, stream))


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, stream=None):
    """(dx, dweight, dbias) of ``layer_norm(x, weight, bias, stats=True)``
    for the output's gradient dy.  dx has x's dtype; dweight and dbias are
    float32, the same bit for bit on every run."""
    return _torch_side().layer_norm_backward(dy, x, mean, rstd, weight, stream)


# ----- clipping ----------------------------------------------------------------------

def clip_grad_norm(grads, max_norm: float, *, eps: float = 1e-6, out=None,
                   stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global
    2-norm.  Returns (norm, scaled), norm a float32 tensor of no dimension
    that stays on the GPU.  ``out``: tensors of the same dtypes, shapes and
    strides (None: new ones; ``grads`` itself: in place).  Every gradient is
    float32, float16 or bfloat16 and fills one stretch of memory."""
    return _torch_side().clip_grad_norm(grads, max_norm, eps, out, stream)


def _dense(t) -> bool:
    """Whether a gradient's elements fill one stretch of memory, in any order."""
    return _torch_side().is_dense(t)
