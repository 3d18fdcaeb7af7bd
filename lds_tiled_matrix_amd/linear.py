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
current one.
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
_DTYPES = None


def _dtype(t, what: str) -> int:
    """XPOSE_F32, _F16 or _BF16 for a torch dtype: here the type matters, not
    only its size."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: _base.XPOSE_F32,
                   torch.float16: _base.XPOSE_F16,
                   torch.bfloat16: _base.XPOSE_BF16}
    code = _DTYPES.get(t)
    if code is None:
        raise TypeError(f"{what}: expected float32, float16 or bfloat16, got {t}")
    return code


def _stream(device, stream) -> int:
    import torch
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _on_device(first, *others) -> None:
    """Device tensors of one device: checked before anything is launched, so a
    host tensor is a Python error, not a GPU fault."""
    if not first.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {first.device}")
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on different devices: {first.device}, {t.device}")


def _record(stream, *tensors) -> None:
    """Tensors allocated on the current stream but used on ``stream`` are kept
    from being reused before its work has run."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _matrix(t, what: str):
    """(rows, cols, pitch) of a 2-D tensor whose last dim is contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return rows, cols, (t.stride(0) if rows > 1 else max(cols, 1))


def _vector(t, n: int, dtype, what: str) -> int:
    """The address of n contiguous values (None: 0)."""
    if t is None:
        return 0
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what}: expected {n} contiguous values")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _empty_e4m3(rows: int, cols: int, device):
    """Uninitialised e4m3 values, rows at multiples of 16 bytes, long ones at
    whole 128-byte lines."""
    import torch
    pitch = (cols + 15) & ~15 if cols < 1024 else (cols + 127) & ~127
    q = torch.empty((rows, pitch), dtype=torch.float8_e4m3fn, device=device)
    return q if pitch == cols else q[:, :cols]


# ----- matrix product ----------------------------------------------------------

def fp8_gemm_plan(m: int, n: int, k: int, *, block_rows: int = 1,
                  out_dtype=None, pow2: bool = False) -> dict:
    """The kernel and workspace of a product of these sizes (host only)."""
    info = XposeFp8GemmInfo()
    out = _base.XPOSE_BF16 if out_dtype is None else _dtype(out_dtype, "out_dtype")
    _check(_lib.xpose_fp8_gemm_plan(m, n, k, block_rows, out,
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
    import torch
    _on_device(a, scale_a, b, scale_b, out)
    e4m3 = torch.float8_e4m3fn
    if a.dtype != e4m3 or b.dtype != e4m3:
        raise TypeError(f"a, b: expected {e4m3}, got {a.dtype}, {b.dtype}")
    if scale_a.dtype != torch.float32 or scale_b.dtype != torch.float32:
        raise TypeError("scale_a, scale_b: expected float32")
    m, k, lda = _matrix(a, "a")
    n, kb, ldb = _matrix(b, "b")
    if kb != k:
        raise ValueError("inner dimensions differ")
    blocks = (k + 127) // 128
    sa_rows, sa_cols, ldsa = _matrix(scale_a, "scale_a")
    sb_rows, sb_cols, ldsb = _matrix(scale_b, "scale_b")
    if sa_rows != blocks or sa_cols != m:
        raise ValueError(f"scale_a: expected ({blocks}, {m}), got {tuple(scale_a.shape)}")
    if sb_cols == n:
        block_rows = 1
    elif sb_cols == (n + 127) // 128:
        block_rows = 128
    else:
        block_rows = 0
    if sb_rows != blocks or not block_rows:
        raise ValueError(f"scale_b: expected ({blocks}, {n}) or "
                         f"({blocks}, {(n + 127) // 128}), got {tuple(scale_b.shape)}")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=a.device)
    elif tuple(out.shape) != (m, n):
        raise ValueError("out has the wrong shape")
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out and out_dtype differ")
    code = _dtype(out.dtype, "out")
    _, _, ldc = _matrix(out, "out")
    flags = LINEAR_POW2 if pow2 else 0
    info = XposeFp8GemmInfo()
    _check(_lib.xpose_fp8_gemm_plan(m, n, k, block_rows, code, flags,
                                    ctypes.byref(info)), "xpose_fp8_gemm_plan")
    size = info.workspace_bytes
    ws = torch.empty(size, dtype=torch.uint8, device=a.device) if size else None
    _check(_lib.xpose_fp8_gemm(
        m, n, k, a.data_ptr(), lda, scale_a.data_ptr(), ldsa, b.data_ptr(),
        ldb, scale_b.data_ptr(), ldsb, block_rows, out.data_ptr(), ldc, code,
        flags, ws.data_ptr() if size else 0, size, _stream(a.device, stream)),
        "xpose_fp8_gemm")
    _record(stream, ws, out)
    return out


# ----- quantisation --------------------------------------------------------------

def fp8_quantize(x, *, block_rows: int = 1, pow2: bool = False,
                 transposed: bool = False, stream=None):
    """(q, scale) of a float32, float16 or bfloat16 matrix; with
    ``transposed`` (q, scale, qt, scale_t), the latter two of x.T, from one
    pass over x.  ``block_rows`` 1: a scale for each row and 128 columns (in
    each direction); 128: one for each 128 x 128 tile."""
    import torch
    _on_device(x)
    code = _dtype(x.dtype, "x")
    rows, cols, ldx = _matrix(x, "x")
    if block_rows not in (1, 128):
        raise ValueError("block_rows is 1 or 128")
    blocks_r, blocks_c = (rows + 127) // 128, (cols + 127) // 128
    tiles = block_rows == 128
    dev = x.device
    q = _empty_e4m3(rows, cols, dev)
    scale = torch.empty((blocks_c, blocks_r if tiles else rows),
                        dtype=torch.float32, device=dev)
    qt = scale_t = None
    turned = (0, max(rows, 1), 0, 1)
    if transposed:
        qt = _empty_e4m3(cols, rows, dev)
        scale_t = torch.empty((blocks_r, blocks_c if tiles else cols),
                              dtype=torch.float32, device=dev)
        turned = (qt.data_ptr(), max(qt.stride(0), 1), scale_t.data_ptr(),
                  max(scale_t.shape[1], 1))
    if rows and cols:
        _check(_lib.xpose_fp8_quantize(
            rows, cols, x.data_ptr(), ldx, code, block_rows,
            LINEAR_POW2 if pow2 else 0, q.data_ptr(), q.stride(0),
            scale.data_ptr(), scale.shape[1], *turned,
            _stream(dev, stream)), "xpose_fp8_quantize")
    _record(stream, q, scale, qt, scale_t)
    return (q, scale, qt, scale_t) if transposed else (q, scale)


# ----- layer norm ------------------------------------------------------------------

def _norm_args(x, weight, bias, stats: bool):
    import torch
    _on_device(x, weight, bias)
    code = _dtype(x.dtype, "x")
    rows, cols, ldx = _matrix(x, "x")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias have different dtypes")
    param = weight if weight is not None else bias
    pcode = 0 if param is None else _dtype(param.dtype, "weight, bias")
    mean = rstd = None
    if stats:
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    head = (rows, cols, x.data_ptr(), ldx, code, _vector(weight, cols, None, "weight"),
            _vector(bias, cols, None, "bias"), pcode)
    tail = (mean.data_ptr(), rstd.data_ptr()) if stats and rows else (0, 0)
    return rows, cols, head, tail, mean, rstd


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5,
               stats: bool = False, out=None, stream=None):
    """Layer norm over the last dimension of a matrix: y, or with ``stats``
    (y, mean, rstd), what ``layer_norm_backward`` needs.  ``weight`` and
    ``bias`` (None: ones, zeros) are both float32 or both of a 16-bit type;
    y has x's dtype; ``out`` may be x."""
    import torch
    rows, cols, head, tail, mean, rstd = _norm_args(x, weight, bias, stats)
    if cols == 0:
        raise ValueError("layer norm over no columns")
    if out is None:
        out = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    else:
        _on_device(x, out)
        if out.dtype != x.dtype or out.shape != x.shape:
            raise ValueError("out must match x's dtype and shape")
    _, _, ldy = _matrix(out, "out")
    _check(_lib.xpose_layer_norm(*head, eps, out.data_ptr(), ldy, *tail,
                                 _stream(x.device, stream)), "xpose_layer_norm")
    _record(stream, out, mean, rstd)
    return (out, mean, rstd) if stats else out


def layer_norm_quantize(x, weight=None, bias=None, *, eps: float = 1e-5,
                        pow2: bool = False, stats: bool = False, stream=None):
    """Layer norm straight to a quantised matrix: (q, scale), or with
    ``stats`` (q, scale, mean, rstd).  The normalised values are quantised
    from float32, with a scale for each row and 128 columns."""
    import torch
    rows, cols, head, tail, mean, rstd = _norm_args(x, weight, bias, stats)
    if cols == 0:
        raise ValueError("layer norm over no columns")
    q = _empty_e4m3(rows, cols, x.device)
    scale = torch.empty(((cols + 127) // 128, rows), dtype=torch.float32,
                        device=x.device)
    _check(_lib.xpose_layer_norm_quantize(
        *head, eps, LINEAR_POW2 if pow2 else 0, q.data_ptr(), q.stride(0),
        scale.data_ptr(), max(rows, 1), *tail, _stream(x.device, stream)),
        "xpose_layer_norm_quantize")
    _record(stream, q, scale, mean, rstd)
    return (q, scale, mean, rstd) if stats else (q, scale)


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, stream=None):
    """(dx, dweight, dbias) of ``layer_norm(x, weight, bias, stats=True)``
    for the output's gradient dy.  dx has x's dtype; dweight and dbias are
    float32, the same bit for bit on every run."""
    import torch
    _on_device(x, dy, mean, rstd, weight)
    code = _dtype(x.dtype, "x")
    rows, cols, ldx = _matrix(x, "x")
    if cols == 0:
        raise ValueError("layer norm over no columns")
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError("dy must match x's dtype and shape")
    _, _, lddy = _matrix(dy, "dy")
    dev, f32 = x.device, torch.float32
    pcode = 0 if weight is None else _dtype(weight.dtype, "weight")
    args = (_vector(mean, rows, f32, "mean"), _vector(rstd, rows, f32, "rstd"),
            _vector(weight, cols, None, "weight"), pcode)
    dx = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    dweight = torch.empty(cols, dtype=f32, device=dev)
    dbias = torch.empty(cols, dtype=f32, device=dev)
    size = ctypes.c_int64()
    _check(_lib.xpose_layer_norm_backward_workspace(rows, cols, ctypes.byref(size)),
           "xpose_layer_norm_backward_workspace")
    ws = torch.empty(size.value // 4, dtype=f32, device=dev)
    _check(_lib.xpose_layer_norm_backward(
        rows, cols, dy.data_ptr(), lddy, x.data_ptr(), ldx, code, *args,
        dx.data_ptr(), cols, dweight.data_ptr(), dbias.data_ptr(),
        ws.data_ptr(), size.value, _stream(dev, stream)),
        "xpose_layer_norm_backward")
    _record(stream, ws, dx, dweight, dbias)
    return dx, dweight, dbias


# ----- clipping ----------------------------------------------------------------------

def _dense(t) -> bool:
    """Whether the elements fill one stretch of memory, in any order."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size == 1:
            continue
        if stride != step:
            return False
        step *= size
    return True


def clip_grad_norm(grads, max_norm: float, *, eps: float = 1e-6, out=None,
                   stream=None):
    """Scales gradients by min(1, max_norm / (norm + eps)), norm their global
    2-norm.  Returns (norm, scaled), norm a float32 tensor of no dimension
    that stays on the GPU.  ``out``: tensors of the same dtypes, shapes and
    strides (None: new ones; ``grads`` itself: in place).  Every gradient is
    float32, float16 or bfloat16 and fills one stretch of memory."""
    import torch
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    if out is None:
        out = [torch.empty_like(g) for g in grads]
    elif len(out) != len(grads):
        raise ValueError(f"{len(grads)} gradients, {len(out)} outputs")
    device = grads[0].device
    if device.type != "cuda":
        raise ValueError(f"expected a CUDA tensor, got one on {device}")
    table = (XposeClipTensor * len(grads))()
    for entry, g, o in zip(table, grads, out):
        if g.device != device or o.device != device:
            raise ValueError(f"tensors on different devices: {g.device}, {o.device}, {device}")
        if o.dtype != g.dtype or o.shape != g.shape:
            raise ValueError("an output differs from its gradient in dtype or shape")
        if o is not g and o.stride() != g.stride() and g.numel():
            raise ValueError("an output differs from its gradient in strides")
        if not _dense(g):
            raise ValueError("a gradient does not fill one stretch of memory")
        entry.inp = g.data_ptr()
        entry.out = o.data_ptr()
        entry.count = g.numel()
        entry.dtype = _dtype(g.dtype, "grads")
    size = ctypes.c_int64()
    _check(_lib.xpose_clip_grad_norm_workspace(len(grads), table, ctypes.byref(size)),
           "xpose_clip_grad_norm_workspace")
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws = torch.empty(size.value // 8, dtype=torch.float64, device=device)
    _check(_lib.xpose_clip_grad_norm(len(grads), table, max_norm, eps,
                                     norm.data_ptr(), ws.data_ptr(), size.value,
                                     _stream(device, stream)), "xpose_clip_grad_norm")
    _record(stream, norm, ws, *out)
    return norm, out
