"""The C ABI of a residual block's operators (include/linear/xpose_block.h)
without a GPU: the header is C, its functions are the binding's, and every
refusal comes back before anything is launched (addresses here are made up and
never dereferenced)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import lds_tiled_matrix_amd as X
from lds_tiled_matrix_amd import block as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "linear", "xpose_block.h")
lib = L._lib
A, B, C, D, E, F, G, H, WS, I = (0x7f0000000000 + (i << 42) for i in range(10))
OK, EINVAL, EALIAS, EDTYPE, EALIGN = X.XPOSE_OK, X.XPOSE_EINVAL, X.XPOSE_EALIAS, X.XPOSE_EDTYPE, X.XPOSE_EALIGN
EWORKSPACE = X.XPOSE_EWORKSPACE
BF16, F32, F16 = X.XPOSE_BF16, X.XPOSE_F32, X.XPOSE_F16


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = re.findall(r"\bint (xpose_\w+)\s*\(([^;]*)\)\s*;", text)
    assert tuple(name for name, _ in declared) == L.BLOCK_EXPORTS
    kinds = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "uint64_t": ctypes.c_uint64,
             "float": ctypes.c_float, "double": ctypes.c_double}
    signatures = L._signatures()
    assert sorted(signatures) == sorted(name for name, _ in declared)
    for name, args in declared:
        want = [ctypes.POINTER(ctypes.c_int64) if re.search(r"int64_t \*bytes", p) else ctypes.c_void_p if "*" in p
                else kinds[p.split()[0]] for p in (q.strip() for q in args.split(","))]
        assert signatures[name] == want, name


def test_header_is_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "linear/xpose_block.h"\nint main(void) { return 0; }\n')
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


# ----- root-mean-square norm -----------------------------------------------------

def norm(rows=20, cols=300, x=A, ldx=300, dtype=BF16, res=B, ldr=300, h=C, ldh=300, w=D, pd=F32, eps=1e-5, y=E,
         ldy=300, rstd=F):
    return lib.xpose_rms_norm(rows, cols, x, ldx, dtype, res, ldr, h, ldh, w, pd, eps, y, ldy, rstd, None)


NORM_REFUSALS = [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(rows=1 << 31), EINVAL), (dict(x=0), EINVAL),
    (dict(res=0), EINVAL), (dict(h=0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(ldx=299), EINVAL), (dict(ldr=299), EINVAL), (dict(ldh=299), EINVAL),
    (dict(dtype=X.XPOSE_U8), EDTYPE), (dict(pd=X.XPOSE_F64), EDTYPE),
    (dict(x=A + 1), EALIGN), (dict(res=B + 1), EALIGN), (dict(h=C + 1), EALIGN), (dict(w=D + 2), EALIGN),
    (dict(rstd=F + 2), EALIGN), (dict(h=A, ldh=304), EALIAS), (dict(h=A + 2), EALIAS), (dict(h=B + 300), EALIAS),
    (dict(h=D), EALIAS), (dict(rstd=A), EALIAS), (dict(rstd=C), EALIAS),
    (dict(rows=0), OK), (dict(cols=0), OK), (dict(rows=0, x=0, res=B, h=C, w=0, y=0, rstd=0), OK),
]


@pytest.mark.parametrize("args,want", NORM_REFUSALS + [
    (dict(y=0), EINVAL), (dict(ldy=299), EINVAL), (dict(y=E + 1), EALIGN), (dict(y=A, ldy=304), EALIAS),
    (dict(y=A + 2), EALIAS), (dict(y=D), EALIAS), (dict(y=C), EALIAS), (dict(y=A, h=A), EALIAS),
    (dict(y=B, h=B), EALIAS), (dict(y=F), EALIAS)])
def test_norm_refusals(args, want):
    assert norm(**args) == want


def norm_q(rows=20, cols=300, x=A, ldx=300, dtype=F16, res=B, ldr=300, h=C, ldh=300, w=D, pd=F32, eps=1e-5, flags=0,
           q=E, ldq=304, scale=G, lds=20, rstd=F):
    return lib.xpose_rms_norm_quantize(rows, cols, x, ldx, dtype, res, ldr, h, ldh, w, pd, eps, flags, q, ldq, scale,
                                       lds, rstd, None)


@pytest.mark.parametrize("args,want", NORM_REFUSALS[:-1] + [
    (dict(flags=2), EINVAL), (dict(q=0), EINVAL), (dict(scale=0), EINVAL), (dict(lds=19), EINVAL),
    (dict(ldq=300), EALIGN), (dict(q=E + 4), EALIGN), (dict(q=A), EALIAS), (dict(q=C), EALIAS),
    (dict(scale=E), EALIAS), (dict(scale=C), EALIAS), (dict(rows=0, lds=1), OK)])
def test_norm_quantize_refusals(args, want):
    assert norm_q(**args) == want


def backward(rows=20, cols=300, dy=A, lddy=300, h=B, ldh=300, dtype=F32, rstd=F, dres=C, lddr=300, w=D, pd=F32, dx=E,
             lddx=300, dw=G, ws=WS, size=1 << 30):
    return lib.xpose_rms_norm_backward(rows, cols, dy, lddy, h, ldh, dtype, rstd, dres, lddr, w, pd, dx, lddx, dw, ws,
                                       size, None)


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), EINVAL), (dict(rows=1 << 31), EINVAL), (dict(dy=0), EINVAL), (dict(h=0), EINVAL),
    (dict(rstd=0), EINVAL), (dict(dx=0), EINVAL), (dict(lddy=1), EINVAL), (dict(lddr=299), EINVAL),
    (dict(size=-1), EINVAL), (dict(dtype=X.XPOSE_F64), EDTYPE), (dict(dx=E + 2), EALIGN), (dict(dres=C + 2), EALIGN),
    (dict(dx=B), EALIAS), (dict(dx=A, lddx=301), EALIAS), (dict(dx=C, lddx=301), EALIAS), (dict(dx=C + 4), EALIAS),
    (dict(dw=E), EALIAS), (dict(dw=A), EALIAS), (dict(ws=E), EALIAS), (dict(ws=C), EALIAS), (dict(ws=0), EWORKSPACE),
    (dict(size=100), EWORKSPACE), (dict(cols=0), OK), (dict(rows=256, cols=1 << 28, lddy=1 << 28, ldh=1 << 28,
                                                            lddr=1 << 28, lddx=1 << 28, size=1 << 50), EINVAL)])
def test_backward_refusals(args, want):
    assert backward(**args) == want


def test_backward_workspace():
    size = ctypes.c_int64()
    ask = lambda r, c: lib.xpose_rms_norm_backward_workspace(r, c, ctypes.byref(size))  # noqa: E731
    assert ask(0, 100) == OK and size.value == 0
    assert ask(1, 100) == OK and size.value == 400
    assert ask(7, 10000) == OK and size.value == 4 * (7 + 7 * 10000)
    assert ask(-1, 1) == EINVAL and ask(1 << 30, 1 << 61) == EINVAL
    assert lib.xpose_rms_norm_backward_workspace(1, 1, None) == EINVAL


# ----- low-rank adapters -----------------------------------------------------------

def adapt(m=200, n=300, k=256, rank=16, count=5, x=A, ldx=256, sx=None, ldsx=0, a=B, lda=256, sa=16 * 256, b=C, ldb=16,
          sb=300 * 16, dtype=BF16, ids=I, scale=D, alpha=1.0, base=E, ldbase=300, out=F, ldout=300, od=BF16, hidden=G,
          ws=WS, size=1 << 40):
    return lib.xpose_adapters(m, n, k, rank, count, x, ldx, sx, ldsx, a, lda, sa, b, ldb, sb, dtype, ids, scale, alpha,
                              base, ldbase, out, ldout, od, hidden, ws, size, None)


SIZES = [(dict(m=-1), EINVAL), (dict(n=-1), EINVAL), (dict(k=-1), EINVAL), (dict(rank=-1), EINVAL),
         (dict(count=-1), EINVAL), (dict(m=(1 << 26) + 1), EINVAL), (dict(n=1 << 31), EINVAL), (dict(k=1 << 31), EINVAL),
         (dict(rank=4097), EINVAL), (dict(count=65536), EINVAL), (dict(x=0), EINVAL), (dict(a=0), EINVAL),
         (dict(b=0), EINVAL), (dict(ids=0), EINVAL), (dict(ldx=255), EINVAL), (dict(lda=255), EINVAL),
         (dict(ldb=15), EINVAL), (dict(sa=-1), EINVAL), (dict(sb=-1), EINVAL), (dict(size=-1), EINVAL),
         (dict(sa=1 << 62), EINVAL), (dict(dtype=X.XPOSE_U8), EDTYPE), (dict(od=X.XPOSE_F64), EDTYPE),
         (dict(od=F16), EDTYPE), (dict(dtype=F32, od=BF16), EDTYPE), (dict(x=A + 1), EALIGN), (dict(a=B + 1), EALIGN),
         (dict(b=C + 1), EALIGN), (dict(ids=I + 2), EALIGN), (dict(scale=D + 2), EALIGN)]


@pytest.mark.parametrize("args,want", SIZES + [
    (dict(out=0), EINVAL), (dict(ldout=299), EINVAL), (dict(ldbase=299), EINVAL),
    (dict(sx=H, ldsx=199, ldx=256), EINVAL), (dict(sx=H, ldsx=200, ldx=260), EALIGN),
    (dict(sx=H, ldsx=200, x=A + 8), EALIGN), (dict(sx=H + 2, ldsx=200), EALIGN),
    (dict(out=F + 1), EALIGN), (dict(hidden=G + 2), EALIGN), (dict(out=A), EALIAS), (dict(out=B + 64), EALIAS),
    (dict(out=C), EALIAS), (dict(out=I), EALIAS), (dict(out=D), EALIAS), (dict(out=E + 2), EALIAS),
    (dict(out=E, ldout=301), EALIAS), (dict(hidden=F), EALIAS), (dict(hidden=E), EALIAS), (dict(hidden=A), EALIAS),
    (dict(ws=F, hidden=None), EALIAS), (dict(ws=E, hidden=None), EALIAS), (dict(ws=WS + 4, hidden=None), EALIGN),
    (dict(ws=0, hidden=None), EWORKSPACE), (dict(size=64, hidden=None), EWORKSPACE),
    (dict(m=0, x=0, a=0, b=0, ids=0, base=0, out=0, hidden=0), OK)])
def test_adapters_refusals(args, want):
    assert adapt(**args) == want


def test_adapters_workspace():
    size = ctypes.c_int64()
    ask = lambda *v: lib.xpose_adapters_workspace(*v, ctypes.byref(size))  # noqa: E731
    assert ask(100, 0, 16, 4, 2, 0) == OK and size.value == 100 * 16 * 4
    assert ask(100, 0, 16, 4, 2, 1) == OK and size.value == 0
    assert ask(0, 4096, 16, 4, 2, 0) == OK and size.value == 0
    assert ask(100, 4096, 0, 4, 2, 0) == OK and size.value == 0
    for x_size in (1, 2, 4):
        assert ask(1, 4096, 16, 4, x_size, 0) == OK and size.value % 64 == 0 and 64 <= size.value <= 16 * 64
    assert ask(-1, 1, 1, 1, 2, 0) == EINVAL and ask(1, 1, 5000, 1, 2, 0) == EINVAL and ask(1, 1, 1, 1, 3, 0) == EINVAL
    assert lib.xpose_adapters_workspace(1, 1, 1, 1, 2, 0, None) == EINVAL


def back(m=200, n=300, k=256, rank=16, count=5, dout=F, lddout=300, x=A, ldx=256, a=B, lda=256, sa=16 * 256, b=C,
         ldb=16, sb=300 * 16, dtype=BF16, ids=I, scale=D, alpha=1.0, hidden=G, base=E, ldbase=256, dx=H, lddx=256,
         od=BF16, da=H + (1 << 38), db=H + (2 << 38), ws=WS, size=1 << 40):
    return lib.xpose_adapters_backward(m, n, k, rank, count, dout, lddout, x, ldx, a, lda, sa, b, ldb, sb, dtype, ids,
                                       scale, alpha, hidden, base, ldbase, dx, lddx, od, da, db, ws, size, None)


@pytest.mark.parametrize("args,want", SIZES + [
    (dict(dout=0), EINVAL), (dict(lddout=299), EINVAL), (dict(hidden=0), EINVAL), (dict(lddx=255), EINVAL),
    (dict(ldbase=255), EINVAL), (dict(dout=F + 1), EALIGN), (dict(hidden=G + 2), EALIGN), (dict(da=H + 2), EALIGN),
    (dict(dx=E + 2), EALIAS), (dict(dx=E, lddx=257), EALIAS), (dict(dx=A), EALIAS), (dict(dx=F), EALIAS),
    (dict(da=H), EALIAS), (dict(db=B), EALIAS), (dict(da=G), EALIAS), (dict(ws=H), EALIAS), (dict(ws=A), EALIAS),
    (dict(ws=0), EWORKSPACE), (dict(size=64), EWORKSPACE), (dict(ws=WS + 8), EALIGN),
    (dict(m=1 << 26, count=60000, n=1 << 20, k=1 << 20, ldx=1 << 20, lda=1 << 20, lddout=1 << 20, lddx=1 << 20, ldbase=1 << 20,
          dtype=F32, od=F32, size=1 << 62), EINVAL),
    (dict(dx=None, da=None, db=None), OK)])
def test_adapters_backward_refusals(args, want):
    assert back(**args) == want


def test_adapters_backward_workspace():
    size = ctypes.c_int64()
    ask = lambda *v: lib.xpose_adapters_backward_workspace(*v, ctypes.byref(size))  # noqa: E731
    assert ask(200, 300, 256, 16, 5, BF16) == OK
    rows = 4 * (200 + 6) + 4 * 200 * 16  # their order by adapter, and their gradients of rank numbers
    assert rows <= size.value <= rows + 64  # one piece an adapter: no partial sums
    assert ask(8192, 300, 256, 16, 5, BF16) == OK and size.value > 4 * 8192 * 16 + 4 * 16 * (300 + 256)
    assert ask(0, 0, 0, 0, 0, F32) == OK and size.value > 0
    assert ask(-1, 1, 1, 1, 1, F32) == EINVAL and ask(1, 1, 1, 1, 1, X.XPOSE_U8) == EDTYPE
    assert lib.xpose_adapters_backward_workspace(1, 1, 1, 1, 1, F32, None) == EINVAL


def test_adapters_limits():
    """The largest sizes are taken as far as their workspace, one more is refused before it."""
    big = dict(x=A, a=B, b=C, ids=I, base=0, ws=0, hidden=None, sa=0, sb=0)
    rows = dict(big, m=1 << 26, n=1, ldout=1, out=H + (1 << 39), a=A + (1 << 37), b=A + (1 << 38), k=1, ldx=1, lda=1)
    assert adapt(**rows) == EWORKSPACE and adapt(**dict(rows, m=(1 << 26) + 1)) == EINVAL
    wide = dict(m=2, n=1 << 30, k=1 << 30, ldx=1 << 30, lda=1 << 30, ldout=1 << 30, rank=1, ldb=1, x=1 << 44, a=2 << 44,
                b=3 << 44, out=4 << 44, base=0, ws=0, hidden=None, sa=0, sb=0)
    assert adapt(**wide) == EWORKSPACE
    assert adapt(**dict(wide, n=(1 << 30) + 1, ldout=1 << 31)) == EINVAL
    assert adapt(**dict(wide, k=(1 << 30) + 1, ldx=1 << 31, lda=1 << 31)) == EINVAL
    size = ctypes.c_int64()
    ask = lambda *v: lib.xpose_adapters_backward_workspace(*v, BF16, ctypes.byref(size))  # noqa: E731
    tiles = 64  # of n and k together
    most = ((1 << 23) - 256 - 1) // tiles - 1  # adapters next to fewer than 4096 rows
    assert most > 65535 and ask(100, 4096, 4096, 16, 65535) == OK and ask(100, 4096, 4096, 16, 65536) == EINVAL
    tiles = 512
    most = ((1 << 23) - 256 - 1) // tiles - 1
    assert ask(4095, 1 << 15, 1 << 15, 16, most) == OK and ask(4095, 1 << 15, 1 << 15, 16, most + 1) == EINVAL
    assert ask(4096, 1 << 15, 1 << 15, 16, most) == EINVAL and ask(4096, 1 << 15, 1 << 15, 16, most - 1) == OK
    assert ask(1 << 26, 1, 1, 4096, 65535) == OK and size.value > (1 << 38)


# ----- dropout -----------------------------------------------------------------------

def drop(rows=20, cols=300, x=A, ldx=300, dtype=BF16, p=0.1, seed=1, dseed=None, offset=0, res=B, ldr=300, y=C,
         ldy=300):
    return lib.xpose_dropout(rows, cols, x, ldx, dtype, p, seed, dseed, offset, res, ldr, y, ldy, None)


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), EINVAL), (dict(rows=1 << 31), EINVAL), (dict(cols=1 << 34, ldx=1 << 34, ldr=1 << 34, ldy=1 << 34), EINVAL),
    (dict(p=-0.1), EINVAL), (dict(p=1.1), EINVAL), (dict(p=float("nan")), EINVAL), (dict(x=0), EINVAL),
    (dict(y=0), EINVAL), (dict(ldx=299), EINVAL), (dict(ldr=299), EINVAL), (dict(ldy=299), EINVAL),
    (dict(dtype=X.XPOSE_F64), EDTYPE), (dict(x=A + 1), EALIGN), (dict(res=B + 1), EALIGN), (dict(y=C + 1), EALIGN),
    (dict(dseed=D + 4), EALIGN), (dict(y=A, ldy=301), EALIAS), (dict(y=A + 2), EALIAS), (dict(y=B + 2), EALIAS),
    (dict(dseed=C + 8), EALIAS), (dict(rows=0), OK), (dict(cols=0), OK)])
def test_dropout_refusals(args, want):
    assert drop(**args) == want


# ----- the binding's own checks ---------------------------------------------------------

torch = pytest.importorskip("torch")
_z = torch.zeros


@pytest.mark.parametrize("call", [
    lambda: X.rms_norm(_z(4, 4)),
    lambda: X.rms_norm(_z(4, 4), residual=_z(4, 4)),
    lambda: X.rms_norm_quantize(_z(4, 4)),
    lambda: X.rms_norm_backward(_z(4, 4), _z(4, 4), _z(4)),
    lambda: X.adapters(_z(4, 4), _z(1, 2, 4), _z(1, 4, 2), _z(4, dtype=torch.int32)),
    lambda: X.adapters_backward(_z(4, 4), _z(4, 4), _z(1, 2, 4), _z(1, 4, 2), _z(4, dtype=torch.int32), _z(4, 2)),
    lambda: X.dropout(_z(4, 4), 0.1, 1),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError):
        call()
