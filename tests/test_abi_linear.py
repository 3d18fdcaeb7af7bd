"""The FP8 linear layer's C ABI (include/linear/xpose_linear.h) without a GPU:
the header is C, its functions are the binding's, plans follow their rules,
and every refusal comes back before anything is launched (addresses here are
made up and never dereferenced)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import lds_tiled_matrix_amd as X
from lds_tiled_matrix_amd import linear as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "linear", "xpose_linear.h")
lib = L._lib
A, B, C, SA, SB, WS, Q, QT = (0x7f0000000000 + (i << 40) for i in range(8))


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = re.findall(r"\bint (xpose_\w+)\s*\(", text)
    assert tuple(declared) == L.LINEAR_EXPORTS
    assert sorted(L._signatures()) == sorted(declared)


def test_header_is_c_and_structs_match(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n'
                   '#include "linear/xpose_linear.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %d", sizeof(xpose_fp8_gemm_info),'
                   'offsetof(xpose_fp8_gemm_info, workspace_bytes), sizeof(xpose_clip_tensor),'
                   'offsetof(xpose_clip_tensor, dtype), XPOSE_LINEAR_POW2); return 0; }\n')
    exe = tmp_path / "t"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in got.split()] == [
        ctypes.sizeof(L.XposeFp8GemmInfo), L.XposeFp8GemmInfo.workspace_bytes.offset,
        ctypes.sizeof(L.XposeClipTensor), L.XposeClipTensor.dtype.offset, L.LINEAR_POW2]


# ----- matrix product -----------------------------------------------------------

def gemm(m=200, n=300, k=256, a=A, lda=256, sa=SA, ldsa=200, b=B, ldb=256, sb=SB,
         ldsb=300, rows=1, c=C, ldc=300, out=X.XPOSE_BF16, flags=0, ws=WS, size=1 << 40):
    return lib.xpose_fp8_gemm(m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, rows, c, ldc,
                              out, flags, ws, size, None)


@pytest.mark.parametrize("args,want", [
    (dict(m=-1), X.XPOSE_EINVAL), (dict(n=-1), X.XPOSE_EINVAL), (dict(k=-1), X.XPOSE_EINVAL),
    (dict(a=0), X.XPOSE_EINVAL), (dict(b=0), X.XPOSE_EINVAL), (dict(c=0), X.XPOSE_EINVAL),
    (dict(sa=0), X.XPOSE_EINVAL), (dict(sb=0), X.XPOSE_EINVAL),
    (dict(lda=255), X.XPOSE_EINVAL), (dict(ldb=240), X.XPOSE_EINVAL), (dict(ldc=299), X.XPOSE_EINVAL),
    (dict(ldsa=199), X.XPOSE_EINVAL), (dict(ldsb=299), X.XPOSE_EINVAL),
    (dict(rows=128, ldsb=2), X.XPOSE_EINVAL), (dict(rows=64), X.XPOSE_EINVAL),
    (dict(lda=1 << 23), X.XPOSE_EINVAL), (dict(ldb=1 << 23), X.XPOSE_EINVAL),
    (dict(k=1 << 23, lda=1 << 23), X.XPOSE_EINVAL),
    (dict(flags=2), X.XPOSE_EINVAL), (dict(size=-1), X.XPOSE_EINVAL),
    (dict(m=1 << 62, ldsa=1 << 62), X.XPOSE_EINVAL), (dict(ldc=1 << 62), X.XPOSE_EINVAL),
    (dict(out=X.XPOSE_U8), X.XPOSE_EDTYPE), (dict(out=9), X.XPOSE_EDTYPE),
    (dict(a=A + 8), X.XPOSE_EALIGN), (dict(b=B + 1), X.XPOSE_EALIGN), (dict(c=C + 1), X.XPOSE_EALIGN),
    (dict(lda=264), X.XPOSE_EALIGN), (dict(ldb=257), X.XPOSE_EALIGN), (dict(sa=SA + 2), X.XPOSE_EALIGN),
    (dict(c=A), X.XPOSE_EALIAS), (dict(c=B + 64), X.XPOSE_EALIAS), (dict(c=SA), X.XPOSE_EALIAS),
    (dict(c=SB), X.XPOSE_EALIAS),
    (dict(k=16384, lda=16384, ldb=16384, ws=0), X.XPOSE_EWORKSPACE),
    (dict(k=16384, lda=16384, ldb=16384, size=64), X.XPOSE_EWORKSPACE),
    (dict(k=16384, lda=16384, ldb=16384, ws=C), X.XPOSE_EALIAS),
    (dict(k=16384, lda=16384, ldb=16384, ws=WS + 4), X.XPOSE_EALIGN),
    (dict(m=0, ldsa=1), X.XPOSE_OK), (dict(n=0), X.XPOSE_OK), (dict(m=0, a=0, b=0, c=0, sa=0, sb=0), X.XPOSE_OK),
])
def test_gemm_refusals(args, want):
    assert gemm(**args) == want


def plan(m, n, k, rows=1, out=X.XPOSE_BF16, flags=0):
    info = L.XposeFp8GemmInfo()
    return lib.xpose_fp8_gemm_plan(m, n, k, rows, out, flags, ctypes.byref(info)), info


@pytest.mark.parametrize("m", [1, 16, 17, 64, 65, 200, 1000, 8192])
@pytest.mark.parametrize("n", [16, 300, 2999, 8192])
@pytest.mark.parametrize("k", [0, 1, 128, 1000, 12345, 1 << 20])
def test_gemm_plans_cover_the_product(m, n, k):
    rc, i = plan(m, n, k)
    assert rc == X.XPOSE_OK
    tiles = -(-m // i.tile_m) * -(-n // i.tile_n)
    assert i.workgroups == tiles * i.splits and i.splits >= 1
    assert i.splits <= max(1, -(-k // 128))
    assert i.workspace_bytes == (4 * m * n * i.splits if i.splits > 1 else 0)


def test_gemm_plan_refusals():
    assert plan(-1, 1, 1)[0] == X.XPOSE_EINVAL
    assert plan(1, 1, 1, rows=2)[0] == X.XPOSE_EINVAL
    assert plan(1, 1, 1, out=X.XPOSE_F64)[0] == X.XPOSE_EDTYPE
    assert plan(1 << 40, 1 << 40, 1)[0] == X.XPOSE_EINVAL
    assert lib.xpose_fp8_gemm_plan(1, 1, 1, 1, 0, 0, None) == X.XPOSE_EINVAL
    rc, info = plan(0, 5, 5)
    assert rc == X.XPOSE_OK and info.workgroups == 0


# ----- quantisation ---------------------------------------------------------------

def quantize(rows=200, cols=300, x=A, ldx=300, dtype=X.XPOSE_BF16, block=1, flags=0, q=Q,
             ldq=304, scale=SA, lds=200, qt=QT, ldqt=208, scale_t=SB, ldst=300):
    return lib.xpose_fp8_quantize(rows, cols, x, ldx, dtype, block, flags, q, ldq, scale,
                                  lds, qt, ldqt, scale_t, ldst, None)


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), X.XPOSE_EINVAL), (dict(x=0), X.XPOSE_EINVAL), (dict(q=0), X.XPOSE_EINVAL),
    (dict(scale=0), X.XPOSE_EINVAL), (dict(scale_t=0), X.XPOSE_EINVAL), (dict(block=2), X.XPOSE_EINVAL),
    (dict(flags=4), X.XPOSE_EINVAL), (dict(ldx=299), X.XPOSE_EINVAL), (dict(ldq=296), X.XPOSE_EINVAL),
    (dict(lds=199), X.XPOSE_EINVAL), (dict(ldqt=192), X.XPOSE_EINVAL), (dict(ldst=299), X.XPOSE_EINVAL),
    (dict(rows=1 << 40, cols=1 << 40, ldx=1 << 40, ldq=1 << 40), X.XPOSE_EINVAL),
    (dict(dtype=X.XPOSE_F64), X.XPOSE_EDTYPE),
    (dict(x=A + 1), X.XPOSE_EALIGN), (dict(q=Q + 4), X.XPOSE_EALIGN), (dict(ldq=301), X.XPOSE_EALIGN),
    (dict(qt=QT + 1), X.XPOSE_EALIGN), (dict(ldqt=204), X.XPOSE_EALIGN),
    (dict(q=A), X.XPOSE_EALIAS), (dict(qt=Q), X.XPOSE_EALIAS), (dict(scale=Q), X.XPOSE_EALIAS),
    (dict(scale_t=SA), X.XPOSE_EALIAS),
    (dict(rows=0, x=0, q=0, qt=0, scale=0, scale_t=0, lds=1), X.XPOSE_OK), (dict(cols=0), X.XPOSE_OK),
])
def test_quantize_refusals(args, want):
    assert quantize(**args) == want


# ----- layer norm -------------------------------------------------------------------

def norm(rows=20, cols=300, x=A, ldx=300, dtype=X.XPOSE_BF16, w=B, b=SB, pd=X.XPOSE_F32, eps=1e-5,
         y=C, ldy=300, mean=Q, rstd=QT):
    return lib.xpose_layer_norm(rows, cols, x, ldx, dtype, w, b, pd, eps, y, ldy, mean, rstd, None)


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), X.XPOSE_EINVAL), (dict(x=0), X.XPOSE_EINVAL), (dict(y=0), X.XPOSE_EINVAL),
    (dict(mean=0), X.XPOSE_EINVAL), (dict(rstd=0), X.XPOSE_EINVAL), (dict(eps=-1.0), X.XPOSE_EINVAL),
    (dict(eps=float("nan")), X.XPOSE_EINVAL), (dict(ldx=299), X.XPOSE_EINVAL), (dict(ldy=299), X.XPOSE_EINVAL),
    (dict(dtype=X.XPOSE_U8), X.XPOSE_EDTYPE), (dict(pd=X.XPOSE_U8), X.XPOSE_EDTYPE),
    (dict(x=A + 1), X.XPOSE_EALIGN), (dict(w=B + 2), X.XPOSE_EALIGN), (dict(mean=Q + 2), X.XPOSE_EALIGN),
    (dict(y=A, ldy=304), X.XPOSE_EALIAS), (dict(y=A + 2), X.XPOSE_EALIAS), (dict(y=B), X.XPOSE_EALIAS),
    (dict(mean=A), X.XPOSE_EALIAS), (dict(rstd=Q), X.XPOSE_EALIAS),
    (dict(rows=0), X.XPOSE_OK), (dict(cols=0), X.XPOSE_OK),
])
def test_norm_refusals(args, want):
    assert norm(**args) == want


def norm_q(rows=20, cols=300, x=A, ldx=300, w=B, b=SB, eps=1e-5, flags=0, q=C, ldq=304, scale=SA, lds=20,
           mean=Q, rstd=QT):
    return lib.xpose_layer_norm_quantize(rows, cols, x, ldx, X.XPOSE_F16, w, b, X.XPOSE_F32, eps, flags, q,
                                         ldq, scale, lds, mean, rstd, None)


@pytest.mark.parametrize("args,want", [
    (dict(flags=2), X.XPOSE_EINVAL), (dict(q=0), X.XPOSE_EINVAL), (dict(scale=0), X.XPOSE_EINVAL),
    (dict(lds=19), X.XPOSE_EINVAL), (dict(ldq=300), X.XPOSE_EALIGN), (dict(q=C + 4), X.XPOSE_EALIGN),
    (dict(q=A), X.XPOSE_EALIAS), (dict(scale=C), X.XPOSE_EALIAS), (dict(rows=0, lds=1), X.XPOSE_OK),
])
def test_norm_quantize_refusals(args, want):
    assert norm_q(**args) == want


def backward(rows=20, cols=300, dy=A, lddy=300, x=B, ldx=300, dtype=X.XPOSE_F32, mean=SA, rstd=SB, w=Q,
             pd=X.XPOSE_F32, dx=C, lddx=300, dw=QT, db=QT + (1 << 20), ws=WS, size=1 << 30):
    return lib.xpose_layer_norm_backward(rows, cols, dy, lddy, x, ldx, dtype, mean, rstd, w, pd, dx, lddx,
                                         dw, db, ws, size, None)


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), X.XPOSE_EINVAL), (dict(dy=0), X.XPOSE_EINVAL), (dict(x=0), X.XPOSE_EINVAL),
    (dict(mean=0), X.XPOSE_EINVAL), (dict(rstd=0), X.XPOSE_EINVAL), (dict(dx=0), X.XPOSE_EINVAL),
    (dict(lddy=1), X.XPOSE_EINVAL), (dict(size=-1), X.XPOSE_EINVAL), (dict(dtype=X.XPOSE_F64), X.XPOSE_EDTYPE),
    (dict(dx=C + 2), X.XPOSE_EALIGN), (dict(dx=B), X.XPOSE_EALIAS), (dict(dx=A, lddx=301), X.XPOSE_EALIAS),
    (dict(dw=C), X.XPOSE_EALIAS), (dict(db=QT), X.XPOSE_EALIAS), (dict(ws=C), X.XPOSE_EALIAS),
    (dict(ws=0), X.XPOSE_EWORKSPACE), (dict(size=100), X.XPOSE_EWORKSPACE), (dict(cols=0), X.XPOSE_OK),
])
def test_backward_refusals(args, want):
    assert backward(**args) == want


def test_backward_workspace():
    size = ctypes.c_int64()
    assert lib.xpose_layer_norm_backward_workspace(0, 100, ctypes.byref(size)) == X.XPOSE_OK and size.value == 0
    assert lib.xpose_layer_norm_backward_workspace(1, 100, ctypes.byref(size)) == X.XPOSE_OK
    assert size.value == 800
    assert lib.xpose_layer_norm_backward_workspace(-1, 1, ctypes.byref(size)) == X.XPOSE_EINVAL
    assert lib.xpose_layer_norm_backward_workspace(1, 1, None) == X.XPOSE_EINVAL
    assert lib.xpose_layer_norm_backward_workspace(1 << 30, 1 << 61, ctypes.byref(size)) == X.XPOSE_EINVAL


# ----- clipping ------------------------------------------------------------------------

def clip(entries, max_norm=1.0, eps=1e-6, norm=C, ws=WS, size=1 << 20):
    table = (L.XposeClipTensor * max(1, len(entries)))(*[L.XposeClipTensor(*e) for e in entries])
    return lib.xpose_clip_grad_norm(len(entries), table, max_norm, eps, norm, ws, size, None)


F32 = X.XPOSE_F32


@pytest.mark.parametrize("entries,more,want", [
    ([(A, B, -1, F32, 0)], {}, X.XPOSE_EINVAL), ([(0, B, 1, F32, 0)], {}, X.XPOSE_EINVAL),
    ([(A, 0, 1, F32, 0)], {}, X.XPOSE_EINVAL), ([(A, B, 1, F32, 1)], {}, X.XPOSE_EINVAL),
    ([(A, B, 1 << 62, F32, 0)], {}, X.XPOSE_EINVAL), ([(A, B, 1, X.XPOSE_U8, 0)], {}, X.XPOSE_EDTYPE),
    ([(A, B, 1, F32, 0)], dict(max_norm=-1.0), X.XPOSE_EINVAL),
    ([(A, B, 1, F32, 0)], dict(max_norm=float("nan")), X.XPOSE_EINVAL),
    ([(A, B, 1, F32, 0)], dict(eps=-1.0), X.XPOSE_EINVAL), ([(A, B, 1, F32, 0)], dict(norm=0), X.XPOSE_EINVAL),
    ([(A + 2, B, 1, F32, 0)], {}, X.XPOSE_EALIGN), ([(A, B, 1, F32, 0)], dict(ws=WS + 4), X.XPOSE_EALIGN),
    ([(A, A + 4, 2, F32, 0)], {}, X.XPOSE_EALIAS), ([(A, B, 4, F32, 0), (B + 8, Q, 1, F32, 0)], {}, X.XPOSE_EALIAS),
    ([(A, A, 4, F32, 0), (B, A + 8, 4, F32, 0)], {}, X.XPOSE_EALIAS),
    ([(A, B, 1, F32, 0)], dict(norm=B), X.XPOSE_EALIAS), ([(A, B, 1, F32, 0)], dict(ws=A), X.XPOSE_EALIAS),
    # an input inside another input is fine, so an output further on in the longer one must still be found
    ([(A, B, 100, F32, 0), (A + 8, Q, 1, F32, 0), (QT, A + 200, 1, F32, 0)], {}, X.XPOSE_EALIAS),
    ([(A, B, 1, F32, 0)], dict(ws=0), X.XPOSE_EWORKSPACE), ([(A, B, 1, F32, 0)], dict(size=4), X.XPOSE_EWORKSPACE),
])
def test_clip_refusals(entries, more, want):
    assert clip(entries, **more) == want


def test_clip_workspace():
    size = ctypes.c_int64()
    ask = lambda n, t: lib.xpose_clip_grad_norm_workspace(n, t, ctypes.byref(size))  # noqa: E731
    assert ask(0, None) == X.XPOSE_OK and size.value == 0
    assert ask(1, None) == X.XPOSE_EINVAL
    many = (L.XposeClipTensor * 300)(*[L.XposeClipTensor(A, B, 1, F32, 0)] * 300)
    assert ask(300, many) == X.XPOSE_OK and size.value == 8 * 300
    many[0].count = 1 << 40
    assert ask(300, many) == X.XPOSE_OK and 0 < size.value <= 8 * 4 * 2048
    assert ask(-1, many) == X.XPOSE_EINVAL


# ----- the binding's own checks -----------------------------------------------------------

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("call", [
    lambda: X.fp8_quantize(torch.zeros(4, 4)),
    lambda: X.layer_norm(torch.zeros(4, 4)),
    lambda: X.layer_norm_quantize(torch.zeros(4, 4)),
    lambda: X.layer_norm_backward(*[torch.zeros(4, 4)] * 2, *[torch.zeros(4)] * 2),
    lambda: X.clip_grad_norm([torch.zeros(4)], 1.0),
    lambda: X.clip_grad_norm([], 1.0),
    lambda: X.fp8_gemm(*[torch.zeros(4, 4)] * 4),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError):
        call()


def test_dense():
    t = torch.zeros(4, 6, 5)
    assert L._dense(t) and L._dense(t.transpose(0, 2)) and L._dense(t[1]) and L._dense(t[:0])
    assert not L._dense(t[:, :3]) and not L._dense(t[..., ::2]) and not L._dense(t[:, 0])
    assert L._dense(torch.zeros(1, 5)[:, :1])
