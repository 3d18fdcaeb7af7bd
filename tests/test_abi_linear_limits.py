"""Sizes at the limits of a launch (2^32 - 1 threads): plans stay under them and
what cannot be launched is refused before the GPU is asked (addresses here are
made up and never dereferenced)."""
import ctypes

import pytest

import lds_tiled_matrix_amd as X
from lds_tiled_matrix_amd import linear as L

lib = L._lib
A, B, C, SA, SB, WS, Q, QT = (0x7f0000000000 + (i << 44) for i in range(8))
MAX_THREADS = (1 << 32) - 1


def plan(m, n, k, out):
    info = L.XposeFp8GemmInfo()
    return lib.xpose_fp8_gemm_plan(m, n, k, 1, out, 0, ctypes.byref(info)), info


@pytest.mark.parametrize("out", [X.XPOSE_BF16, X.XPOSE_F32])
@pytest.mark.parametrize("k", [0, 16, 1000, 100000])
@pytest.mark.parametrize("m", [1, 16, 30, 60, 128, 200, 5000, 1 << 16, 1 << 20])
@pytest.mark.parametrize("n", [(1 << 20) + 1, (1 << 26) + 5, 1 << 27, (1 << 27) + 1, (1 << 30) + 3, (1 << 31) - 129,
                               1 << 31, 1 << 34])
def test_gemm_plans_are_launches_that_exist(m, n, k, out):
    rc, info = plan(m, n, k, out)
    if -(-m // 128) * -(-n // 128) < 1 << 24:
        assert rc == X.XPOSE_OK
    if rc == X.XPOSE_OK:
        assert info.workgroups * info.threads <= MAX_THREADS
    else:
        assert rc == X.XPOSE_EINVAL


def test_gemm_past_a_launch():
    assert plan(1, 1 << 34, 16, X.XPOSE_BF16)[0] == X.XPOSE_EINVAL
    assert plan(1, 1 << 31, 16, X.XPOSE_F32)[0] == X.XPOSE_EINVAL
    n = 1 << 31
    assert lib.xpose_fp8_gemm(1, n, 16, A, 16, SA, 1, B, 16, SB, n, 1, C, n, X.XPOSE_F32, 0, WS, 0, None) \
        == X.XPOSE_EINVAL


@pytest.mark.parametrize("rows,cols", [(1 << 31, 1), (1, 1 << 31), (1 << 19, 1 << 19), ((1 << 31) - 127, 100)])
def test_quantize_past_a_launch(rows, cols):
    tiles_r, tiles_c = -(-rows // 128), -(-cols // 128)
    up = lambda v: -(-v // 8) * 8  # noqa: E731
    assert lib.xpose_fp8_quantize(rows, cols, A, cols, X.XPOSE_BF16, 128, 0, Q, up(cols), SA, tiles_r, QT, up(rows),
                                  SB, tiles_c, None) == X.XPOSE_EINVAL


def test_backward_past_a_launch():
    rows, cols = 256, 1 << 28
    assert lib.xpose_layer_norm_backward(rows, cols, A, cols, B, cols, X.XPOSE_BF16, SA, SB, None, X.XPOSE_F32, C,
                                         cols, QT, QT + 4 * cols, WS, 1 << 42, None) == X.XPOSE_EINVAL
