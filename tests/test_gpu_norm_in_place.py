"""Layer norm over x itself and its backward pass over dy itself, with more rows
than run at once, so that later rows are loaded beside earlier ones' stores:
the same bits as into tensors of their own."""
import ctypes

import pytest

from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")
L = pytest.importorskip("lds_tiled_matrix_amd.linear")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODE = {F32: X.XPOSE_F32, F16: X.XPOSE_F16, BF16: X.XPOSE_BF16}

# every split of a row over lanes: less than a load, a quarter wave, a wave, a
# workgroup, three chunks a lane, three sweeps
SIZES = [(50000, 5), (100000, 100), (60000, 250), (20003, 510), (20000, 900), (5200, 1500), (9000, 2001), (5000, 2900),
         (5000, 4000), (1700, 5500), (3000, 6789), (2000, 9000), (1500, 16001), (600, 20000)]


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


def _matrix(rows, cols, dtype, pad, seed):
    """A matrix of pitch cols + pad and what lies around it, of a value of its own."""
    gen = torch.Generator(device=_dev()).manual_seed(seed)
    store = torch.full((rows, cols + pad), 77.0, dtype=dtype, device=_dev())
    view = store[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen, device=_dev()))
    return store, view


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 3])
def test_layer_norm_over_its_input(rows, cols, dtype, pad):
    store, x = _matrix(rows, cols, dtype, pad, cols)
    w, b = torch.randn(cols, device=_dev()), torch.randn(cols, device=_dev())
    say(f"in place {rows} {cols} {dtype} {pad}")
    want = X.layer_norm(x, w, b, stats=True)
    got = X.layer_norm(x, w, b, stats=True, out=x)
    assert got[0] is x
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    assert not pad or (store[:, cols:] == 77).all()


def _backward(rows, cols, dtype, dy, lddy, x, ldx, mean, rstd, w, dx, lddx):
    size = ctypes.c_int64()
    assert L._lib.xpose_layer_norm_backward_workspace(rows, cols, ctypes.byref(size)) == X.XPOSE_OK
    ws = torch.empty(max(1, size.value), dtype=torch.uint8, device=_dev())
    dw, db = torch.empty(cols, device=_dev()), torch.empty(cols, device=_dev())
    rc = L._lib.xpose_layer_norm_backward(rows, cols, dy.data_ptr(), lddy, x.data_ptr(), ldx, CODE[dtype],
                                          mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), X.XPOSE_F32, dx.data_ptr(),
                                          lddx, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), size.value,
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == X.XPOSE_OK
    torch.cuda.synchronize()
    return dw, db


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 3])
def test_backward_over_its_dy(rows, cols, dtype, pad):
    _, x = _matrix(rows, cols, dtype, 0, cols)
    store, dy = _matrix(rows, cols, dtype, pad, cols + 1)
    w = torch.randn(cols, device=_dev())
    _, mean, rstd = X.layer_norm(x, w, stats=True)
    say(f"backward in place {rows} {cols} {dtype} {pad}")
    dx, dw, db = X.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    got = _backward(rows, cols, dtype, dy, cols + pad, x, cols, mean, rstd, w, dy, cols + pad)
    assert torch.equal(dy, dx) and torch.equal(got[0], dw) and torch.equal(got[1], db)
    assert not pad or (store[:, cols:] == 77).all()
