"""Layer norm and its backward pass where a row's end, a large mean or the
number of rows could show through."""
import numpy as np
import pytest

from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U32 = 2.0 ** -24


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


@pytest.mark.parametrize("cols", [1, 7, 100, 200, 300, 700, 1500, 2999, 5001, 8201, 10003])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("weighted", [False, True])
def test_backward_of_a_row_far_from_zero(cols, dtype, weighted):
    """Rows of one value, x - mean = 0, whose mean times rstd is over float32:
    what is not there has no x of 0 to be that far away."""
    rng = np.random.default_rng(cols)
    rows, far, rstd = 5, 2.0 ** 100, 2.0 ** 40
    x = torch.full((rows, cols), far).to(dtype).to(_dev())
    x[3] = 0
    mean = torch.full((rows,), far).to(_dev())
    mean[3] = 0
    dy = torch.from_numpy(rng.standard_normal((rows, cols))).to(dtype)
    w = torch.from_numpy(rng.standard_normal(cols)).float() if weighted else None
    say(f"far mean {cols} {dtype} {weighted}")
    got = X.layer_norm_backward(dy.to(_dev()), x, mean, torch.full((rows,), rstd).to(_dev()),
                                w.to(_dev()) if weighted else None)
    g = dy.double().numpy() * (w.double().numpy() if weighted else 1)
    want = (g - g.mean(1, keepdims=True)) * rstd
    # a product, a sum of cols terms and its division, a difference and a product, and the result's rounding
    tol = ((cols + 4) * U32 * np.abs(g).mean(1, keepdims=True) + 3 * U32 * np.abs(g)) * rstd * 1.01 \
        + torch.finfo(dtype).eps / 2 * np.abs(want) * 1.01
    assert (np.abs(got[0].cpu().double().numpy() - want) <= tol).all()
    assert not got[1].any()
    s = dy.double().numpy()
    assert (np.abs(got[2].cpu().double().numpy() - s.sum(0)) <= rows * U32 * np.abs(s).sum(0)).all()
