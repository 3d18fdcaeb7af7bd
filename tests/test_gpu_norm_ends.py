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


MANY = (1 << 22) + 3  # rows: of a workgroup of 1024 threads each, more than a launch has


def test_more_rows_than_a_launch_of_workgroups():
    """Rows of a few columns, of which a workgroup then takes several."""
    cols = 4
    gen = torch.Generator(device=_dev()).manual_seed(1)
    x = torch.randn(MANY, cols, generator=gen, device=_dev())
    dy = torch.randn(MANY, cols, generator=gen, device=_dev())
    w, b = torch.randn(cols, generator=gen, device=_dev()), torch.randn(cols, generator=gen, device=_dev())
    say("many rows, forward")
    y, mean, rstd = X.layer_norm(x, w, b, stats=True)
    # rows that a launch of their own takes have the same bits
    for part in (slice(0, 1000), slice(MANY - 1000, MANY)):
        for got, want in zip((y, mean, rstd), X.layer_norm(x[part], w, b, stats=True)):
            assert torch.equal(got[part], want)
    xd = x.double()
    m = xd.mean(1)
    r = 1 / ((xd - m[:, None]).square().mean(1) + 1e-5).sqrt()
    # four terms and their division; the mean's error in the variance, twice
    assert ((mean - m).abs() <= 5 * U32 * xd.abs().mean(1)).all()
    assert ((rstd - r).abs() <= r * (12 * U32 + r.square() * 20 * U32 * xd.square().mean(1))).all()
    say("many rows, quantised")
    q, s = X.layer_norm_quantize(x, w, b)
    for part in (slice(0, 1000), slice(MANY - 1000, MANY)):
        q1, s1 = X.layer_norm_quantize(x[part], w, b)
        assert torch.equal(q[part].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, part], s1)
    scale = (y.abs().amax(1) / torch.full((MANY,), 448.0, device=_dev())).clamp(min=2.0 ** -126)
    assert torch.equal(s[0], scale)
    assert torch.equal(q.float(), (y / scale[:, None]).to(torch.float8_e4m3fn).float())
    del q, s, scale, xd
    say("many rows, backward")
    dx, dw, db = X.layer_norm_backward(dy, x, mean, rstd, w)
    xhat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy.double() * w.double()
    want = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd.double()[:, None]
    size = (g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True)) \
        * rstd.double()[:, None]
    assert ((dx - want).abs() <= 16 * U32 * size).all()
    terms = 16384 + 600  # a workgroup's rows and the workgroups
    assert ((dw - (dy * xhat).sum(0)).abs() <= terms * U32 * (dy * xhat).abs().sum(0)).all()
    assert ((db - dy.double().sum(0)).abs() <= terms * U32 * dy.double().abs().sum(0)).all()


def test_more_columns_than_a_launch_of_parameter_sums():
    """One row of over 2^28 columns: its gradients of weight and bias are a
    product each, and dy itself."""
    cols = (1 << 28) + 100
    gen = torch.Generator(device=_dev()).manual_seed(2)
    x = torch.randn(1, cols, generator=gen, device=_dev())
    dy = torch.randn(1, cols, generator=gen, device=_dev())
    mean, rstd = torch.full((1,), 0.25, device=_dev()), torch.full((1,), 1.5, device=_dev())
    say("many columns")
    _, dw, db = X.layer_norm_backward(dy, x, mean, rstd)
    assert torch.equal(db, dy[0])
    assert torch.equal(dw, dy[0] * ((x[0] - 0.25) * 1.5))
