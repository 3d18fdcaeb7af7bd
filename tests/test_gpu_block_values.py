"""Values at the ends of their types in a residual block's operators: what is
finite in float32 stays finite, numbers that are not there (ranks past the last
one) reach nothing, zeros keep their sign."""
import math

import pytest

from test_gpu_block import BF16, F16, F32, TYPES, _dev
from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

# from the largest bfloat16 to the largest float32: the nearest bfloat16 of all but the first is infinite
LARGE = [3.3895313892515355e38, 3.3961775292304601e38, 3.4e38, 3.4028234663852886e38]


def _full(v, *shape, dtype=F32):
    return torch.full(shape, v, dtype=dtype, device=_dev())


def _f32(v):
    return torch.tensor(v, dtype=F32).item()


@pytest.mark.parametrize("value", [s * v for v in LARGE for s in (1, -1)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rank", [5, 16, 40])
def test_finite_numbers_stay_finite(value, dtype, rank):
    """A scaled hidden, a dh and a hidden of the largest magnitudes next to
    weights and rows of 2^-14: powers of two, so that each product is exact."""
    m, n, k = 20, 130, 200
    value = _f32(value)
    small, want = 2.0 ** -14, value * 2.0 ** -14
    ids = torch.arange(m, dtype=torch.int32, device=_dev()) % 2 - 1
    mine = (ids == 0).cpu()
    one = torch.zeros(m, k, dtype=dtype, device=_dev())
    one[:, 3] = 1
    a, b = torch.zeros(1, rank, k, dtype=dtype, device=_dev()), torch.zeros(1, n, rank, dtype=dtype, device=_dev())
    a[0, rank - 1, 3], b[0, :, rank - 1] = 1, small
    say(f"large values {value} {dtype} {rank}")
    scale = _full(value, 1)
    out = X.adapters(one, a, b, ids, base=_full(0.0, m, n), scale=scale).cpu()
    assert (out[mine] == want).all() and not out[~mine].any()
    # dh = value at the last rank; dx = dh A, da = dh^T x
    a[0, rank - 1], b[0, :, rank - 1] = small, 0
    b[0, 7, rank - 1] = 1
    dout = torch.zeros(m, n, dtype=dtype, device=_dev())
    dout[5, 7] = 1  # a row of the adapter
    x = _full(small, m, k, dtype=dtype)
    hidden = torch.zeros(m, rank, device=_dev())
    dx, da, _ = X.adapters_backward(dout, x, a, b, ids, hidden, base=_full(0.0, m, k), scale=scale)
    assert (dx[5] == want).all() and not dx[:5].any() and not dx[6:].any()
    assert (da[0, rank - 1] == want).all() and not da[0, :rank - 1].any()
    # db = dout^T hidden
    hidden[5, rank - 1] = value
    dout[5, 7] = small
    _, _, db = X.adapters_backward(dout, x, a, b, ids, hidden)
    assert db[0, 7, rank - 1] == want
    db[0, 7, rank - 1] = 0
    assert not db.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_nan_stays_one(dtype):
    """Whatever bits it has: cut off after 16 of them the first one is an infinity."""
    hidden = torch.zeros(3, 16, device=_dev())
    hidden[0, 2] = torch.tensor([0x7f800001], dtype=torch.int32).view(F32)[0]
    hidden.view(torch.int32)[1, 3] = 0x7f800001
    hidden.view(torch.int32)[2, 4] = -0x7fffff
    assert hidden.isnan().sum() == 3
    ones = lambda *s: _full(1.0, *s, dtype=dtype)  # noqa: E731
    _, _, db = X.adapters_backward(ones(3, 40), ones(3, 50), ones(1, 16, 50), ones(1, 40, 16),
                                   torch.zeros(3, dtype=torch.int32, device=_dev()), hidden)
    assert db[0, :, 2:5].isnan().all() and not db[0, :, :2].any() and not db[0, :, 5:].any()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_all_bits_of_hidden(dtype):
    """Numbers of 24 bits next to ones: the sum of the parts is the number."""
    gen = torch.Generator(device=_dev()).manual_seed(1)
    r = lambda: torch.rand(4000, 16, generator=gen, device=_dev())  # noqa: E731
    hidden = (1 + r()) * torch.exp2(160 * r() - 80) * (1 - 2 * (r() < 0.5).float())  # each part in bfloat16's range
    ids = torch.arange(4000, dtype=torch.int32, device=_dev())  # a row each, so no sums
    one = _full(1.0, 4000, 8, dtype=dtype)
    _, _, db = X.adapters_backward(one, one, _full(0.0, 1, 16, 8, dtype=dtype).expand(4000, 16, 8),
                                   _full(0.0, 1, 8, 16, dtype=dtype).expand(4000, 8, 16), ids, hidden)
    assert torch.equal(db, hidden[:, None].expand(4000, 8, 16))


@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rank", [1, 5, 8, 16, 31, 32, 40, 64])
def test_an_infinite_scale(dtype, out, rank):
    """Infinities of the products' sign, whatever the rank: numbers past the
    last one are not multiplied by it, and other adapters' rows stay.  (float16
    weights are the sum of two numbers, one of them 0 here: a NaN is right too.)"""
    m, n, k = 12, 130, 64
    gen = torch.Generator(device=_dev()).manual_seed(rank)
    ids = torch.arange(m, dtype=torch.int32, device=_dev()) % 3 - 1
    x, a = _full(1.0, m, k, dtype=dtype), _full(0.5, 2, rank, k, dtype=dtype)
    b = torch.where(torch.rand(2, n, 1, generator=gen, device=_dev()) < 0.5, -1.0, 1.0).to(dtype).repeat(1, 1, rank)
    base = torch.randn(m, n, generator=gen, device=_dev()).to(out)
    say(f"infinite scale {dtype} {out} {rank}")
    got = X.adapters(x, a, b, ids, base=base, scale=torch.tensor([1.0, math.inf], device=_dev()))
    want = X.adapters(x, a, b, ids, base=base, scale=torch.tensor([1.0, 1.0], device=_dev()))
    assert torch.equal(got[ids != 1], want[ids != 1])
    if dtype == F16:
        assert not got[ids == 1].isfinite().any()
        return
    assert torch.equal(got[ids == 1].float(), (b[1, :, 0].float() * math.inf).expand(int((ids == 1).sum()), n))


@pytest.mark.parametrize("dtype", TYPES)
def test_dropped_elements_are_the_residual(dtype):
    """Bit for bit: a zero of it keeps its sign."""
    x = torch.randn(50, 300, device=_dev()).to(dtype)
    res = torch.where(torch.rand(50, 300, device=_dev()) < 0.5, -0.0, 0.0).to(dtype)
    keep = X.dropout(torch.ones_like(x), 0.5, 3) != 0
    y = X.dropout(x, 0.5, 3, residual=res)
    assert not keep.all() and torch.equal(y.signbit()[~keep], res.signbit()[~keep]) and not y[~keep].any()
    assert torch.equal(X.dropout(x, 1.0, 3, residual=res).signbit(), res.signbit())
    assert not X.dropout(-x.abs(), 1.0, 3).signbit().any()  # zeros without one


@pytest.mark.parametrize("call", [
    lambda z, i: X.adapters(z(4, 8), z(2, 3, 8), z(2, 5, 3), i(4), scale="1"),
    lambda z, i: X.adapters(z(4, 8), z(2, 3, 8), z(2, 5, 3), i(4), scale=None),
    lambda z, i: X.adapters(z(4, 8), z(2, 3, 8), z(2, 5, 3), i(4), scale=[1.0, 2.0]),
    lambda z, i: X.adapters_backward(z(4, 5), z(4, 8), z(2, 3, 8), z(2, 5, 3), i(4), z(4, 3), scale=(1.0,)),
    lambda z, i: X.dropout(z(4, 4), 0.5, 1.5),
    lambda z, i: X.dropout(z(4, 4), 0.5, None),
    lambda z, i: X.dropout(z(4, 4), 0.5, "1"),
])
def test_numbers_of_another_type(call):
    with pytest.raises(TypeError):
        call(lambda *s: torch.zeros(*s, device=_dev()), lambda m: torch.zeros(m, dtype=torch.int32, device=_dev()))


@pytest.mark.parametrize("cols", [5, 100, 3000, 20000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_squares_outside_float32(cols, dtype):
    """Over it rstd is 0; under it infinite with eps 0, and eps's with one."""
    x = torch.stack([_full(v, cols, dtype=dtype) for v in (1e30, 1e-30, 0.0, 1.0)])
    y, rstd = X.rms_norm(x, eps=0.0, stats=True)
    assert rstd.tolist() == [0.0, float("inf"), float("inf"), 1.0]
    assert not y[0].any() and y[1].isinf().all() and y[2].isnan().all() and (y[3] == 1).all()
    y, rstd = X.rms_norm(x, eps=0.25, stats=True)
    assert rstd[:3].tolist() == [0.0, 2.0, 2.0] and not y[0].any() and torch.equal(y[1], x[1] * 2) and not y[2].any()
