"""The FP8 linear layer's operators on the GPU against the float64 oracle.

Tolerances.  u(t) = eps(t) / 2 is the relative error of one rounding to t.
A sum of n terms in float32 is within n u of the sum of magnitudes whatever
its order; the matrix cores' own additions may cut bits off instead of
rounding them, twice that.  Quantised values have to be equal: their
definition has no freedom."""
import math

import numpy as np
import pytest

import oracle.linear as ol
from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U32 = 2.0 ** -24


def u(dtype):
    return torch.finfo(dtype).eps / 2


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


def _np(t):
    return t.detach().cpu().double().numpy()


def _bytes(q):
    return q.cpu().contiguous().view(torch.uint8).numpy()


def _close(got, want, tol, what):
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(off / np.maximum(tol, 1e-300))))


def _strided(x, pad, fill=float("nan")):
    """x on the GPU as a view into a wider matrix of `fill`."""
    rows, cols = x.shape
    store = torch.full((rows, cols + pad), fill, dtype=x.dtype, device=_dev())
    view = store[:, pad // 2:pad // 2 + cols] if pad else store
    view.copy_(x)
    return view


# ----- matrix product -------------------------------------------------------------

def _e4m3(bits, pad_bytes=0x7f):
    """Bytes on the GPU with rows at multiples of 16 and NaN between."""
    rows, cols = bits.shape
    pitch = -(-max(cols, 1) // 16) * 16 + 16
    store = torch.full((rows, pitch), pad_bytes, dtype=torch.uint8, device=_dev())
    store[:, :cols] = torch.from_numpy(bits).to(_dev())
    return store.view(torch.float8_e4m3fn)[:, :cols]


def _operands(m, n, k, block_rows, pow2, seed):
    rng = np.random.default_rng(seed)
    a = rng.standard_normal((m, k)) * np.exp(rng.uniform(-3, 3, (m, 1)))
    b = rng.standard_normal((n, k)) * 0.02
    if m > 2:
        a[1] = 0
    return ol.quantize(a, 1, pow2) + ol.quantize(b, block_rows, pow2)


def _gemm(qa, sa, qb, sb, dtype, pow2, **more):
    up = lambda s: torch.from_numpy(s).to(_dev())  # noqa: E731
    return X.fp8_gemm(_e4m3(qa), up(sa), _e4m3(qb), up(sb), out_dtype=dtype, pow2=pow2, **more)


SIZES = [(1, 1, 1), (1, 16, 16), (1, 4096, 512), (3, 17, 129), (16, 100, 1000), (17, 33, 128), (33, 70, 300),
         (64, 257, 640), (65, 64, 64), (100, 130, 127), (128, 128, 128), (200, 300, 777), (129, 1, 256),
         (255, 257, 384), (300, 500, 4096), (1000, 129, 2222)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_gemm(m, n, k, block_rows, pow2):
    say(f"gemm {m} {n} {k} rows {block_rows} pow2 {pow2}")
    ops = _operands(m, n, k, block_rows, pow2, m + 7 * n + k)
    want, mag = ol.gemm(*ops, block_rows)
    for dtype in (F32, F16, BF16):
        got = _np(_gemm(*ops, dtype, pow2))
        # k products in sums that may cut, a scaling and an addition a block
        tol = (2 * k + 4) * U32 * mag + u(dtype) * np.abs(want)
        if dtype != F32:
            # each of 8 neighbouring products cut under 2^-13 of the largest
            # one's leading bit: 8 * 2^-13 of the largest
            tol = tol + 2.0 ** -10 * mag
        tol = tol * (1 + u(dtype)) + (2.0 ** -25 if dtype == F16 else 0)  # half of fp16's last step at 0
        _close(got, want, tol, dtype)


@pytest.mark.parametrize("m,n,k", [(3, 200, 8200), (24, 90, 7360), (60, 33, 9001)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_gemm_few_rows_in_slices(m, n, k, block_rows):
    info = X.fp8_gemm_plan(m, n, k, block_rows=block_rows)
    assert info["tile_n"] == 16 and info["splits"] > 1
    test_gemm(m, n, k, block_rows, False)


@pytest.mark.parametrize("m,n,k,block_rows,pow2", [
    (4000, 4090, 400, 128, False), (3850, 4096, 400, 1, False), (4096, 3999, 400, 128, True),
    (3901, 4090, 390, 1, True), (4000, 4090, 512, 1, False)])
def test_gemm_large_tiles(m, n, k, block_rows, pow2):
    """Enough tiles of 256 x 256 for those to be taken, with ragged edges."""
    assert X.fp8_gemm_plan(m, n, k, block_rows=block_rows)["tile_m"] == 256
    test_gemm(m, n, k, block_rows, pow2)


@pytest.mark.parametrize("m,n,k", [(5, 40, 300), (100, 200, 1500), (2048, 5130, 200)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_gemm_is_exact_on_small_integers(m, n, k, block_rows, pow2):
    """Integers times powers of two: every partial sum is a float32, so any
    wrong index shows as a wrong number."""
    rng = np.random.default_rng(k)
    ints = lambda r: ol.e4m3_encode(rng.integers(-8, 9, (r, k)).astype(np.float32))  # noqa: E731
    scales = lambda c: (2.0 ** rng.integers(-2, 3, (-(-k // 128), c))).astype(np.float32)  # noqa: E731
    ops = ints(m), scales(m), ints(n), scales(n if block_rows == 1 else -(-n // 128))
    say(f"gemm integers {m} {n} {k} {block_rows} {pow2}")
    got = _np(_gemm(*ops, F32, pow2))
    want = ol.gemm(*ops, block_rows)[0]
    assert np.array_equal(got, want)
    # products of up to 2^6 in whole steps: nothing to cut
    for dtype in (F16, BF16):
        assert np.array_equal(_np(_gemm(*ops, dtype, pow2)), _np(torch.from_numpy(want).to(dtype)))


def test_gemm_splits_of_k_and_their_sum():
    info = X.fp8_gemm_plan(300, 500, 8200, out_dtype=F32)
    assert info["splits"] > 1
    test_gemm(300, 500, 8200, 1, False)
    ops = _operands(300, 500, 8200, 1, False, 3)
    first = _gemm(*ops, F32, False)
    for _ in range(3):
        assert torch.equal(first, _gemm(*ops, F32, False))


@pytest.mark.parametrize("m,n,k", [(3, 50, 400), (150, 200, 400)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gemm_special_values(m, n, k, pow2):
    """NaN elements, and scales of inf and NaN, reach the outputs that use them
    and no others."""
    qa, sa, qb, sb = _operands(m, n, k, 1, pow2, 5)
    qa[2, 130] = 0x7f
    sb[1, 7] = np.inf
    sb[0, 9] = np.nan
    say(f"gemm special {m} {n} {k} {pow2}")
    got = _np(_gemm(qa, sa, qb, sb, F32, pow2))
    bad = np.zeros((m, n), bool)
    bad[2] = True
    bad[:, 9] = True
    assert np.isnan(got[bad]).all()
    rest = ~bad
    rest[:, 7] = False
    assert np.isfinite(got[rest]).all()
    assert not np.isfinite(got[[i for i in range(m) if i != 1], 7]).any()


def test_gemm_no_columns_to_sum_and_empty():
    dev = _dev()
    e = lambda r, c: torch.zeros((r, c), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)  # noqa: E731
    s = lambda r, c: torch.zeros((r, c), device=dev)  # noqa: E731
    for m in (3, 100):
        out = torch.full((m, 20), 7.0, device=dev)
        X.fp8_gemm(e(m, 0), s(0, m), e(20, 0), s(0, 20), out=out)
        assert not out.any()
    assert X.fp8_gemm(e(0, 64), s(1, 0), e(20, 64), s(1, 20)).shape == (0, 20)
    assert X.fp8_gemm(e(4, 64), s(1, 4), e(0, 64), s(1, 0)).shape == (4, 0)


@pytest.mark.parametrize("m", [5, 200, 2048])
def test_gemm_writes_its_region_alone(m):
    n, k = 5003 if m == 2048 else 203, 256
    ops = _operands(m, n, k, 128, False, 9)
    store = torch.full((m, n + 9), -5.0, dtype=BF16, device=_dev())
    _gemm(*ops, BF16, False, out=store[:, 3:3 + n])
    assert torch.equal(store[:, 3:3 + n], _gemm(*ops, BF16, False))
    assert (store[:, :3] == -5).all() and (store[:, 3 + n:] == -5).all()


def test_gemm_rows_past_32_bits():
    """b's last rows start over 2^32 bytes into their buffer."""
    n, k, pitch = 520, 256, (1 << 23) - 16
    rng = np.random.default_rng(11)
    store = torch.zeros(n * pitch, dtype=torch.uint8, device=_dev())
    b = ol.quantize(rng.standard_normal((n, k)))
    view = torch.as_strided(store, (n, k), (pitch, 1))
    view.copy_(torch.from_numpy(b[0]))
    for m in (4, 90):
        a = ol.quantize(rng.standard_normal((m, k)))
        say(f"gemm far rows m {m}")
        got = X.fp8_gemm(_e4m3(a[0]), torch.from_numpy(a[1]).to(_dev()), view.view(torch.float8_e4m3fn),
                         torch.from_numpy(b[1]).to(_dev()), out_dtype=F32)
        assert torch.equal(got, _gemm(*a, *b, F32, False))


# ----- quantisation -----------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (3, 7), (128, 128), (130, 257), (1000, 129), (127, 640),
                                       (129, 2048)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize(rows, cols, dtype, block_rows, pow2):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-6, 3, (rows, 1)))
    if rows > 2:
        x[1] = 0
    x = torch.from_numpy(x).to(dtype)
    say(f"quantize {rows} {cols} {dtype} {block_rows} {pow2}")
    for pad in (0, 5, 8):
        v = _strided(x, pad)
        q, s, qt, st = X.fp8_quantize(v, block_rows=block_rows, pow2=pow2, transposed=True)
        for got, scale, of in ((q, s, x), (qt, st, x.t())):
            wq, ws = ol.quantize(of.float().numpy(), block_rows, pow2)
            assert np.array_equal(scale.cpu().numpy(), ws)
            assert np.array_equal(_bytes(got), wq)
        q1, s1 = X.fp8_quantize(v, block_rows=block_rows, pow2=pow2)
        assert np.array_equal(_bytes(q1), _bytes(q)) and torch.equal(s1, s)


@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_over_the_whole_range(pow2):
    """Every size of block maximum down to the least float32, and quotients on
    and next to the borders between e4m3 values."""
    rng = np.random.default_rng(21)
    rows = 600
    x = rng.uniform(-1, 1, (rows, 256))
    amax = np.ldexp(rng.uniform(1, 2, rows), rng.integers(-149, 127, rows))
    x[:, 0] = 1
    x[:, 128] = 1
    x = (x * amax[:, None]).astype(np.float32)
    # ties: 448 s (j + 1/2) / 16 for a scale s of few bits, nudged by one step
    s = np.float32(1.0) if pow2 else np.float32(1.37)
    ties = (np.arange(16, 31) + 0.5) / 2 * s
    for r, step in ((0, 0), (1, 1), (2, -1)):
        t = ties.astype(np.float32)
        t = np.nextafter(t, np.float32(np.inf * step)) if step else t
        x[r, :] = 0
        x[r, 1:16] = t
        x[r, 0] = np.float32(448) * s
    say("quantize range")
    for block_rows in (1, 128):
        q, sc, qt, st = X.fp8_quantize(torch.from_numpy(x).to(_dev()), block_rows=block_rows, pow2=pow2,
                                       transposed=True)
        for got, scale, of in ((q, sc, x), (qt, st, np.ascontiguousarray(x.T))):
            wq, ws = ol.quantize(of, block_rows, pow2)
            assert np.array_equal(scale.cpu().numpy(), ws)
            assert np.array_equal(_bytes(got), wq)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_special_values(block_rows, pow2):
    x = np.ones((256, 256), np.float32)
    x[5, 3] = np.inf
    x[200, 130] = np.nan
    x[7, 9] = -0.0
    say(f"quantize special {block_rows} {pow2}")
    q, s, qt, st = X.fp8_quantize(torch.from_numpy(x).to(_dev()), block_rows=block_rows, pow2=pow2, transposed=True)
    for got, scale, of in ((q, s, x), (qt, st, np.ascontiguousarray(x.T))):
        wq, ws = ol.quantize(of, block_rows, pow2)
        assert np.array_equal(scale.cpu().numpy(), ws, equal_nan=True)
        assert np.array_equal(ol.e4m3_decode(_bytes(got)), ol.e4m3_decode(wq), equal_nan=True)


def test_quantize_empty():
    for rows, cols in ((0, 5), (5, 0)):
        q, s, qt, st = X.fp8_quantize(torch.zeros(rows, cols, device=_dev()), transposed=True)
        assert q.shape == (rows, cols) and qt.shape == (cols, rows)
        assert s.shape == (-(-cols // 128), rows) and st.shape == (-(-rows // 128), cols)


# ----- layer norm ----------------------------------------------------------------------

COLS = [1, 7, 8, 100, 512, 513, 1024, 1500, 2048, 2999, 4096, 5000, 8192, 10001, 16384, 20000]


def _norm_inputs(rows, cols, dtype, seed, params=F32):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2 + 0.5
    if rows > 2:
        x[2] = 0.75  # no variance
    w, b = 1 + 0.1 * rng.standard_normal(cols), 0.1 * rng.standard_normal(cols)
    return (torch.from_numpy(x).to(dtype), torch.from_numpy(w).to(params), torch.from_numpy(b).to(params))


def _terms(cols):
    """The longest chain of additions behind a row's sum, roundings of the
    terms included: a lane's columns, the lanes of a wave, the waves."""
    return 32 + cols // 1024 + 6 + 16


def _norm_tol(x, w, b, y, rstd, dtype):
    d = _terms(x.shape[1]) * U32
    centred = np.abs(x - x.mean(1, keepdims=True))
    mean_off = d * np.abs(x).mean(1, keepdims=True) + U32 * np.abs(x)
    xhat = centred * rstd[:, None]
    # the variance's own error, from its sum and from the mean
    rel = d + mean_off.max(1, keepdims=True) * (centred * rstd[:, None] ** 2).mean(1, keepdims=True) * 2 + 4 * U32
    return (np.abs(w) * (mean_off * rstd[:, None] + xhat * (rel + 4 * U32)) + U32 * (np.abs(y) + np.abs(b))) \
        * 1.01 + u(dtype) * np.abs(y) + (2.0 ** -25 if dtype == F16 else 0)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_layer_norm(cols, dtype):
    x, w, b = _norm_inputs(6, cols, dtype, cols)
    say(f"layer_norm {cols} {dtype}")
    xd, wd, bd = x.double().numpy(), w.double().numpy(), b.double().numpy()
    want, mean, rstd = ol.layer_norm(xd, wd, bd, 1e-5)
    tol = _norm_tol(xd, wd, bd, want, rstd, dtype)
    for pad in (0, 3, 8):
        v = _strided(x, pad)
        y, m, r = X.layer_norm(v, w.to(_dev()), b.to(_dev()), stats=True)
        _close(_np(y), want, tol, ("y", pad))
        mean_tol = (_terms(cols) + 2) * U32 * np.abs(xd).mean(1)
        _close(_np(m), mean, mean_tol, "mean")
        var_off = 2 * (mean_tol + U32 * np.abs(xd).max(1)) * np.abs(xd - mean[:, None]).mean(1) \
            + (mean_tol + U32 * np.abs(xd).max(1)) ** 2
        _close(_np(r), rstd, rstd * ((_terms(cols) + 4) * U32 + rstd ** 2 * var_off), "rstd")
        assert torch.equal(X.layer_norm(v, w.to(_dev()), b.to(_dev())), y)


@pytest.mark.parametrize("params", [F16, BF16, None])
@pytest.mark.parametrize("cols", [100, 3001, 20000])
def test_layer_norm_parameter_types(cols, params):
    x, w, b = _norm_inputs(5, cols, BF16, cols, params or F32)
    if params is None:
        w, b = torch.ones_like(w), torch.zeros_like(b)
    args = (None, None) if params is None else (w.to(_dev()), b.to(_dev()))
    want = X.layer_norm(x.to(_dev()), w.float().to(_dev()), b.float().to(_dev()), stats=True)
    got = X.layer_norm(x.to(_dev()), *args, stats=True)
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    q = X.layer_norm_quantize(x.to(_dev()), *args)
    p = X.layer_norm_quantize(x.to(_dev()), w.float().to(_dev()), b.float().to(_dev()))
    assert np.array_equal(_bytes(q[0]), _bytes(p[0])) and torch.equal(q[1], p[1])
    g = X.layer_norm_backward(x.to(_dev()), x.to(_dev()), *got[1:], args[0])
    h = X.layer_norm_backward(x.to(_dev()), x.to(_dev()), *got[1:], w.float().to(_dev()))
    assert all(torch.equal(i, j) for i, j in zip(g, h))


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pow2", [False, True])
def test_layer_norm_quantize(cols, dtype, pow2):
    """The float32 result's quantisation: that of the kernel's own float32
    tensor where the input is float32, bit for bit."""
    x, w, b = _norm_inputs(5, cols, dtype, cols)
    say(f"layer_norm_quantize {cols} {dtype} {pow2}")
    for pad in (0, 3):
        v = _strided(x, pad)
        q, s, m, r = X.layer_norm_quantize(v, w.to(_dev()), b.to(_dev()), pow2=pow2, stats=True)
        y, m2, r2 = X.layer_norm(v.float(), w.to(_dev()), b.to(_dev()), stats=True)
        wq, ws = ol.quantize(y.cpu().numpy(), 1, pow2)
        assert torch.equal(m, m2) and torch.equal(r, r2)
        assert np.array_equal(s.cpu().numpy(), ws)
        assert np.array_equal(_bytes(q), wq)


def test_layer_norm_of_many_rows_and_none():
    x, w, b = _norm_inputs(3001, 96, BF16, 4)
    xd = x.double().numpy()
    want, _, rstd = ol.layer_norm(xd, w.double().numpy(), b.double().numpy(), 1e-5)
    y = X.layer_norm(x.to(_dev()), w.to(_dev()), b.to(_dev()))
    _close(_np(y), want, _norm_tol(xd, w.double().numpy(), b.double().numpy(), want, rstd, BF16), "rows")
    e = torch.zeros(0, 96, dtype=BF16, device=_dev())
    assert X.layer_norm(e, w.to(_dev()), b.to(_dev())).shape == (0, 96)
    assert X.layer_norm_quantize(e)[1].shape == (1, 0)
    dx, dw, db = X.layer_norm_backward(e, e, torch.zeros(0, device=_dev()), torch.zeros(0, device=_dev()))
    assert dx.shape == (0, 96) and not dw.any() and not db.any()


def test_layer_norm_in_place_and_special_values():
    x, w, b = _norm_inputs(6, 700, F32, 8)
    v = x.to(_dev())
    want = X.layer_norm(v, w.to(_dev()), b.to(_dev()))
    assert X.layer_norm(v, w.to(_dev()), b.to(_dev()), out=v) is v and torch.equal(v, want)
    x[1, 5], x[3, 699] = math.nan, math.inf
    y = X.layer_norm(x.to(_dev()), w.to(_dev()), b.to(_dev())).cpu()
    assert y[1].isnan().all() and y[3].isnan().all()
    rest = [0, 2, 4, 5]
    assert torch.equal(y[rest], want.cpu()[rest])


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (5, 8), (37, 513), (700, 1000), (9, 1500), (1300, 2048),
                                       (40, 2999), (40, 4096), (30, 5000), (30, 8192), (20, 8193), (21, 20001),
                                       (5000, 64)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_layer_norm_backward(rows, cols, dtype):
    x, w, b = _norm_inputs(rows, cols, dtype, rows + cols)
    rng = np.random.default_rng(cols)
    dy = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))).to(dtype)
    xd, wd, dyd = x.double().numpy(), w.double().numpy(), dy.double().numpy()
    _, mean, rstd = ol.layer_norm(xd, wd, 0.0, 1e-5)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    want = ol.layer_norm_backward(dyd, xd, mean.astype(np.float64), rstd.astype(np.float64), wd)
    say(f"layer_norm_backward {rows} {cols} {dtype}")
    up = lambda v: torch.from_numpy(v).to(_dev())  # noqa: E731
    # x - mean and its product with rstd: two roundings of xhat
    r = rstd.astype(np.float64)[:, None]
    xhat = np.abs(xd - mean[:, None].astype(np.float64)) * r
    xhat_off = 2 * U32 * xhat
    g = np.abs(dyd * wd)
    d = _terms(cols) * U32
    s1, s2 = g.mean(1, keepdims=True), (g * xhat).mean(1, keepdims=True)
    dx_tol = (6 * U32 * (g + s1 + xhat * s2) + d * (s1 + xhat * s2) + xhat_off * s2
              + xhat * (g * xhat_off).mean(1, keepdims=True)) * r * 1.01
    dx_tol = dx_tol + u(dtype) * np.abs(want[0]) + (2.0 ** -25 if dtype == F16 else 0)
    sums = (rows + 4) * U32
    dw_tol = sums * np.abs(dyd * xhat).sum(0) + (np.abs(dyd) * xhat_off).sum(0)
    db_tol = sums * np.abs(dyd).sum(0)
    for pad in (0, 5):
        got = X.layer_norm_backward(_strided(dy, pad), _strided(x, pad), up(mean), up(rstd), w.to(_dev()))
        for name, v, t, tol in zip(("dx", "dweight", "dbias"), got, want, (dx_tol, dw_tol, db_tol)):
            _close(_np(v), t, tol, (name, pad))
        again = X.layer_norm_backward(_strided(dy, pad), _strided(x, pad), up(mean), up(rstd), w.to(_dev()))
        assert all(torch.equal(i, j) for i, j in zip(got, again))


@pytest.mark.parametrize("rows,cols", [(1, 7), (15, 128), (17, 120), (33, 129), (257, 256), (4099, 64), (9001, 201),
                                       (33000, 128), (5, 257), (1021, 512), (1025, 1024), (8200, 260)])
def test_layer_norm_of_short_rows(rows, cols):
    """Several rows a workgroup, joined into one sum of the parameters'
    gradients: numbers of rows that fill no workgroup, few and many."""
    x, w, b = _norm_inputs(rows, cols, F32, rows * cols)
    dy = torch.from_numpy(np.random.default_rng(rows).standard_normal((rows, cols))).float()
    xd, wd, bd, dyd = (v.double().numpy() for v in (x, w, b, dy))
    say(f"short rows {rows} {cols}")
    want, _, rstd = ol.layer_norm(xd, wd, bd, 1e-5)
    y, m, r = X.layer_norm(x.to(_dev()), w.to(_dev()), b.to(_dev()), stats=True)
    _close(_np(y), want, _norm_tol(xd, wd, bd, want, rstd, F32), "y")
    for pow2 in (False, True):
        q, s = X.layer_norm_quantize(x.to(_dev()), w.to(_dev()), b.to(_dev()), pow2=pow2)
        wq, ws = ol.quantize(y.cpu().numpy(), 1, pow2)
        assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(_bytes(q), wq)
    mean, rs = _np(m), _np(r)
    want = ol.layer_norm_backward(dyd, xd, mean, rs, wd)
    got = X.layer_norm_backward(dy.to(_dev()), x.to(_dev()), m, r, w.to(_dev()))
    xhat = np.abs(xd - mean[:, None]) * rs[:, None]
    g, d = np.abs(dyd * wd), _terms(cols) * U32
    s1, s2 = g.mean(1, keepdims=True), (g * xhat).mean(1, keepdims=True)
    dx_tol = (7 * U32 * (g + s1 + xhat * s2) + (d + 3 * U32) * (s1 + 2 * xhat * s2)) * rs[:, None] * 1.01
    _close(_np(got[0]), want[0], dx_tol, "dx")
    sums = (rows + 6) * U32
    _close(_np(got[1]), want[1], sums * np.abs(dyd * xhat).sum(0), "dweight")
    _close(_np(got[2]), want[2], sums * np.abs(dyd).sum(0), "dbias")


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(r, c) for r in (1, 5, 130) for c in (*range(1, 18), *range(121, 140), 261)])
def test_quantize_reads_nothing_past_the_matrix(rows, cols, dtype, block_rows):
    x = torch.from_numpy(np.random.default_rng(cols).standard_normal((rows, cols))).to(dtype).to(_dev())
    big = torch.full((rows + 3, cols + 19), math.nan, dtype=dtype, device=_dev())
    big[1:rows + 1, 9:9 + cols] = x
    say(f"matrix ends {rows} {cols} {dtype} {block_rows}")
    want = X.fp8_quantize(x, block_rows=block_rows, transposed=True)
    got = X.fp8_quantize(big[1:rows + 1, 9:9 + cols], block_rows=block_rows, transposed=True)
    wq, ws = ol.quantize(x.float().cpu().numpy(), block_rows, False)
    assert np.array_equal(_bytes(want[0]), wq) and np.array_equal(want[1].cpu().numpy(), ws)
    for g, w in zip(got, want):
        same = np.array_equal(_bytes(g), _bytes(w)) if g.dtype != F32 else torch.equal(g, w)
        assert same


@pytest.mark.parametrize("rows,cols", [(5200, 1025), (5121, 1536), (2600, 2049), (2561, 2900), (1300, 4097), (1281, 6144),
                                       (700, 8193), (641, 12288)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_many_rows(rows, cols, dtype):
    """Many rows may take another split of a row over lanes, with another order
    of a row's sums: against float64, the quantised form too."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=gen, device=_dev()).to(dtype)
    w, b = torch.randn(cols, generator=gen, device=_dev()), torch.randn(cols, generator=gen, device=_dev())
    say(f"many rows {rows} {cols} {dtype}")
    y, m, r = X.layer_norm(x, w, b, stats=True)
    xd, wd, bd = x[::7].double().cpu().numpy(), w.double().cpu().numpy(), b.double().cpu().numpy()
    want, mean, rstd = ol.layer_norm(xd, wd, bd, 1e-5)
    _close(_np(y[::7]), want, _norm_tol(xd, wd, bd, want, rstd, dtype), "y")
    q, s, m2, r2 = X.layer_norm_quantize(x, w, b, stats=True)
    back = (q.float().cpu().double().numpy()[::7]
            * np.repeat(s.cpu().double().numpy().T[::7], 128, axis=1)[:, :cols])
    # half a step of e4m3, or of its subnormals, whose step is 2^-9 of the scale
    step = np.repeat(s.cpu().double().numpy().T[::7], 128, axis=1)[:, :cols]
    tol = _norm_tol(xd, wd, bd, want, rstd, F32) * 1.07
    _close(back, want, tol + np.maximum((2.0 ** -4 + U32) * (np.abs(want) + tol), 2.0 ** -10 * step), "quantised")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cols", [*range(1, 25), *range(120, 137), 1021, 2045, 4093, 4099, 8189, 16381])
def test_norm_reads_no_column_past_the_row(cols, dtype):
    """Rows inside larger ones that hold NaN: the same bits as rows of their own."""
    rows = 21
    x, w, b = _norm_inputs(rows, cols, dtype, cols)
    dy = torch.from_numpy(np.random.default_rng(cols).standard_normal((rows, cols))).to(dtype).to(_dev())
    x, w, b = x.to(_dev()), w.to(_dev()), b.to(_dev())
    def among_nan(t):
        big = torch.full((rows, cols + 19), math.nan, dtype=dtype, device=_dev())
        big[:, 9:9 + cols] = t
        return big[:, 9:9 + cols]
    say(f"row ends {cols} {dtype}")
    want = X.layer_norm(x, w, b, stats=True)
    got = X.layer_norm(among_nan(x), w, b, stats=True)
    q, s = X.layer_norm_quantize(x, w, b)
    p, t = X.layer_norm_quantize(among_nan(x), w, b)
    assert np.array_equal(_bytes(q), _bytes(p)) and torch.equal(s, t)
    g = X.layer_norm_backward(dy, x, *want[1:], w)
    h = X.layer_norm_backward(among_nan(dy), among_nan(x), *want[1:], w)
    for i, j in zip((*want, *g), (*got, *h)):
        assert torch.equal(i, j) and not i.isnan().any()


def test_layer_norm_backward_is_the_differences_of_the_forward():
    """Central differences of the oracle's forward pass in float64, so that
    only the kernel's own float32 rounding remains: 1e-5 of values near 1
    allows for 100 of them."""
    rng = np.random.default_rng(6)
    x, dy = rng.standard_normal((4, 50)), rng.standard_normal((4, 50))
    w, b = rng.standard_normal(50), rng.standard_normal(50)
    up = lambda v: torch.from_numpy(v).float().to(_dev())  # noqa: E731
    x, dy, w = (v.astype(np.float32).astype(np.float64) for v in (x, dy, w))
    _, m, r = X.layer_norm(up(x), up(w), up(b), stats=True)
    got = X.layer_norm_backward(up(dy), up(x), m, r, up(w))
    loss = lambda x, w, b: (ol.layer_norm(x, w, b, 1e-5)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for grad, arg in zip(got, (0, 1, 2)):
        for at in np.ndindex(*grad.shape):
            lo, hi = [x.copy(), w.copy(), b.copy()], [x.copy(), w.copy(), b.copy()]
            lo[arg][at] -= h
            hi[arg][at] += h
            diff = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(diff - float(grad[at])) < 1e-5 * max(1.0, abs(diff))


# ----- clipping ----------------------------------------------------------------------------

def _grads(shapes, seed, size=1e-2):
    rng = np.random.default_rng(seed)
    types = (F32, F16, BF16)
    return [torch.from_numpy(rng.standard_normal(s) * size).to(types[i % 3]).to(_dev())
            for i, s in enumerate(shapes)]


@pytest.mark.parametrize("shapes", [[(1,)], [(7,), (0,), (3, 5)], [(16384,), (16385,)], [(1000, 333), (5,), (2049, 77)], [(3,), (4,), (7,), (8,), (9,)],
                                    [(i % 9 + 1, 3) for i in range(250)]])
@pytest.mark.parametrize("max_norm", [1e9, 0.01, 0.0])
def test_clip(shapes, max_norm):
    grads = _grads(shapes, len(shapes))
    before = [g.clone() for g in grads]
    say(f"clip {len(shapes)} {max_norm}")
    norm, out = X.clip_grad_norm(grads, max_norm)
    want, factor = ol.clip([_np(g) for g in grads], max_norm, 1e-6)
    # the one rounding of a sum of 64 bits
    assert abs(norm.item() - want) <= U32 * want * (1 + 1e-6) and norm.dim() == 0
    for g, o, b in zip(grads, out, before):
        assert torch.equal(g, b)
        # the factor's rounding, the product's, the type's
        tol = np.abs(_np(g)) * factor * (2 * U32 + u(g.dtype)) * 1.01 + (2.0 ** -25 if g.dtype == F16 else 2.0 ** -149)
        _close(_np(o), _np(g) * factor, tol, "clipped")
    n2, same = X.clip_grad_norm(grads, max_norm, out=grads)
    assert torch.equal(n2, norm) and all(a is b for a, b in zip(same, grads))
    assert all(torch.equal(g, o) for g, o in zip(grads, out))


def test_clip_views_and_orders():
    base = torch.randn(40, 30, device=_dev())
    flat = torch.randn(5000, device=_dev())
    grads = [base.t(), flat[1:4000], flat[4001:]]
    norm, out = X.clip_grad_norm(grads, 0.5)
    factor = min(1.0, 0.5 / (norm.item() + 1e-6))
    for g, o in zip(grads, out):
        _close(_np(o), _np(g) * factor, np.abs(_np(g)) * 4 * U32, "view")
    with pytest.raises(ValueError):
        X.clip_grad_norm([base[:, :7]], 0.5)


def test_clip_special_values():
    big = torch.full((100,), 1e30, device=_dev())
    norm, out = X.clip_grad_norm([big], 1.0)  # its square is over float32
    assert norm.item() == pytest.approx(1e31, rel=1e-6) and out[0][0].item() == pytest.approx(0.1, rel=1e-6)
    g = torch.tensor([1.0, math.inf], device=_dev())
    norm, out = X.clip_grad_norm([g, big], 1.0)
    assert norm.item() == math.inf and out[0][0].item() == 0 and out[0][1].isnan() and not out[1].any()
    g[0] = math.nan
    norm, out = X.clip_grad_norm([g, big], 1.0)
    assert norm.isnan() and out[1].isnan().all()
    norm, out = X.clip_grad_norm([torch.zeros(0, device=_dev())], 1.0)
    assert norm.item() == 0


# ----- streams, graphs, refusals -------------------------------------------------------------

def _step(x, w, b, weight_q, weight_s, grads, **more):
    q, s = X.layer_norm_quantize(x, w, b, **more)
    c = X.fp8_gemm(q, s, weight_q, weight_s, out_dtype=F32, **more)
    y, m, r = X.layer_norm(x, w, b, stats=True, **more)
    dx, dw, db = X.layer_norm_backward(y, x, m, r, w, **more)
    q2, s2, qt, st = X.fp8_quantize(y, transposed=True, **more)
    norm, out = X.clip_grad_norm([dx, dw, db, *grads], 0.1, **more)
    return [q.float(), s, c, y, dx, dw, db, q2.float(), s2, qt.float(), st, norm, *out]


def _step_inputs(m):
    x, w, b = (t.to(_dev()) for t in _norm_inputs(m, 640, BF16, 12))
    wq, ws = X.fp8_quantize(torch.randn(384, 640, device=_dev()) * 0.02, block_rows=128)
    return x, w, b, wq, ws, _grads([(100, 7), (33,)], 2)


@pytest.mark.parametrize("m", [4, 300])
def test_on_another_stream(m):
    args = _step_inputs(m)
    want = _step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # the calls on `side` by name; casts of the results once it is done
    x, w, b, wq, ws, grads = args
    q, s = X.layer_norm_quantize(x, w, b, stream=side)
    c = X.fp8_gemm(q, s, wq, ws, out_dtype=F32, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c, want[2]) and torch.equal(q.float(), want[0])
    with torch.cuda.stream(side):
        got = _step(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(g, v) for g, v in zip(got, want))


@pytest.mark.parametrize("m", [4, 300])
def test_in_a_graph(m):
    args = _step_inputs(m)
    x = args[0]
    _step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(*args)
    for seed in range(4):
        x.copy_(_norm_inputs(m, 640, BF16, 30 + seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        want = _step(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))


def test_refusals():
    dev = _dev()
    z = lambda *s, **k: torch.zeros(*s, device=dev, **k)  # noqa: E731
    q, s = X.fp8_quantize(z(32, 256))
    for call, error in [
        (lambda: X.fp8_gemm(q, s, q[:, :128], s), ValueError),
        (lambda: X.fp8_gemm(q, s[:1], q, s), ValueError),
        (lambda: X.fp8_gemm(q, s, q, s[:, :5]), ValueError),
        (lambda: X.fp8_gemm(q.float(), s, q, s), TypeError),
        (lambda: X.fp8_gemm(q, s.half(), q, s), TypeError),
        (lambda: X.fp8_gemm(q, s, q, s, out_dtype=torch.float64), TypeError),
        (lambda: X.fp8_gemm(q, s, q, s, out=z(32, 31)), ValueError),
        (lambda: X.fp8_gemm(q, s.cpu(), q, s), ValueError),
        (lambda: X.fp8_gemm(q[:, 8:], s, q[:, 8:], s), X.XposeError),
        (lambda: X.fp8_quantize(z(4, 4, dtype=torch.float64)), TypeError),
        (lambda: X.fp8_quantize(z(4, 4), block_rows=64), ValueError),
        (lambda: X.fp8_quantize(z(4, 8)[:, ::2]), ValueError),
        (lambda: X.fp8_quantize(z(4)), ValueError),
        (lambda: X.layer_norm(z(4, 4), z(3)), ValueError),
        (lambda: X.layer_norm(z(4, 4), z(4), z(4, dtype=BF16)), TypeError),
        (lambda: X.layer_norm(z(4, 4), out=z(4, 5)), ValueError),
        (lambda: X.layer_norm(z(4, 0)), ValueError),
        (lambda: X.layer_norm(z(4, 4), eps=-1.0), X.XposeError),
        (lambda: X.layer_norm_backward(z(4, 4), z(4, 5), z(4), z(4)), ValueError),
        (lambda: X.layer_norm_backward(z(4, 4), z(4, 4), z(4), z(5)), ValueError),
        (lambda: X.layer_norm_backward(z(4, 4), z(4, 4), z(4, dtype=BF16), z(4)), TypeError),
        (lambda: X.clip_grad_norm([z(4)], 1.0, out=[z(5)]), ValueError),
        (lambda: X.clip_grad_norm([z(4)], 1.0, out=[]), ValueError),
        (lambda: X.clip_grad_norm([z(4, dtype=torch.float64)], 1.0), TypeError),
        (lambda: X.clip_grad_norm([z(4)], -1.0), X.XposeError),
    ]:
        with pytest.raises(error):
            call()


# ----- the layer of examples/fp8_linear.py ------------------------------------------------------

def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_linear.py")
    spec = importlib.util.spec_from_file_location("fp8_linear_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,width,outputs", [(700, 333, 200), (1000, 1024, 640)])
def test_layer_gradients(tokens, width, outputs):
    """The whole step against float64 autograd of the unquantised layer: e4m3
    keeps each operand within 2^-4 of itself, so each product within 2^-3 of
    its magnitudes and far nearer in the norm of the whole."""
    ex = _example()
    layer = ex.Fp8Linear(width, outputs, _dev(), seed=4)
    layer.gain += 0.1 * torch.randn(width, device=_dev())
    layer.bias += 0.1 * torch.randn(width, device=_dev())
    x = (torch.randn(tokens, width, device=_dev()) + 0.3).bfloat16()
    grad = (torch.randn(tokens, outputs, device=_dev()) * 1e-2).bfloat16()
    wq = layer.quantized_weight()
    out, saved = layer.forward(x, wq)
    gx, grads = layer.backward(grad, saved, wq)
    ref = [t.double().cpu().requires_grad_() for t in (x, *layer.parameters())]
    y = torch.nn.functional.layer_norm(ref[0], (width,), ref[1], ref[2], 1e-5) @ ref[3].t()
    y.backward(grad.double().cpu())
    for got, want in zip([out, gx, *grads], [y.detach()] + [r.grad for r in ref]):
        off = (got.double().cpu() - want).norm() / want.norm()
        assert off < 2.0 ** -3, off
    served = layer.serve(x[:3], wq)
    assert (served.double().cpu() - y.detach()[:3]).norm() / y.detach()[:3].norm() < 2.0 ** -3


def test_training_learns():
    losses = _example().train(tokens=512, width=256, outputs=192, steps=12, log=None)
    assert losses[-1] < 0.5 * losses[0]
