"""A residual block's operators on the GPU against the float64 oracle.

Tolerances.  u(t) = eps(t) / 2 is the relative error of one rounding to t.  A
sum of n terms in float32 is within n u of the sum of magnitudes whatever its
order; the matrix cores' own additions may cut bits off instead of rounding
them, twice that.  What has one answer (the stored sum of a norm, quantised
values, the dropout mask, rows without an adapter) has to be equal."""
import math

import numpy as np
import pytest

import oracle.block as ob
import oracle.linear as ol
from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
U32 = 2.0 ** -24


def u(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half a step of dtype at 0."""
    return {F16: 2.0 ** -25, F32: 2.0 ** -150, BF16: 2.0 ** -134}[dtype]


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


def _np(t):
    return t.detach().cpu().double().numpy()


def _up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a
    return (t if dtype is None else t.to(dtype)).to(_dev())


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


# ----- root-mean-square norm ------------------------------------------------------

COLS = [1, 5, 8, 100, 200, 257, 513, 1024, 1500, 2048, 2999, 4096, 5000, 8192, 10001, 16384, 20000]


def _terms(cols):
    """The longest chain of additions behind a row's sum, roundings of the
    terms included: a lane's columns, the lanes of a wave, the waves."""
    return 32 + cols // 1024 + 6 + 16


def _norm_inputs(rows, cols, dtype, seed, params=F32):
    rng = np.random.default_rng(seed)
    x, r = rng.standard_normal((rows, cols)) * 2, rng.standard_normal((rows, cols)) * 3
    if rows > 2:
        x[2], r[2] = 0, 0
    w = 1 + 0.1 * rng.standard_normal(cols)
    return tuple(torch.from_numpy(v).to(t) for v, t in ((x, dtype), (r, dtype), (w, params)))


def _norm_tol(y, cols, dtype):
    # half of the mean square's error, square root, quotient, two products
    return np.abs(y) * ((_terms(cols) / 2 + 6) * U32 + u(dtype)) * 1.01 + least(dtype)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(cols, dtype, residual):
    x, r, w = _norm_inputs(6, cols, dtype, cols)
    h = (x.float() + r.float()).to(dtype) if residual else x
    want, rstd = ob.rms_norm(_np(h), _np(w), 1e-5)
    say(f"rms_norm {cols} {dtype} {residual}")
    for pad in (0, 3, 8):
        v, res = _strided(x, pad), _strided(r, pad) if residual else None
        got = X.rms_norm(v, _up(w), residual=res, stats=True)
        assert len(got) == 2 + residual
        _close(_np(got[0]), want, _norm_tol(want, cols, dtype), ("y", pad))
        _close(_np(got[-1]), rstd, rstd * (_terms(cols) / 2 + 5) * U32, "rstd")
        if residual:
            assert torch.equal(got[1].cpu(), h)
            y, same = X.rms_norm(v, _up(w), residual=res)
            assert torch.equal(y, got[0]) and torch.equal(same, got[1])
        else:
            assert torch.equal(X.rms_norm(v, _up(w)), got[0])


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_quantize(cols, dtype, pow2, residual):
    """The float32 result's quantisation: that of the kernel's own float32
    tensor over the same h, bit for bit."""
    x, r, w = _norm_inputs(5, cols, dtype, cols)
    h = (x.float() + r.float()).to(dtype) if residual else x
    say(f"rms_norm_quantize {cols} {dtype} {pow2} {residual}")
    y, rstd = X.rms_norm(_up(h).float(), _up(w), stats=True)
    wq, ws = ol.quantize(y.cpu().numpy(), 1, pow2)
    for pad in (0, 3):
        v, res = _strided(x, pad), _strided(r, pad) if residual else None
        got = X.rms_norm_quantize(v, _up(w), residual=res, pow2=pow2, stats=True)
        assert np.array_equal(got[1].cpu().numpy(), ws) and np.array_equal(_bytes(got[0]), wq)
        assert torch.equal(got[-1], rstd)
        if residual:
            assert torch.equal(got[2].cpu(), h)
        assert len(X.rms_norm_quantize(v, residual=res)) == 2 + residual


@pytest.mark.parametrize("params", [F16, BF16, None])
@pytest.mark.parametrize("cols", [4, 100, 3001, 20000])
def test_rms_norm_parameter_types(cols, params):
    x, r, w = _norm_inputs(5, cols, BF16, cols, params or F32)
    if params is None:
        w = torch.ones_like(w)
    arg = None if params is None else _up(w)
    want = X.rms_norm(_up(x), _up(w.float()), residual=_up(r), stats=True)
    got = X.rms_norm(_up(x), arg, residual=_up(r), stats=True)
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    q, p = X.rms_norm_quantize(_up(x), arg), X.rms_norm_quantize(_up(x), _up(w.float()))
    assert np.array_equal(_bytes(q[0]), _bytes(p[0])) and torch.equal(q[1], p[1])
    g = X.rms_norm_backward(_up(r), got[1], got[2], arg)
    v = X.rms_norm_backward(_up(r), got[1], got[2], _up(w.float()))
    assert all(torch.equal(i, j) for i, j in zip(g, v))


@pytest.mark.parametrize("rows,cols", [(3001, 96), (5000, 3), (2500, 640), (1100, 1500), (700, 5000)])
def test_rms_norm_of_many_rows(rows, cols):
    """More rows than workgroups run at once."""
    x, r, w = _norm_inputs(rows, cols, BF16, rows)
    h = (x.float() + r.float()).to(BF16)
    want, rstd = ob.rms_norm(_np(h), _np(w), 1e-5)
    say(f"rms_norm rows {rows} {cols}")
    y, got, s = X.rms_norm(_up(x), _up(w), residual=_up(r), stats=True)
    assert torch.equal(got.cpu(), h)
    _close(_np(y), want, _norm_tol(want, cols, BF16), "y")
    _close(_np(s), rstd, rstd * (_terms(cols) / 2 + 5) * U32, "rstd")


@pytest.mark.parametrize("cols", [5, 96, 700, 3001, 9000, 20000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rms_norm_in_place(cols, dtype):
    x, r, w = _norm_inputs(700 if cols < 9000 else 40, cols, dtype, cols)
    want = X.rms_norm(_up(x), _up(w), residual=_up(r))
    alone = X.rms_norm(_up(x), _up(w))
    say(f"rms_norm in place {cols} {dtype}")
    for out, res_out in (("x", "r"), ("r", "x"), ("x", None), (None, "x"), (None, "r"), ("r", None)):
        t = {"x": _up(x), "r": _up(r), None: None}
        y, h = X.rms_norm(t["x"], _up(w), residual=t["r"], out=t[out], residual_out=t[res_out])
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
        assert (out is None or y is t[out]) and (res_out is None or h is t[res_out])
    v = _up(x)
    assert X.rms_norm(v, _up(w), out=v) is v and torch.equal(v, alone)
    q = X.rms_norm_quantize(_up(x), _up(w), residual=_up(r))
    t = _up(r)
    p = X.rms_norm_quantize(_up(x), _up(w), residual=t, residual_out=t)
    assert np.array_equal(_bytes(q[0]), _bytes(p[0])) and torch.equal(p[2], q[2]) and p[2] is t


def test_rms_norm_writes_its_region_alone():
    x, r, w = _norm_inputs(40, 333, BF16, 3)
    want = X.rms_norm(_up(x), _up(w), residual=_up(r))
    y, h = (torch.full((40, 350), -5.0, dtype=BF16, device=_dev()) for _ in range(2))
    X.rms_norm(_up(x), _up(w), residual=_up(r), out=y[:, 3:336], residual_out=h[:, 7:340])
    assert torch.equal(y[:, 3:336], want[0]) and torch.equal(h[:, 7:340], want[1])
    assert (y[:, :3] == -5).all() and (y[:, 336:] == -5).all() and (h[:, :7] == -5).all() and (h[:, 340:] == -5).all()


def test_rms_norm_special_values_and_none():
    x, r, w = _norm_inputs(6, 700, F32, 8)
    clean = X.rms_norm(_up(x), _up(w), residual=_up(r))[0].cpu()
    x[1, 5], r[3, 699], x[4, 0] = math.nan, math.inf, 3e38
    y, h, rstd = (t.cpu() for t in X.rms_norm(_up(x), _up(w), residual=_up(r), stats=True))
    assert y[1].isnan().all() and rstd[3] == 0 and y[3, 699].isnan() and not y[3, :699].any()
    assert rstd[4] == 0 and not y[4].any()  # squares over float32
    assert torch.equal(y[[0, 2, 5]], clean[[0, 2, 5]])
    assert rstd[2].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    e = torch.zeros(0, 96, dtype=BF16, device=_dev())
    assert X.rms_norm(e, residual=e)[1].shape == (0, 96)
    assert X.rms_norm_quantize(e)[1].shape == (1, 0)
    dx, dw = X.rms_norm_backward(e, e, torch.zeros(0, device=_dev()))
    assert dx.shape == (0, 96) and dw.shape == (96,) and not dw.any()


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (5, 8), (700, 5), (37, 200), (37, 513), (700, 1000), (9, 1500),
                                       (1300, 2048), (40, 2999), (40, 4096), (30, 5000), (30, 8192), (20, 8193),
                                       (21, 20001), (5000, 64)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_backward(rows, cols, dtype, residual):
    h, res, w = _norm_inputs(rows, cols, dtype, rows + cols)
    rng = np.random.default_rng(cols)
    dy = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))).to(dtype)
    _, rstd = ob.rms_norm(_np(h), 1.0, 1e-5)
    rstd = rstd.astype(np.float32)
    if rows > 2:
        rstd[2] = 1.0  # of a row of zeros: else its inverse root of eps alone
    r64, hd, wd, dyd = rstd.astype(np.float64), _np(h), _np(w), _np(dy)
    want, dw = ob.rms_norm_backward(dyd, hd, r64, wd, _np(res) if residual else 0.0)
    say(f"rms_norm_backward {rows} {cols} {dtype} {residual}")
    xhat, g = np.abs(hd * r64[:, None]), np.abs(dyd * wd)
    d = (_terms(cols) + 4) * U32
    mean_off = d * (g * xhat).mean(1, keepdims=True)
    along = np.abs((dyd * wd * hd * r64[:, None]).mean(1, keepdims=True))
    # g, xhat s, their difference, the product with rstd, the residual's addition
    tol = r64[:, None] * (3 * U32 * g + xhat * (mean_off + 5 * U32 * along)) + 2 * U32 * (np.abs(want) + np.abs(_np(res)))
    tol = tol * 1.01 + u(dtype) * np.abs(want) * 1.01 + least(dtype)
    dw_tol = (rows + 40) * U32 * np.abs(dyd * hd * r64[:, None]).sum(0)
    for pad in (0, 3):
        got, gw = X.rms_norm_backward(_strided(dy, pad), _strided(h, pad), _up(rstd), _up(w),
                                      dresidual=_strided(res, pad) if residual else None)
        _close(_np(got), want, tol, ("dx", pad))
        _close(_np(gw), dw, dw_tol, ("dweight", pad))


@pytest.mark.parametrize("cols", [6, 100, 20001])
def test_rms_norm_backward_against_differences(cols):
    """(f(h + t d) - f(h - t d)) / 2 t of the norm itself, in float32."""
    gen = torch.Generator(device=_dev()).manual_seed(cols)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    h, w, dy, d = r(4, cols), r(cols), r(4, cols), r(4, cols)
    _, rstd = X.rms_norm(h, w, stats=True)
    dx, dw = X.rms_norm_backward(dy, h, rstd, w)
    t = 2.0 ** -6
    f = lambda v, p: X.rms_norm(v, p).double()  # noqa: E731
    slope = ((f(h + t * d, w) - f(h - t * d, w)) * dy).sum() / (2 * t)
    terms = (dx.double() * d).abs().sum() + 1
    assert abs(slope - (dx.double() * d).sum()) < 0.02 * terms
    slope = ((f(h, w + t * d[0]) - f(h, w - t * d[0])) * dy).sum() / (2 * t)
    assert abs(slope - (dw.double() * d[0]).sum()) < 1e-3 * ((dw.double() * d[0]).abs().sum() + 1)


# ----- low-rank adapters ------------------------------------------------------------

def _adapter_case(m, n, k, rank, count, dtype, out, seed, quantized=False, ids=None):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((m, k)) * np.exp(rng.uniform(-2, 2, (m, 1)))).to(dtype)
    a = torch.from_numpy(rng.standard_normal((count, rank, k)) * max(k, 1) ** -0.5).to(dtype)
    b = torch.from_numpy(rng.standard_normal((count, n, rank))).to(dtype)
    base = torch.from_numpy(rng.standard_normal((m, n))).to(out)
    if ids is None:
        ids = rng.integers(-1, count + 1, m)
    scale = torch.from_numpy(rng.uniform(0.5, 2, count)).float()
    xs = None
    if quantized:
        q, s = ol.quantize(x.float().numpy())
        xs = (q, s, ol.dequantize(q, s))
    return dict(x=x, a=a, b=b, base=base, ids=np.asarray(ids, np.int32), scale=scale, xs=xs)


def _e4m3(bits):
    """Bytes on the GPU with rows at multiples of 16 and NaN between."""
    rows, cols = bits.shape
    pitch = -(-max(cols, 1) // 16) * 16 + 16
    store = torch.full((rows, pitch), 0x7f, dtype=torch.uint8, device=_dev())
    store[:, :cols] = _up(bits)
    return store.view(torch.float8_e4m3fn)[:, :cols]


def _stack(t, pad):
    """Adapters as views into larger ones of NaN, in every dimension."""
    count, rows, cols = t.shape
    store = torch.full((count, rows + pad, cols + pad), math.nan, dtype=t.dtype, device=_dev())
    view = store[:, :rows, :cols]
    view.copy_(t)
    return view


def _adapters_want(c):
    """(out, hidden and their tolerances before the last rounding)."""
    xd = c["xs"][2] if c["xs"] else _np(c["x"])
    a, b, s, base = _np(c["a"]), _np(c["b"]), _np(c["scale"]), _np(c["base"])
    want, hidden = ob.adapters(xd, a, b, c["ids"], s, base)
    k, rank = xd.shape[1], a.shape[1]
    mag, hmag = ob.adapters(np.abs(xd), np.abs(a), np.abs(b), c["ids"], s, 0 * base)
    # k products in sums that may cut, a block's scale and its addition, the slices' sums
    hrel = (2 * k + 24 + (k // 64 if c["xs"] else 0)) * U32
    # the scale, h as three parts (2^-24 of it left), rank products of each, base's addition
    tol = (hrel + (6 * rank + 12) * U32) * mag + 2 * U32 * (np.abs(base) + np.abs(want))
    return want, hidden, tol, hrel * hmag


def _run_adapters(c, pad=0, **more):
    x = _strided(c["x"], pad)
    if c["xs"]:
        x, more["scale_x"] = _e4m3(c["xs"][0]), _up(c["xs"][1])
    a, b = (_stack(c["a"], pad), _stack(c["b"], pad)) if pad else (_up(c["a"]), _up(c["b"]))
    more.setdefault("base", _strided(c["base"], pad))
    more.setdefault("scale", _up(c["scale"]))
    return X.adapters(x, a, b, _up(c["ids"]), **more)


def _check_adapters(c, pads=(0, 3)):
    want, hidden, tol, htol = _adapters_want(c)
    out = c["base"].dtype
    tol = tol * (1 + u(out)) + u(out) * np.abs(want) + least(out)
    for pad in pads:
        got, h = _run_adapters(c, pad, hidden=True)
        assert got.dtype == out and h.dtype == F32
        _close(_np(h), hidden, htol + least(F32), ("hidden", pad))
        _close(_np(got), want, tol, ("out", pad))
        again = _run_adapters(c, pad)
        _close(_np(again), want, tol, ("out without hidden", pad))
        none = (c["ids"] < 0) | (c["ids"] >= len(c["a"]))
        assert torch.equal(got.cpu()[none], c["base"][none]) and not h.cpu()[none].any()


ADAPTER_SIZES = [(1, 1, 1, 1, 1), (1, 300, 128, 16, 3), (2, 17, 1000, 8, 1), (5, 64, 257, 4, 2), (16, 257, 130, 16, 9),
                 (17, 40, 3, 5, 4), (31, 256, 4100, 12, 40), (64, 333, 640, 16, 64), (65, 513, 127, 24, 3),
                 (100, 100, 300, 32, 2), (150, 70, 1222, 64, 5), (33, 90, 200, 100, 3), (7, 5, 7, 2, 3),
                 (90, 130, 1500, 72, 3), (40, 1100, 6, 128, 2), (70, 6, 515, 33, 4)]


@pytest.mark.parametrize("m,n,k,rank,count", ADAPTER_SIZES)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("quantized", [False, True])
def test_adapters(m, n, k, rank, count, dtype, out, quantized):
    say(f"adapters {m} {n} {k} {rank} {count} {dtype} {out} {quantized}")
    _check_adapters(_adapter_case(m, n, k, rank, count, dtype, out, m + n + k, quantized))


@pytest.mark.parametrize("m,k", [(4097, 200), (5001, 300)])
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("kind", ["one", "requests", "mixed", "none"])
def test_adapters_of_many_rows(m, k, quantized, kind):
    rng = np.random.default_rng(m)
    ids = {"one": np.zeros(m), "requests": np.repeat(rng.integers(-1, 5, 20), -(-m // 20))[:m],
           "mixed": rng.integers(-1, 5, m), "none": np.full(m, -1)}[kind]
    say(f"adapters rows {m} {k} {quantized} {kind}")
    _check_adapters(_adapter_case(m, 300, k, 16, 5, BF16, BF16, m, quantized, ids), pads=(0,))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("rank", [5, 16, 40])
def test_adapters_of_many_e4m3_rows(dtype, rank):
    say(f"adapters e4m3 rows {dtype} {rank}")
    ids = np.arange(4500) * 7 // 300 % 6 - 1
    _check_adapters(_adapter_case(4500, 130, 333, rank, 4, dtype, dtype, rank, True, ids), pads=(0,))


def test_adapters_slices_and_slots():
    """One token with a long k; rows with an adapter each and all the same."""
    _check_adapters(_adapter_case(1, 100, 8200, 16, 4, BF16, F32, 1, ids=[2]))
    _check_adapters(_adapter_case(16, 100, 8200, 16, 16, BF16, F32, 2, ids=np.arange(16)))
    _check_adapters(_adapter_case(16, 100, 8200, 16, 16, F16, F16, 3, True, ids=np.full(16, 7)))
    _check_adapters(_adapter_case(40, 100, 8200, 16, 40, BF16, F32, 4, ids=np.arange(40)[::-1]))
    c = _adapter_case(16, 100, 8200, 16, 16, BF16, F32, 2, ids=np.arange(16))
    first = _run_adapters(c, hidden=True)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, _run_adapters(c, hidden=True)))


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F16, F32)])
def test_adapters_in_place_and_without_base(dtype, out):
    c = _adapter_case(90, 300, 260, 16, 4, dtype, out, 6)
    want = _run_adapters(c)
    store = torch.full((97, 310), -5.0, dtype=out, device=_dev())
    view = store[:90, 3:303]
    view.copy_(_up(c["base"]))
    say(f"adapters in place {dtype} {out}")
    assert _run_adapters(c, base=view, out=view) is view and torch.equal(view, want)
    assert (store[90:] == -5).all() and (store[:, :3] == -5).all() and (store[:, 303:] == -5).all()
    bare = _run_adapters(c, base=None, out=torch.full((90, 300), 7.0, dtype=out, device=_dev()))
    c["base"] = torch.zeros_like(c["base"])
    assert torch.equal(bare, _run_adapters(c))
    assert X.adapters(_up(c["x"]), _up(c["a"]), _up(c["b"]), _up(c["ids"])).dtype == dtype
    ones = _run_adapters(c, scale=torch.full((4,), 0.25, device=_dev()))
    assert torch.equal(_run_adapters(c, scale=0.25), ones)


def test_adapters_keep_what_rows_without_one_hold():
    """Whatever their x and base are: NaN and infinities stay where they are,
    and a zero keeps its sign."""
    for out in (BF16, F32):
        c = _adapter_case(40, 70, 200, 16, 3, BF16, out, 7)
        ids = c["ids"] = np.where(np.arange(40) % 3 == 0, -1, np.arange(40) % 3).astype(np.int32)
        clean = _run_adapters(c)
        c["x"][::3] = math.nan
        c["base"][0], c["base"][3], c["base"][6] = math.nan, math.inf, -0.0
        got = _run_adapters(c)
        mine = torch.from_numpy(ids >= 0)
        assert torch.equal(got.cpu()[mine], clean.cpu()[mine])
        assert torch.equal(got.cpu()[6].signbit(), c["base"][6].signbit()) and got[0].isnan().all()


def test_adapters_do_not_reach_into_each_other():
    """An adapter of NaN and infinities, and a row of them, among others."""
    c = _adapter_case(64, 150, 300, 16, 5, BF16, BF16, 8, ids=np.arange(64) % 5)
    clean, h = _run_adapters(c, hidden=True)
    c["a"][2], c["b"][2], c["b"][3, 5] = math.nan, math.inf, math.inf
    c["x"][10, 7] = math.inf
    got, hid = _run_adapters(c, hidden=True)
    same = torch.tensor([i % 5 not in (2, 3) and i != 10 for i in range(64)])
    assert torch.equal(got.cpu()[same], clean.cpu()[same]) and torch.equal(hid.cpu()[same], h.cpu()[same])
    three = torch.tensor([i % 5 == 3 for i in range(64)])
    cols = torch.arange(150) != 5
    assert torch.equal(got.cpu()[three][:, cols], clean.cpu()[three][:, cols])
    assert not got.cpu()[three][:, 5].isfinite().any()
    assert not got.cpu()[2::5].isfinite().any()
    assert not torch.isfinite(hid.cpu()[10]).any()


def test_adapters_without_sizes():
    z = lambda *s, **k: torch.zeros(*s, device=_dev(), **k)  # noqa: E731
    i = lambda m: z(m, dtype=torch.int32)  # noqa: E731
    base = torch.randn(9, 20, device=_dev())
    for x, a, b in ((z(9, 6), z(0, 4, 6), z(0, 20, 4)), (z(9, 6), z(2, 0, 6), z(2, 20, 0)),
                    (z(9, 0), z(2, 4, 0), z(2, 20, 4))):
        out, h = X.adapters(x, a, b, i(9), base=base, hidden=True)
        assert torch.equal(out, base) and h.shape == (9, a.shape[1]) and not h.any()
        dx, da, db = X.adapters_backward(torch.ones(9, 20, device=_dev()), x, a, b, i(9), h,
                                         base=torch.ones(9, x.shape[1], device=_dev()))
        assert dx.shape == x.shape and (dx == 1).all() and da.shape == a.shape and db.shape == b.shape
        assert not da.any() and not db.any()
    out, h = X.adapters(z(0, 6), z(2, 4, 6), z(2, 20, 4), i(0), hidden=True)
    assert out.shape == (0, 20) and h.shape == (0, 4)
    dx, da, db = X.adapters_backward(z(0, 20), z(0, 6), z(2, 4, 6), z(2, 20, 4), i(0), h)
    assert dx.shape == (0, 6) and da.shape == (2, 4, 6) and not da.any() and not db.any()
    out, h = X.adapters(torch.ones(3, 6, device=_dev()), torch.ones(1, 4, 6, device=_dev()), z(1, 0, 4), i(3), hidden=True)
    assert out.shape == (3, 0) and (h == 6).all()


def test_adapters_of_far_rows():
    """Rows of x and adapters that start over 2^31 elements into their buffers."""
    m, k, rank, n = 40, 256, 16, 48
    c = _adapter_case(m, n, k, rank, 3, BF16, BF16, 9)
    want = _run_adapters(c, hidden=True)
    pitch, step = 1 << 26, 1 << 30
    sx = torch.zeros((m - 1) * pitch + k, dtype=BF16, device=_dev())
    x = torch.as_strided(sx, (m, k), (pitch, 1))
    x.copy_(_up(c["x"]))
    sw = torch.zeros(2 * step + rank * k, dtype=BF16, device=_dev())
    a = torch.as_strided(sw, (3, rank, k), (step, k, 1))
    a.copy_(_up(c["a"]))
    say("adapters far rows")
    got = X.adapters(x, a, _up(c["b"]), _up(c["ids"]), base=_up(c["base"]), scale=_up(c["scale"]), hidden=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    dout = torch.randn(m, n, device=_dev()).to(BF16)
    args = (_up(c["b"]), _up(c["ids"]), want[1])
    p = X.adapters_backward(dout, x, a, *args)
    q = X.adapters_backward(dout, _up(c["x"]), _up(c["a"]), *args)
    assert all(torch.equal(i, j) for i, j in zip(p, q))


def _backward_case(m, n, k, rank, count, dtype, out, seed, ids=None):
    c = _adapter_case(m, n, k, rank, count, dtype, out, seed, ids=ids)
    rng = np.random.default_rng(seed + 1)
    c["dout"] = torch.from_numpy(rng.standard_normal((m, n)) * 0.1).to(dtype)
    c["base"] = torch.from_numpy(rng.standard_normal((m, k))).to(out)
    c["hidden"] = torch.from_numpy(ob.adapters(_np(c["x"]), _np(c["a"]), _np(c["b"]), c["ids"], _np(c["scale"]),
                                               np.zeros((m, n)))[1]).float()
    return c


def _run_backward(c, pad=0, **more):
    a, b = (_stack(c["a"], pad), _stack(c["b"], pad)) if pad else (_up(c["a"]), _up(c["b"]))
    more.setdefault("base", _strided(c["base"], pad))
    more.setdefault("scale", _up(c["scale"]))
    return X.adapters_backward(_strided(c["dout"], pad), _strided(c["x"], pad), a, b, _up(c["ids"]), _up(c["hidden"]),
                               **more)


def _check_backward(c, pads=(0, 3)):
    n64 = {v: _np(c[v]) for v in ("dout", "x", "a", "b", "scale", "hidden", "base")}
    m, n = n64["dout"].shape
    rank = n64["a"].shape[1]
    dx, da, db, _ = ob.adapters_backward(n64["dout"], n64["x"], n64["a"], n64["b"], c["ids"], n64["scale"],
                                         n64["hidden"], n64["base"])
    mag = {v: np.abs(n64[v]) for v in n64}
    mx, ma, mb, _ = ob.adapters_backward(mag["dout"], mag["x"], mag["a"], mag["b"], c["ids"], mag["scale"],
                                         mag["hidden"], 0 * n64["base"])
    dh_rel = (2 * n + 24) * U32  # n products in sums that may cut, the scale, the slices' sums
    out = c["base"].dtype
    tol = (dh_rel + (6 * rank + 12) * U32) * mx + 2 * U32 * (mag["base"] + np.abs(dx))
    tol = tol * (1 + u(out)) + u(out) * np.abs(dx) + least(out)
    # m products in sums that may cut
    grad_rel = (2 * m + 24) * U32
    for pad in pads:
        got = _run_backward(c, pad)
        assert got[0].dtype == out and got[1].dtype == F32 and got[2].dtype == F32
        _close(_np(got[0]), dx, tol, ("dx", pad))
        _close(_np(got[1]), da, (dh_rel + grad_rel) * ma + least(F32), ("da", pad))
        _close(_np(got[2]), db, grad_rel * mb + least(F32), ("db", pad))


@pytest.mark.parametrize("m,n,k,rank,count", ADAPTER_SIZES + [(300, 129, 127, 16, 2), (1000, 40, 300, 16, 3)])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
def test_adapters_backward(m, n, k, rank, count, dtype, out):
    say(f"adapters_backward {m} {n} {k} {rank} {count} {dtype} {out}")
    _check_backward(_backward_case(m, n, k, rank, count, dtype, out, m + n + k))


@pytest.mark.parametrize("kind", ["one", "requests", "mixed", "none", "last"])
@pytest.mark.parametrize("m", [64, 65, 1001, 4500])
def test_adapters_backward_rows(m, kind):
    """Pieces of an adapter's rows: none, one, several, and sorted by hand."""
    rng = np.random.default_rng(m)
    ids = {"one": np.zeros(m), "requests": np.repeat(rng.integers(-1, 6, 20), -(-m // 20))[:m],
           "mixed": rng.integers(-1, 7, m), "none": np.full(m, 6), "last": np.full(m, 5)}[kind]
    say(f"adapters_backward rows {m} {kind}")
    c = _backward_case(m, 70, 90, 16, 6, BF16, F32, m, ids)
    _check_backward(c, pads=(0,))
    first = _run_backward(c)
    assert all(torch.equal(p, q) for p, q in zip(first, _run_backward(c)))


@pytest.mark.parametrize("rank", [3, 24, 40, 64, 65, 136])
@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_backward_ranks(rank, dtype):
    """Ranks in one, two and more workgroups, of several pieces each."""
    ids = np.arange(1500) * 9 // 1500 % 4 - 1
    say(f"adapters_backward ranks {rank} {dtype}")
    c = _backward_case(1500, 190, 260, rank, 3, dtype, dtype, rank, ids)
    _check_backward(c, pads=(0, 3))
    whole = _run_backward(c)
    for wanted in ((1, 0, 0), (0, 1, 1)):
        got = _run_backward(c, wanted=wanted, **({} if wanted[0] else {"base": None}))
        assert all(g is None or torch.equal(g, v) for g, v in zip(got, whole))


def test_adapters_backward_infinities():
    """An infinity among what is summed reaches its own sums and no others."""
    for dtype in TYPES:
        c = _backward_case(150, 100, 140, 16, 2, dtype, dtype, 5, ids=np.arange(150) % 3)
        clean = [t.cpu() for t in _run_backward(c)]
        c["x"][33, 7], c["hidden"][36, 2], c["dout"][39, 5] = math.inf, -math.inf, math.inf
        got = [t.cpu() for t in _run_backward(c)]
        rows, ranks, cols = torch.arange(150) != 39, torch.arange(16) != 2, torch.arange(100) != 5
        assert torch.equal(got[0][rows], clean[0][rows]) and not got[0][39].isfinite().any()
        assert torch.equal(got[1][1], clean[1][1]) and torch.equal(got[2][1], clean[2][1])
        assert not got[1][0].isfinite().any()  # dh of row 39 is not finite
        assert torch.equal(got[2][0][cols][:, ranks], clean[2][0][cols][:, ranks])
        assert not got[2][0][5].isfinite().any() and not got[2][0][:, 2].isfinite().any()


def test_adapters_backward_large_pieces():
    """Enough columns that a workgroup takes thousands of rows; integers, whose
    sums are exact, so that a wrong or missing row shows."""
    m, n, k = 9000, 5200, 2600
    rng = np.random.default_rng(5)
    ints = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).to(BF16).to(_dev())  # noqa: E731
    x, a, b, dout = ints(m, k), ints(3, 4, k), ints(3, n, 4), ints(m, n)
    ids = torch.from_numpy(np.repeat([1, 0, 1, -1, 2], m // 5).astype(np.int32)).to(_dev())
    hidden = ints(m, 4).float()
    dx, da, db = X.adapters_backward(dout, x, a, b, ids, hidden, base=torch.zeros(m, k, device=_dev()))
    for l in range(3):
        at = torch.nonzero(ids == l).flatten()
        dh = dout[at].double() @ b[l].double()
        assert torch.equal(dx[at].double(), dh @ a[l].double())
        assert torch.equal(da[l].double(), dh.t() @ x[at].double())
        assert torch.equal(db[l].double(), dout[at].double().t() @ hidden[at].double())


def test_adapters_backward_parts_and_places():
    c = _backward_case(200, 150, 130, 16, 3, BF16, BF16, 4)
    want = _run_backward(c)
    for wanted in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1), (1, 0, 1)):
        got = _run_backward(c, wanted=[bool(v) for v in wanted], **({} if wanted[0] else {"base": None}))
        for g, v, w in zip(got, want, wanted):
            assert (g is None) == (not w) and (g is None or torch.equal(g, v))
    assert _run_backward(c, wanted=(False,) * 3, base=None) == (None, None, None)
    store = torch.full((205, 140), -5.0, dtype=BF16, device=_dev())
    view = store[:200, 3:133]
    view.copy_(_up(c["base"]))
    got = _run_backward(c, base=view, out=view)
    assert got[0] is view and all(torch.equal(g, v) for g, v in zip(got, want))
    assert (store[200:] == -5).all() and (store[:, :3] == -5).all() and (store[:, 133:] == -5).all()
    bare = _run_backward(c, base=None)
    c["base"] = torch.zeros_like(c["base"])
    assert all(torch.equal(g, v) for g, v in zip(bare, _run_backward(c)))


def test_adapters_backward_is_not_reached_by_other_rows():
    """NaN in rows of other adapters, and of none, changes no gradient."""
    c = _backward_case(200, 150, 130, 16, 3, BF16, F32, 11, ids=np.arange(200) % 5 - 1)
    clean = [t.cpu() for t in _run_backward(c)]
    bad = np.isin(c["ids"], (1, 3, -1))
    for v in ("x", "dout", "hidden"):
        c[v][bad] = math.nan
    got = [t.cpu() for t in _run_backward(c)]
    good = torch.from_numpy(~bad)
    assert torch.equal(got[0][good], clean[0][good])
    for g, v in zip(got[1:], clean[1:]):
        assert torch.equal(g[[0, 2]], v[[0, 2]]) and g[1].isnan().all()


def test_adapters_gradients_against_differences():
    """Slopes of the forward call itself along random directions, in float32."""
    gen = torch.Generator(device=_dev()).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    m, n, k, rank, count = 50, 40, 70, 12, 3
    x, a, b, dout = r(m, k), r(count, rank, k) * 0.1, r(count, n, rank), r(m, n)
    ids = torch.arange(m, dtype=torch.int32, device=_dev()) % 4
    f = lambda *v: (X.adapters(*v, ids, scale=0.5).double() * dout.double()).sum()  # noqa: E731
    _, hidden = X.adapters(x, a, b, ids, scale=0.5, hidden=True)
    grads = X.adapters_backward(dout, x, a, b, ids, hidden, scale=0.5)
    for i, g in enumerate(grads):
        d = r(*g.shape)
        at = lambda t: [v + t * d if j == i else v for j, v in enumerate((x, a, b))]  # noqa: E731
        slope = (f(*at(0.5)) - f(*at(-0.5)))  # f is linear in each of them
        terms = (g.double() * d).abs().sum()
        assert abs(slope - (g.double() * d).sum()) < 1e-4 * terms


# ----- dropout -----------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (7, 8), (5, 100), (40, 257), (9, 2050), (2, 5001), (300, 9)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(rows, cols, dtype, residual):
    rng = np.random.default_rng(rows + cols)
    x, r = (torch.from_numpy(rng.standard_normal((rows, cols)) + 3).to(dtype) for _ in range(2))
    p, seed, offset = 0.3, -5 - (1 << 40), (7 << 35) + 11
    keep = ob.dropout_mask(rows, cols, p, seed, offset)
    factor = 65536 / (65536 - ob.threshold(p))
    want = _np(x) * keep * factor + (_np(r) if residual else 0)
    # the factor's rounding and the product's, the sum's, the type's
    tol = (2 * U32 * np.abs(_np(x)) * factor + U32 * np.abs(want)) * 1.01 + u(dtype) * np.abs(want) * 1.01 + least(dtype)
    say(f"dropout {rows} {cols} {dtype} {residual}")
    on_gpu = torch.tensor([seed], device=_dev())
    for pad in (0, 3, 8):
        v, res = _strided(x, pad), _strided(r, pad) if residual else None
        y = X.dropout(v, p, seed, offset=offset, residual=res)
        _close(_np(y), want, tol, pad)
        if residual:
            assert torch.equal(y.cpu()[torch.from_numpy(~keep)], r[torch.from_numpy(~keep)])
        else:
            assert np.array_equal(_np(y) != 0, keep)
        assert torch.equal(X.dropout(v, p, on_gpu, offset=offset, residual=res), y)
    for i, place in enumerate((x, r) if residual else (x,)):
        t = [_up(x), _up(r) if residual else None]
        assert X.dropout(t[0], p, seed, offset=offset, residual=t[1], out=t[i]) is t[i] and torch.equal(t[i], y)


def test_dropout_ends_of_p_and_special_values():
    x = torch.randn(50, 300, device=_dev())
    x[3], x[4] = math.nan, math.inf
    assert torch.equal(X.dropout(x, 0.0, 1)[5:], x[5:]) and torch.equal(X.dropout(x, 2.0 ** -18, 1)[5:], x[5:])
    assert not X.dropout(x, 1.0, 1).any() and torch.equal(X.dropout(x, 1.0, 1, residual=x[5:6].expand(50, 300).contiguous()),
                                                          x[5:6].expand(50, 300))
    y = X.dropout(x, 0.5, 9)
    keep = X.dropout(torch.ones_like(x), 0.5, 9) != 0
    assert torch.equal(y[3].isnan(), keep[3]) and torch.equal(y[4].isinf(), keep[4]) and not y[4][~keep[4]].any()
    assert X.dropout(x[:0], 0.5, 1).shape == (0, 300) and X.dropout(x[:, :0], 0.5, 1).shape == (50, 0)


def test_dropout_masks_differ_and_are_the_gradients():
    x = torch.ones(200, 1000, device=_dev())
    masks = [X.dropout(x, 0.25, s, offset=o) != 0 for s, o in ((1, 0), (2, 0), (1, 1), (1 + (1 << 32), 0), (1, 1 << 32))]
    n = x.numel()
    for i, p in enumerate(masks):
        # six deviations of a binomial count
        assert abs(p.sum().item() - 0.75 * n) < 6 * (n * 0.1875) ** 0.5
        for q in masks[:i]:
            assert abs((p & q).sum().item() - 0.5625 * n) < 6 * (n * 0.5625 * 0.4375) ** 0.5
    assert torch.equal(X.dropout(x, 0.25, (1 << 64) + 1) != 0, masks[0])
    assert torch.equal(X.dropout(x, 0.25, np.int64(1), offset=np.uint8(1)) != 0, masks[2])
    assert torch.equal(X.dropout(x, 0.25, np.int64(-1)), X.dropout(x, 0.25, torch.tensor([-1], device=_dev())))
    assert torch.equal(X.dropout(x[:, :501], 0.25, 1) != 0, masks[0][:, :501])
    assert torch.equal(X.dropout(x.bfloat16()[:77], 0.25, 1) != 0, masks[0][:77])
    dy = torch.randn_like(x)
    assert torch.equal(X.dropout(dy, 0.25, 1), torch.where(masks[0], dy * float(np.float32(4 / 3)), 0.0))


# ----- the operators together ---------------------------------------------------------

def _block(c, **more):
    """A block of a residual stream served and trained: everything once."""
    q, s, h, rstd = X.rms_norm_quantize(c["x"], c["w"], residual=c["res"], stats=True, **more)
    shared = X.fp8_gemm(q, s, c["wq"], c["ws"], **more)
    out = X.adapters(q, c["a"], c["b"], c["ids"], base=shared, scale=c["scale"], scale_x=s, **more)
    y, h2 = X.rms_norm(c["x"], c["w"], residual=c["res"], **more)
    out2, hidden = X.adapters(y, c["a"], c["b"], c["ids"], base=shared, scale=c["scale"], hidden=True, **more)
    stream = X.dropout(out2, 0.1, c["seed"], offset=3, residual=c["res2"], **more)
    dout = X.dropout(stream, 0.1, c["seed"], offset=3, **more)
    dy, da, db = X.adapters_backward(dout, y, c["a"], c["b"], c["ids"], hidden, scale=c["scale"], **more)
    dx, dw = X.rms_norm_backward(dy, h, rstd, c["w"], dresidual=c["x"], **more)
    return [q.float(), s, h, rstd, shared, out, y, h2, out2, hidden, stream, dout, dy, da, db, dx, dw]


def _block_inputs(m, seed=0):
    gen = torch.Generator(device=_dev()).manual_seed(m + seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    k, n = 640, 384
    wq, ws = X.fp8_quantize(r(n, k) * 0.05, block_rows=128)
    return dict(x=r(m, k).bfloat16(), res=r(m, k).bfloat16(), res2=r(m, n).bfloat16(), w=1 + 0.1 * r(k), wq=wq, ws=ws,
                a=(r(5, 16, k) * 0.04).bfloat16(), b=r(5, n, 16).bfloat16() * 0.1, scale=r(5),
                ids=(torch.arange(m, device=_dev()) * 7 // 3 % 6 - 1).int(), seed=torch.tensor([seed], device=_dev()))


@pytest.mark.parametrize("m", [1, 4, 300, 5000])
def test_block_against_float64(m):
    """The whole of it: each result against the oracle on what went into it."""
    c = _block_inputs(m)
    q, s, h, rstd, shared, out, y, h2, out2, hidden, stream, dout, dy, da, db, dx, dw = _block(c)
    assert torch.equal(h, h2)
    ids, scale, a, b = c["ids"].cpu().numpy(), _np(c["scale"]), _np(c["a"]), _np(c["b"])
    xq = ol.dequantize(ol.e4m3_encode(q.cpu().numpy()), s.cpu().numpy())
    for got, x in ((out, xq), (out2, _np(y))):
        want, hid = ob.adapters(x, a, b, ids, scale, _np(shared))
        mag, _ = ob.adapters(np.abs(x), np.abs(a), np.abs(b), ids, np.abs(scale), np.abs(_np(shared)))
        _close(_np(got), want, (2 * 640 + 200) * U32 * mag + u(BF16) * np.abs(want) * 1.01, "adapters")
    _close(_np(hidden), hid, (2 * 640 + 24) * U32 * ob.adapters(np.abs(_np(y)), np.abs(a), np.abs(b), ids, scale, 0 * want)[1] + 1e-30, "hidden")
    keep = (stream != c["res2"]).cpu().numpy()
    assert (keep & ~ob.dropout_mask(min(m, 40), 384, 0.1, 0, 3)[:m]).sum() == 0 if m <= 40 else True
    want = ob.adapters_backward(_np(dout), _np(y), a, b, ids, scale, _np(hidden), np.zeros((m, 640)))
    mag = ob.adapters_backward(np.abs(_np(dout)), np.abs(_np(y)), np.abs(a), np.abs(b), ids, np.abs(scale),
                               np.abs(_np(hidden)), np.zeros((m, 640)))
    for got, v, t, extra in zip((dy, da, db), want, mag, (u(BF16), 0, 0)):
        _close(_np(got), v, (2 * m + 2 * 384 + 200) * U32 * t + extra * np.abs(v) * 1.01 + 1e-30, "gradients")


@pytest.mark.parametrize("m", [1, 4, 300])
def test_block_on_another_stream(m):
    c = _block_inputs(m)
    want = _block(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _block(c)
    torch.cuda.synchronize()
    assert all(torch.equal(g, v) for g, v in zip(got, want))


@pytest.mark.parametrize("m", [1, 4, 300])
def test_block_in_graphs(m):
    """Two graphs of the same operators, replayed in turn with new inputs and
    new seeds, eager work between: workspaces and masks are each one's own."""
    cs = [_block_inputs(m, seed) for seed in (0, 50)]
    graphs, outs = [], []
    for c in cs:
        _block(c)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_block(c))
        graphs.append(graph)
    for turn in range(3):
        for c, seed in zip(cs, (10, 20)):
            new = _block_inputs(m, seed + turn)
            for v in ("x", "res", "res2", "ids", "seed", "a", "scale"):
                c[v].copy_(new[v])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, got in zip(cs, outs):
            want = _block(c)
            torch.cuda.synchronize()
            assert all(torch.equal(g, v) for g, v in zip(got, want))


def test_refusals():
    dev = _dev()
    z = lambda *s, **k: torch.zeros(*s, device=dev, **k)  # noqa: E731
    ids = lambda m, **k: z(m, dtype=k.get("dtype", torch.int32))  # noqa: E731
    q, s = X.fp8_quantize(z(4, 256))
    a, b, h = z(2, 8, 256), z(2, 30, 8), z(4, 8)
    for call, error in [
        (lambda: X.rms_norm(z(4)), ValueError),
        (lambda: X.rms_norm(z(4, 0)), ValueError),
        (lambda: X.rms_norm(z(4, 4), z(3)), ValueError),
        (lambda: X.rms_norm(z(4, 4, dtype=torch.float64)), TypeError),
        (lambda: X.rms_norm(z(4, 4), z(4, dtype=torch.float64)), TypeError),
        (lambda: X.rms_norm(z(4, 4), residual=z(4, 5)), ValueError),
        (lambda: X.rms_norm(z(4, 4), residual=z(4, 4, dtype=BF16)), ValueError),
        (lambda: X.rms_norm(z(4, 4), residual_out=z(4, 4)), ValueError),
        (lambda: X.rms_norm(z(4, 4), residual=z(4, 4), residual_out=z(3, 4)), ValueError),
        (lambda: X.rms_norm(z(4, 4), out=z(4, 5)), ValueError),
        (lambda: X.rms_norm(z(4, 4), residual=torch.zeros(4, 4)), ValueError),
        (lambda: X.rms_norm(z(4, 4), eps=-1.0), X.XposeError),
        (lambda: X.rms_norm(z(4, 8)[:, ::2]), ValueError),
        (lambda: (lambda t: X.rms_norm(t, residual=z(4, 4), out=t, residual_out=t))(z(4, 4)), X.XposeError),
        (lambda: X.rms_norm_quantize(z(4, 0)), ValueError),
        (lambda: X.rms_norm_quantize(z(4, 4), residual=z(5, 4)), ValueError),
        (lambda: X.rms_norm_backward(z(4, 4), z(4, 5), z(4)), ValueError),
        (lambda: X.rms_norm_backward(z(4, 4), z(4, 4), z(5)), ValueError),
        (lambda: X.rms_norm_backward(z(4, 4), z(4, 4), z(4, dtype=BF16)), TypeError),
        (lambda: X.rms_norm_backward(z(4, 4), z(4, 4), z(4), dresidual=z(4, 4, dtype=BF16)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(5)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4, dtype=torch.int64)), TypeError),
        (lambda: X.adapters(z(4, 255), a, b, ids(4)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b[:1], ids(4)), ValueError),
        (lambda: X.adapters(z(4, 256), a, z(2, 30, 7), ids(4)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b.half(), ids(4)), TypeError),
        (lambda: X.adapters(z(4, 256), a[0], b, ids(4)), ValueError),
        (lambda: X.adapters(z(4, 256, dtype=BF16), a, b, ids(4)), TypeError),
        (lambda: X.adapters(q, a, b, ids(4)), TypeError),
        (lambda: X.adapters(q, a, b, ids(4), scale_x=s[:1]), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), scale_x=s), TypeError),
        (lambda: X.adapters(q[:, 8:], a[:, :, 8:], b, ids(4), scale_x=s), X.XposeError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), base=z(4, 31)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), base=z(4, 30, dtype=BF16)), TypeError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), base=z(4, 30), out=z(4, 30, dtype=F16)), TypeError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), out=z(3, 30)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), scale=z(3)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), scale=z(2, dtype=BF16)), TypeError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4), scale=torch.ones(2)), ValueError),
        (lambda: X.adapters(z(4, 256), a, b, ids(4).cpu()), ValueError),
        (lambda: X.adapters(z(4, 256), z(2, 8, 512)[:, :, ::2], b, ids(4)), ValueError),
        (lambda: X.adapters_backward(z(5, 30), z(4, 256), a, b, ids(4), h), ValueError),
        (lambda: X.adapters_backward(z(4, 31), z(4, 256), a, b, ids(4), h), ValueError),
        (lambda: X.adapters_backward(z(4, 30), z(4, 256), a, b, ids(4), z(4, 7)), ValueError),
        (lambda: X.adapters_backward(z(4, 30), z(4, 256), a, b, ids(4), h.half()), TypeError),
        (lambda: X.adapters_backward(z(4, 30), z(4, 256), a, b, ids(4), z(4, 16)[:, :8]), ValueError),
        (lambda: X.adapters_backward(z(4, 30, dtype=BF16), z(4, 256), a, b, ids(4), h), TypeError),
        (lambda: X.adapters_backward(z(4, 30), z(4, 256), a, b, ids(4), h, base=z(4, 30)), ValueError),
        (lambda: X.adapters_backward(z(4, 30), z(4, 256), a, b, ids(4), h, base=z(4, 256), wanted=(False, True, True)), ValueError),
        (lambda: X.dropout(z(4, 4), 1.5, 1), X.XposeError),
        (lambda: X.dropout(z(4, 4), 0.5, z(1)), TypeError),
        (lambda: X.dropout(z(4, 4), 0.5, z(2, dtype=torch.int64)), ValueError),
        (lambda: X.dropout(z(4, 4), 0.5, torch.zeros(1, dtype=torch.int64)), ValueError),
        (lambda: X.dropout(z(4, 4), 0.5, 1, residual=z(4, 5)), ValueError),
        (lambda: X.dropout(z(4, 4), 0.5, 1, out=z(4, 4, dtype=BF16)), ValueError),
        (lambda: X.dropout(z(4, 4, dtype=torch.float64), 0.5, 1), TypeError),
    ]:
        with pytest.raises(error):
            call()
