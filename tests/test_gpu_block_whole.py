"""A residual block's operators together, every result of them against the
oracle, and adapters in numbers that earlier tests do not reach: more than a
wave's lanes of them, one for each row, ranks over 32 next to few rows."""
import numpy as np
import pytest

import oracle.block as ob
import oracle.linear as ol
from test_gpu_block import (BF16, F16, F32, TYPES, U32, _adapter_case, _backward_case, _block, _block_inputs,
                            _check_adapters, _check_backward, _close, _dev, _norm_tol, _np, _run_backward, _terms, least, u)
from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")


@pytest.mark.parametrize("m", [1, 4, 40, 300, 5000])
def test_block_values(m):
    """What of the block the oracle has not been asked for elsewhere: the norm
    both ways, the 8-bit product, dropout on the output and on the gradient."""
    c = _block_inputs(m)
    say(f"block {m}")
    q, s, h, rstd, shared, out, y, h2, out2, hidden, stream, dout, dy, da, db, dx, dw = _block(c)
    assert torch.equal(h, (c["x"].float() + c["res"].float()).bfloat16()) and torch.equal(h2, h)
    k, w = 640, _np(c["w"])
    want, r = ob.rms_norm(_np(h), w, 1e-5)
    _close(_np(rstd), r, r * (_terms(k) / 2 + 5) * U32, "rstd")
    _close(_np(y), want, _norm_tol(want, k, BF16), "y")
    # e4m3: half a step of a block's scale at its largest, 2^-4 relative at the most, beside y's float32 error
    xq = ol.dequantize(ol.e4m3_encode(q.cpu().numpy()), s.cpu().numpy())
    blocks = np.repeat(_np(s).T, 128, axis=1)[:, :k]
    _close(xq, want, np.maximum(2.0 ** -4 * np.abs(want), blocks * 2.0 ** -10) * 1.01 + np.abs(want) * (_terms(k) / 2 + 8) * U32,
           "quantised")
    wq = ol.dequantize(ol.e4m3_encode(c["wq"].float().cpu().numpy()), c["ws"].cpu().numpy(), 128)
    product = xq @ wq.T
    # products exact in float32, sums of 640 that may cut, a block's scales and its addition
    _close(_np(shared), product, (2 * k + 40) * U32 * (np.abs(xq) @ np.abs(wq.T)) + u(BF16) * np.abs(product) * 1.01, "shared")

    # dropout of the output with the residual's addition, and of the gradient: the same mask
    keep, factor = np.zeros((m, 384), bool), 65536 / (65536 - ob.threshold(0.1))
    rows = np.arange(m)
    rows = rows[(rows < 14) | (rows >= m - 14) | (np.abs(rows - m // 2) < 7)]
    for row in rows:
        keep[row] = ob.dropout_mask(1, 384, 0.1, 0, 3, int(row))
    res2, o = _np(c["res2"])[rows], _np(out2)[rows]
    for got, v, extra in ((stream, o, res2), (dout, _np(stream)[rows], 0 * res2)):
        want = keep[rows] * v * factor + extra
        tol = (2 * U32 * np.abs(v) * factor + U32 * np.abs(want)) * 1.01 + u(BF16) * np.abs(want) * 1.01 + least(BF16)
        _close(_np(got)[rows], want, tol, "dropout")
        assert np.array_equal(_np(got)[rows][~keep[rows]], extra[~keep[rows]])
    # and everywhere the two agree with each other, with a share of 0.1 dropped within six deviations
    where = X.dropout(torch.ones_like(out2), 0.1, 0, offset=3) != 0
    assert torch.equal(dout != 0, where & (stream != 0))
    assert torch.equal(stream[~where], c["res2"][~where])
    assert abs(where.sum().item() - m * 384 / factor) < 6 * (m * 384 * 0.09) ** 0.5

    # the norm's backward pass, with the residual stream's gradient
    r64, hd, g = _np(rstd)[:, None], _np(h), _np(dy) * w
    want, dwant = ob.rms_norm_backward(_np(dy), hd, _np(rstd), w, _np(c["x"]))
    xhat, d = np.abs(hd * r64), (_terms(k) + 4) * U32
    along = np.abs((g * hd * r64).mean(1, keepdims=True))
    tol = r64 * (3 * U32 * np.abs(g) + xhat * (d * (np.abs(g) * xhat).mean(1, keepdims=True) + 5 * U32 * along))
    tol = (tol + 2 * U32 * (np.abs(want) + np.abs(_np(c["x"])))) * 1.01 + u(BF16) * np.abs(want) * 1.01 + least(BF16)
    _close(_np(dx), want, tol, "dx")
    _close(_np(dw), dwant, (m + 40) * U32 * np.abs(_np(dy) * hd * r64).sum(0) + least(F32), "dweight")


# ----- many adapters -------------------------------------------------------------------

def _ids(kind, m, count):
    """Rows of each adapter: of all, of the first and last alone, of several
    pieces beside one of none; in any order."""
    rng = np.random.default_rng(m + count)
    if kind == "any":
        ids = rng.integers(-1, count + 1, m)
    elif kind == "ends":
        ids = rng.choice([0, count - 1], m)
    elif kind == "middle":
        ids = np.full(m, count // 2)
        ids[::7] = rng.integers(0, count, len(ids[::7]))
    else:
        ids = np.arange(m) % count
    return ids


@pytest.mark.parametrize("count", [63, 64, 65, 127, 130, 1000, 4100, 65535])
@pytest.mark.parametrize("kind", ["any", "ends", "middle", "each"])
@pytest.mark.parametrize("m", [300, 3000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_of_many_adapters(count, kind, m, dtype):
    """Integers, whose sums are exact: a row that is missed, or taken for
    another adapter, shows; adapters of no row get zeros."""
    n, k, rank = 24, 16, 5
    gen = torch.Generator(device=_dev()).manual_seed(count)
    ints = lambda *s: torch.randint(-3, 4, s, generator=gen, device=_dev())  # noqa: E731
    x, dout, a, b = (ints(*s).to(dtype) for s in ((m, k), (m, n), (count, rank, k), (count, n, rank)))
    hidden = ints(m, rank).float()
    ids = torch.from_numpy(_ids(kind, m, count).astype(np.int32)).to(_dev())
    say(f"gradients of many adapters {count} {kind} {m} {dtype}")
    dx, da, db = X.adapters_backward(dout, x, a, b, ids, hidden, base=torch.zeros(m, k, device=_dev()))
    mine = (ids >= 0) & (ids < count)
    at = ids[mine].long()
    do, xs, hs = dout[mine].double(), x[mine].double(), hidden[mine].double()
    dh = (do[:, :, None] * b[at].double()).sum(1)
    want = torch.zeros(m, k, dtype=torch.float64, device=_dev())
    want[mine] = (dh[:, :, None] * a[at].double()).sum(1)
    assert torch.equal(dx.double(), want)
    want = torch.zeros(count, rank, k, dtype=torch.float64, device=_dev()).index_add_(0, at, dh[:, :, None] * xs[:, None])
    assert torch.equal(da.double(), want)
    want = torch.zeros(count, n, rank, dtype=torch.float64, device=_dev()).index_add_(0, at, do[:, :, None] * hs[:, None])
    assert torch.equal(db.double(), want)
    out, h = X.adapters(x, a, b, ids, base=torch.zeros(m, n, device=_dev()), hidden=True)
    hw = (a[at].double() * xs[:, None]).sum(2)
    assert torch.equal(h[mine].double(), hw) and not h[~mine].any()
    assert torch.equal(out[mine].double(), (b[at].double() * hw[:, None]).sum(2)) and not out[~mine].any()


@pytest.mark.parametrize("m", [17, 64, 128, 200, 256, 512])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("quantized", [False, True])
def test_a_row_of_each_request(m, dtype, out, quantized):
    """A token of each of many requests, every one with an adapter of its own."""
    say(f"a row of each request {m} {dtype} {quantized}")
    ids = np.random.default_rng(m).permutation(m)
    _check_adapters(_adapter_case(m, 300, 700, 16, m, dtype, out, m, quantized, ids), pads=(0,))


@pytest.mark.parametrize("m", [64, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_backward_of_a_row_of_each_request(m, dtype):
    ids = np.random.default_rng(m).permutation(m)
    say(f"backward of a row of each request {m} {dtype}")
    _check_backward(_backward_case(m, 130, 200, 16, m, dtype, dtype, m, ids=ids), pads=(0,))


@pytest.mark.parametrize("m", [1, 5, 16])
@pytest.mark.parametrize("rank", [33, 40, 64, 100])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F32), (BF16, BF16)])
@pytest.mark.parametrize("quantized", [False, True])
def test_few_rows_of_high_rank(m, rank, dtype, out, quantized):
    """B's operands are loaded anew for each 32 ranks, hidden comes in slices."""
    say(f"few rows of high rank {m} {rank} {dtype} {quantized}")
    ids = np.arange(m) % 7 - 1 if m > 1 else [3]
    _check_adapters(_adapter_case(m, 600, 4200, rank, 6, dtype, out, m + rank, quantized, ids), pads=(0,))


@pytest.mark.parametrize("m", [1, 5, 16])
@pytest.mark.parametrize("rank", [33, 64, 100])
@pytest.mark.parametrize("dtype", TYPES)
def test_backward_of_few_rows_of_high_rank(m, rank, dtype):
    say(f"backward of few rows of high rank {m} {rank} {dtype}")
    ids = np.arange(m) % 7 - 1 if m > 1 else [3]
    _check_backward(_backward_case(m, 300, 600, rank, 6, dtype, dtype, m + rank, ids=ids), pads=(0,))


@pytest.mark.parametrize("m,count", [(33, 31), (33, 32), (64, 32), (65, 40), (500, 300), (700, 33)])
@pytest.mark.parametrize("rank", [16, 40])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F16, F32), (BF16, BF16)])
def test_many_adapters_of_several_tiles(m, count, rank, dtype, out):
    """More rows than a tile, adapters one after the other and in any order,
    forward and (dx alone too) backward."""
    say(f"many adapters of several tiles {m} {count} {rank} {dtype}")
    for ids in (np.arange(m) * count // m, np.random.default_rng(m).integers(-1, count, m)):
        _check_adapters(_adapter_case(m, 270, 200, rank, count, dtype, out, m, ids=ids), pads=(0, 3))
        c = _backward_case(m, 140, 270, rank, count, dtype, out, m, ids=ids)
        _check_backward(c, pads=(0,))
        whole, alone = _run_backward(c), _run_backward(c, wanted=(True, False, False))
        assert torch.equal(alone[0], whole[0])
