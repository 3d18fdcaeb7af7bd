"""The 8-bit product's scales at the ends of their range, and special values,
through every kernel: few rows, 128 x 128 and 256 x 256 tiles, 16-bit results
(the matrix cores' 8-bit instructions) and float32 ones."""
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


def _gemm(qa, sa, qb, sb, dtype, pow2):
    def e4m3(bits):
        rows, cols = bits.shape
        store = torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.uint8, device=_dev())
        store[:, :cols] = torch.from_numpy(bits).to(_dev())
        return store.view(torch.float8_e4m3fn)[:, :cols]
    up = lambda s: torch.from_numpy(s).to(_dev())  # noqa: E731
    return X.fp8_gemm(e4m3(qa), up(sa), e4m3(qb), up(sb), out_dtype=dtype, pow2=pow2).cpu().double().numpy()


# few rows, 128 x 128 tiles, 256 x 256 tiles (16-bit results)
SIZES = [(3, 50, 400), (40, 70, 300), (150, 200, 400), (3901, 4090, 390)]


def _check(m, n, k, ops, block_rows, pow2, dtypes=(F32, BF16)):
    """Against float64.  Tolerances: k products in sums that may cut, a scaling
    and an addition a block; for 16-bit results products cut under 2^-13 of the
    largest of 8 (8 * 2^-13 of it); the result's rounding; and what lies under
    float32's and the type's normal numbers, which may be flushed.  Past the
    type's largest number the result is inf."""
    want, mag = ol.gemm(*ops, block_rows)
    for dtype in dtypes:
        got = _gemm(*ops, dtype, pow2)
        tol = (2 * k + 4) * U32 * mag + u(dtype) * np.abs(want) + (-(-k // 128) + 1) * 2.0 ** -126
        if dtype != F32:
            tol = tol + 2.0 ** -10 * mag
        tol = tol * (1 + u(dtype))
        over = (got == np.copysign(np.inf, want)) & (np.abs(want) + tol >= torch.finfo(dtype).max)
        bad = ~((np.abs(got - want) <= tol) | over)
        assert not bad.any(), (dtype, int(bad.sum()), got[bad][:3], want[bad][:3])


def _scales(rng, shape, exponent, pow2):
    s = np.full(shape, 2.0 ** exponent)
    return (s if pow2 else s * rng.uniform(1, 2, shape)).astype(np.float32)


def _shapes(m, n, k, block_rows):
    kb = -(-k // 128)
    return (kb, m), (kb, n if block_rows == 1 else -(-n // 128))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("ea,eb", [(-72, -72), (-100, -43), (-43, -100), (-100, 100), (100, -100), (60, 40), (100, 2)])
def test_scales_of_any_size(m, n, k, block_rows, pow2, ea, eb):
    """Values of 256 to 448, so that a block's sum is near 2^24: results are
    normal numbers where the scales' product is not (and past them at the other
    end)."""
    rng = np.random.default_rng(m + 3 * block_rows)
    say(f"scales {m} {n} {k} {block_rows} {pow2} {ea} {eb}")
    values = lambda r: ol.e4m3_encode(rng.uniform(256, 448, (r, k)).astype(np.float32))  # noqa: E731
    shape_a, shape_b = _shapes(m, n, k, block_rows)
    ops = values(m), _scales(rng, shape_a, ea, pow2), values(n), _scales(rng, shape_b, eb, pow2)
    _check(m, n, k, ops, block_rows, pow2)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("ea,eb", [(-72, -72), (-90, -54), (-54, -90)])
def test_scales_whose_product_is_under_float32s_normal_numbers(m, n, k, block_rows, ea, eb):
    """All values 256: a block's sum is 2^23 or less and every step of the right
    result exact, though the scales' product has more bits than float32 keeps."""
    say(f"exact scales {m} {n} {k} {block_rows} {ea} {eb}")
    shape_a, shape_b = _shapes(m, n, k, block_rows)
    sa = np.full(shape_a, (1 + 2.0 ** -6) * 2.0 ** ea, np.float32)
    sb = np.full(shape_b, (1 + 2.0 ** -3) * 2.0 ** eb, np.float32)
    v = ol.e4m3_encode(np.full((1, 1), 256, np.float32))[0, 0]
    qa, qb = np.full((m, k), v, np.uint8), np.full((n, k), v, np.uint8)
    want = 2.0 ** 16 * k * (1 + 2.0 ** -6) * (1 + 2.0 ** -3) * 2.0 ** (ea + eb)
    assert (_gemm(qa, sa, qb, sb, F32, False) == want).all()
    assert (_gemm(qa, sa, qb, sb, BF16, False) == torch.tensor(want, dtype=torch.float64).to(BF16).item()).all()


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_scales_whose_product_is_past_float32(m, n, k, block_rows, pow2):
    """The product of the first block's scales is over 2^128, but its values
    are 0 in a, or so small that the result is finite."""
    rng = np.random.default_rng(7 + m)
    say(f"large scales {m} {n} {k} {block_rows} {pow2}")
    qa = ol.e4m3_encode(rng.standard_normal((m, k)).astype(np.float32))
    qb = ol.e4m3_encode(rng.standard_normal((n, k)).astype(np.float32))
    shape_a, shape_b = _shapes(m, n, k, block_rows)
    sa, sb = _scales(rng, shape_a, 0, pow2), _scales(rng, shape_b, 0, pow2)
    sa[0], sb[0] = _scales(rng, m, 75, pow2), _scales(rng, shape_b[1], 55, pow2)
    qa[:, :128] = 0
    _check(m, n, k, (qa, sa, qb, sb), block_rows, pow2)
    qa[:, 5], qb[:, :128] = 1, 0
    qb[:, 5] = 1  # 2^-9 times 2^-9, the only product of the block
    _check(m, n, k, (qa, sa, qb, sb), block_rows, pow2)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_scales_of_zero_and_below_it(m, n, k, block_rows):
    """Scales of one's own making: 0 takes a block out, negative ones count."""
    rng = np.random.default_rng(9 + m)
    say(f"zero scales {m} {n} {k} {block_rows}")
    qa = ol.e4m3_encode(rng.standard_normal((m, k)).astype(np.float32))
    qb = ol.e4m3_encode(rng.standard_normal((n, k)).astype(np.float32))
    shape_a, shape_b = _shapes(m, n, k, block_rows)
    sa = rng.uniform(-2, 2, shape_a).astype(np.float32)
    sb = rng.uniform(-2, 2, shape_b).astype(np.float32)
    sa[0, ::2], sb[1, :] = 0, 0
    _check(m, n, k, (qa, sa, qb, sb), block_rows, False, (F32, BF16, F16))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_special_values(m, n, k, block_rows, pow2, dtype):
    """NaN elements, and scales of inf and NaN in either operand, reach the
    outputs that use them and no others."""
    rng = np.random.default_rng(11)
    say(f"special {m} {n} {k} {block_rows} {pow2} {dtype}")
    ops = ol.quantize(rng.standard_normal((m, k)) + 3, 1, pow2) + ol.quantize(rng.standard_normal((n, k)), block_rows, pow2)
    qa, sa, qb, sb = ops
    qa[1, 130], qb[7, 2] = 0x7f, 0xff
    sa[1, 2], sa[0, 0] = np.inf, np.nan
    sb[0, 0] = np.inf
    got = _gemm(*ops, dtype, pow2)
    per = block_rows
    bad = np.zeros((m, n), bool)
    bad[:2] = True  # a NaN element; a NaN scale
    bad[2] = True   # an infinite scale, of values that are not 0
    bad[:, 7] = True
    bad[:, :per] = True
    assert not np.isfinite(got[bad]).any()
    assert np.isfinite(got[~bad]).all()
    assert np.isnan(got[:2]).all() and np.isnan(got[:, 7]).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_rows_past_32_bits(block_rows):
    """b's last rows start over 2^32 bytes into their buffer; 16-bit results."""
    n, k, pitch = 520, 256, (1 << 23) - 16
    rng = np.random.default_rng(11)
    store = torch.zeros(n * pitch, dtype=torch.uint8, device=_dev())
    b = ol.quantize(rng.standard_normal((n, k)), block_rows)
    view = torch.as_strided(store, (n, k), (pitch, 1))
    view.copy_(torch.from_numpy(b[0]))
    sb = torch.from_numpy(b[1]).to(_dev())
    near = torch.from_numpy(b[0]).to(_dev()).view(torch.float8_e4m3fn)
    for m in (4, 90):
        a = [torch.from_numpy(t).to(_dev()) for t in ol.quantize(rng.standard_normal((m, k)))]
        say(f"far rows m {m} {block_rows}")
        got = X.fp8_gemm(a[0].view(torch.float8_e4m3fn), a[1], view.view(torch.float8_e4m3fn), sb)
        assert torch.equal(got, X.fp8_gemm(a[0].view(torch.float8_e4m3fn), a[1], near, sb))
