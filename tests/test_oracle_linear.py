"""The oracle of the FP8 linear layer's operators against independent
sources: e4m3 against torch's type, the norm's gradient against differences."""
import numpy as np
import pytest

import oracle.linear as ol

torch = pytest.importorskip("torch")


def test_e4m3_decode_is_torchs_type():
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ol.e4m3_decode(bits), want, equal_nan=True)


def test_e4m3_encode_rounds_to_nearest_even():
    rng = np.random.default_rng(1)
    grid = ol.e4m3_decode(np.arange(127, dtype=np.uint8))
    ties = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, ties, np.nextafter(ties.astype(np.float32), np.float32(0)),
                        np.nextafter(ties.astype(np.float32), np.float32(1e9)),
                        np.exp(rng.uniform(-12, 6, 5000))]).astype(np.float32)
    x = np.concatenate([x, -x])
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ol.e4m3_encode(x), want)
    assert ol.e4m3_encode(np.float32([np.nan, 1e9, np.inf]))[0] & 127 == 127


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_stays_within_half_a_step(block_rows, pow2):
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((130, 200)) * np.exp(rng.uniform(-40, 40, (130, 1)))).astype(np.float32)
    x[3] = 0
    q, scale = ol.quantize(x, block_rows, pow2)
    assert scale.shape == (2, 130 if block_rows == 1 else 2)
    back = ol.dequantize(q, scale, block_rows)
    each = np.repeat(np.repeat(scale.T.astype(np.float64), block_rows, 0), 128, 1)[:130, :200]
    # half a step: 2^-4 of a value with three mantissa bits, 2^-10 scales below
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * each)).all()
    if pow2:
        assert (np.frexp(scale)[0] == 0.5).all()


def test_backward_is_the_differences_of_the_forward():
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((3, 17)), rng.standard_normal((3, 17))
    w, b = rng.standard_normal(17), rng.standard_normal(17)
    _, mean, rstd = ol.layer_norm(x, w, b, 1e-5)
    dx, dw, db = ol.layer_norm_backward(dy, x, mean, rstd, w)
    loss = lambda x, w, b: (ol.layer_norm(x, w, b, 1e-5)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for grad, arg in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        for at in np.ndindex(grad.shape):
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[arg][at] -= h
            hi[arg][at] += h
            # differences of second order: h^2 of a third derivative, and
            # the loss's rounding over h
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - grad[at]) < 1e-7


def test_clip():
    norm, factor = ol.clip([np.float32([3, 0]), np.zeros((0,)), np.float32([[4]])], 1.0, 0.0)
    assert norm == 5 and factor == 0.2
    assert ol.clip([np.float32([0.5])], 1.0, 1e-6)[1] == 1.0
