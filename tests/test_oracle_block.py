"""The oracle of a residual block's operators against torch's autograd in
float64 and the generator's published vectors."""
import numpy as np
import pytest

import oracle.block as ob

torch = pytest.importorskip("torch")


def test_rms_norm_and_its_gradients():
    gen = torch.Generator().manual_seed(1)
    h = torch.randn(5, 12, generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn(12, generator=gen, dtype=torch.float64, requires_grad=True)
    dy, res = torch.randn(2, 5, 12, generator=gen, dtype=torch.float64)
    rstd = (h.square().mean(1) + 1e-3).rsqrt()
    y = h * rstd[:, None] * w
    ((y * dy).sum() + (h * res).sum()).backward()
    got, r = ob.rms_norm(h.detach().numpy(), w.detach().numpy(), 1e-3)
    assert np.allclose(got, y.detach().numpy(), atol=1e-14) and np.allclose(r, rstd.detach().numpy())
    dx, dw = ob.rms_norm_backward(dy.numpy(), h.detach().numpy(), r, w.detach().numpy(), res.numpy())
    assert np.allclose(dx, h.grad.numpy(), atol=1e-13) and np.allclose(dw, w.grad.numpy(), atol=1e-13)


def test_adapters_and_their_gradients():
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64, requires_grad=True)  # noqa: E731
    x, a, b, base = r(7, 6), r(3, 2, 6), r(3, 5, 2), r(7, 5)
    ids = [2, 0, -1, 2, 3, 0, 2]
    scale = np.array([0.5, 2.0, -1.5])
    dout, dbase = torch.randn(7, 5, generator=gen, dtype=torch.float64), np.ones((7, 6))
    rows = []
    for i, l in enumerate(ids):
        rows.append(base[i] + (scale[l] * (b[l] @ (a[l] @ x[i])) if 0 <= l < 3 else 0))
    out = torch.stack(rows)
    (out * dout).sum().backward()
    n = lambda t: t.detach().numpy()  # noqa: E731
    got, hidden = ob.adapters(n(x), n(a), n(b), ids, scale, n(base))
    assert np.allclose(got, n(out), atol=1e-13)
    dx, da, db, _ = ob.adapters_backward(n(dout), n(x), n(a), n(b), ids, scale, hidden, dbase)
    for g, t in ((dx - 1, x), (da, a), (db, b)):
        assert np.allclose(g, t.grad.numpy(), atol=1e-12)


def test_philox_known_answers():
    """The method's published vectors for all zeros and all ones."""
    assert ob.philox((0,) * 4, (0,) * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = 0xFFFFFFFF
    assert ob.philox((ones,) * 4, (ones,) * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]


def test_dropout_mask():
    assert ob.dropout_mask(3, 20, 0.0, 1, 2).all() and not ob.dropout_mask(3, 20, 1.0, 1, 2).any()
    m = ob.dropout_mask(40, 500, 0.25, 77, 1 << 40)
    n = m.size
    assert abs((~m).sum() - n / 4) < 6 * (n * 0.25 * 0.75) ** 0.5
    assert np.array_equal(ob.dropout_mask(2, 500, 0.25, 77, 1 << 40, row0=3), m[3:5])
    assert not np.array_equal(ob.dropout_mask(40, 500, 0.25, 77, 1), m)
    assert ob.threshold(0.1) == 6554 and ob.threshold(1 - 2.0 ** -17) == 65536
