"""How many workgroups a root-mean-square norm takes depends on the rows' number
and bytes; what it gives does not: the same bits as the same rows in shares, at
widths and numbers on both sides of where that changes."""
import pytest

from test_gpu_block import BF16, F16, F32, _dev
from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")


@pytest.mark.parametrize("rows,cols", [(4096, 7680), (4095, 7680), (4100, 7679), (4096, 7500), (4200, 8184), (4097, 4608),
                                       (700, 4609), (700, 4600), (16384, 1920), (16383, 1920), (16400, 1900),
                                       (1500, 3500), (16384, 1250), (8192, 5000), (9000, 4100), (1100, 9001)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_in_shares(rows, cols, dtype, residual):
    gen = torch.Generator(device=_dev()).manual_seed(cols)
    x, r = (torch.randn(rows, cols, generator=gen, device=_dev()).to(dtype) for _ in range(2))
    w = torch.randn(cols, generator=gen, device=_dev())
    res = lambda at: dict(residual=r[at]) if residual else {}  # noqa: E731
    say(f"rms_norm in shares {rows} {cols} {dtype} {residual}")
    whole = X.rms_norm(x, w, stats=True, **res(slice(None)))
    for at in range(0, rows, 255):
        at = slice(at, at + 255)
        assert all(torch.equal(g, v[at]) for g, v in zip(X.rms_norm(x[at], w, stats=True, **res(at)), whole))
    got = X.rms_norm(x, w, stats=True, out=r if residual else x, residual_out=x if residual else None, **res(slice(None)))
    assert all(torch.equal(g, v) for g, v in zip(got, whole))
