"""An output may be the input that its call names, and no other input that lies
at the same address: each such call comes back before anything is launched
(addresses are made up and never dereferenced)."""
import pytest

from test_abi_block import A, BF16, D, E, EALIAS, F32, G, adapt, back, norm

# one row, so that a vector is a matrix of the same range and pitch
NORM = dict(rows=1, ldx=300, dtype=F32, pd=F32)
ONE = dict(m=1, k=16, rank=16, ldx=16, lda=16, ldb=16, dtype=F32, od=F32, sa=256, sb=300 * 16)


@pytest.mark.parametrize("args", [
    dict(NORM, x=A, h=A, w=A), dict(NORM, x=A, y=A, w=A), dict(NORM, res=A, h=A, w=A)])
def test_norm_over_its_weight(args):
    assert norm(**args) == EALIAS


@pytest.mark.parametrize("args", [
    # base and out are the adapters' scales, or B
    dict(m=1, n=5, dtype=F32, od=F32, ldbase=5, ldout=5, sb=80, base=D, out=D, scale=D),
    dict(m=16, n=16, count=1, base=E, out=E, b=E, ldbase=16, ldout=16, od=BF16)])
def test_adapters_over_their_weights(args):
    assert adapt(**args) == EALIAS


@pytest.mark.parametrize("args", [
    # base and dx are hidden, A, B or the scales
    dict(ONE, ldbase=16, lddx=16, base=E, dx=E, hidden=E),
    dict(m=16, count=1, base=E, dx=E, a=E),
    dict(m=300, k=16, n=300, ldx=16, lda=16, count=1, ldbase=16, lddx=16, base=E, dx=E, b=E),
    dict(m=1, k=5, ldx=5, lda=5, dtype=F32, od=F32, sa=80, ldbase=5, lddx=5, base=D, dx=D, scale=D),
    # dx is base, but x and dout only begin there
    dict(m=200, base=E, dx=E, x=E, ldx=257), dict(m=200, base=E, dx=E, dout=E),
    # dx is x or dout without base
    dict(base=None, dx=A), dict(n=256, lddout=256, ldb=16, sb=256 * 16, base=None, dout=G + (1 << 30), dx=G + (1 << 30))])
def test_adapters_backward_over_other_inputs(args):
    assert back(**args) == EALIAS
