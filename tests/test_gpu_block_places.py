"""Adapters whose result goes over their own input: a residual connection in
place, forward and backward.  The same bits as into a tensor of its own, for
every gradient."""
import pytest

from test_gpu_block import BF16, F16, F32, _backward_case, _up
from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

# one launch of dx and the gradients or two; rows of one piece and of several; shorter than a load
SIZES = [(40, 6, 4, 2), (300, 257, 16, 3), (300, 640, 40, 2), (5000, 1024, 16, 4), (3000, 1024, 32, 2), (3000, 512, 72, 2)]


def _case(m, k, rank, count, dtype):
    c = _backward_case(min(m, 64), k, k, rank, count, dtype, dtype, m + k)
    gen = torch.Generator().manual_seed(m)
    for v in ("x", "dout"):
        c[v] = torch.randn(m, k, generator=gen).to(dtype)
    c["hidden"] = torch.randn(m, rank, generator=gen)
    c["ids"] = torch.randint(-1, count, (m,), generator=gen).int()
    return {v: _up(t) if v != "xs" else None for v, t in c.items()}


@pytest.mark.parametrize("m,k,rank,count", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("over", ["dout", "x"])
def test_backward_over_what_it_reads(m, k, rank, count, dtype, over):
    c = _case(m, k, rank, count, dtype)
    say(f"adapters_backward over {over} {m} {k} {rank} {count} {dtype}")
    back = lambda base, out=None, **more: X.adapters_backward(  # noqa: E731
        c["dout"], c["x"], c["a"], c["b"], c["ids"], c["hidden"], base=base, scale=c["scale"], out=out, **more)
    before = c[over].clone()
    want = back(c[over].clone())
    got = back(c[over], c[over])
    assert got[0] is c[over]
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    for wanted in ((True, False, False), (True, True, False), (True, False, True)):
        c[over].copy_(before)
        got = back(c[over], c[over], wanted=wanted)
        assert all(g is None or torch.equal(g, v) for g, v in zip(got, want))


@pytest.mark.parametrize("m,k,rank,count", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("hidden", [False, True])
def test_forward_over_its_input(m, k, rank, count, dtype, hidden):
    c = _case(m, k, rank, count, dtype)
    say(f"adapters over x {m} {k} {rank} {count} {dtype} {hidden}")
    run = lambda base, out=None: X.adapters(c["x"], c["a"], c["b"], c["ids"], base=base, scale=c["scale"],  # noqa: E731
                                            hidden=hidden, out=out)
    want = run(c["x"].clone())
    got = run(c["x"], c["x"])
    for g, v in zip(got, want) if hidden else ((got, want),):
        assert torch.equal(g, v)
    assert (got[0] if hidden else got) is c["x"]


def test_backward_over_dout_in_a_graph():
    c = _case(3000, 1024, 16, 4, BF16)
    dout = c["dout"].clone()
    step = lambda: X.adapters_backward(c["dout"], c["x"], c["a"], c["b"], c["ids"], c["hidden"],  # noqa: E731
                                       base=c["dout"], scale=c["scale"], out=c["dout"])
    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        c["dout"].copy_(dout)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))
        assert torch.randn(1000, device="cuda").isfinite().all()
