"""``transpose``, ``copy`` and ``sgemm`` with the ``stream`` argument: whose
memory they use and what they wait for."""
import types

import pytest

from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

SPIN = 5_000_000  # cycles that queued work waits for


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


def _inputs():
    gen = torch.Generator(device=_dev()).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    return types.SimpleNamespace(x=r(300, 517), a=r(64, 200), b=r(200, 96), long_a=r(128, 8192), long_b=r(8192, 128))


CALLS = {
    "transpose": lambda i, **k: X.transpose(i.x, **k),
    "sgemm": lambda i, **k: X.sgemm(i.a, i.b, **k),
    "sgemm in slices": lambda i, **k: X.sgemm(i.long_a, i.long_b, split_k=16, **k),
}


def _pool(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_given_stream(name):
    i = _inputs()
    torch.cuda.synchronize()
    say(f"pool {name}")
    side = torch.cuda.Stream()
    got = CALLS[name](i, stream=side)
    torch.cuda.synchronize()
    assert _pool(got) == side.cuda_stream != torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("name", CALLS)
def test_memory_that_queued_work_still_uses_is_not_written(name):
    """The current stream has work queued on blocks that were freed on the
    host, of the sizes that the call allocates."""
    i = _inputs()
    want = CALLS[name](i)
    torch.cuda.synchronize()
    say(f"queued work {name}")
    side = torch.cuda.Stream()
    torch.cuda._sleep(SPIN)
    sizes = (want.untyped_storage().nbytes(), 1 << 16, 1 << 20, 1 << 22)
    blocks = [torch.empty(n, dtype=torch.uint8, device=_dev()) for n in sizes]
    ends = []
    for fill, t in enumerate(blocks):
        t.fill_(fill + 1)
        ends.append((t.min().clone(), t.max().clone()))
    del blocks, t
    got = CALLS[name](i, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for fill, (lo, hi) in enumerate(ends):
        assert lo.item() == hi.item() == fill + 1


@pytest.mark.parametrize("name", CALLS)
def test_inputs_outlive_the_calls_work(name):
    """Inputs that the caller drops are not given out again before the given
    stream has read them."""
    i = _inputs()
    want = CALLS[name](i)
    torch.cuda.synchronize()
    say(f"inputs {name}")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    got = CALLS[name](i, stream=side)
    sizes = [t.numel() for t in vars(i).values()]
    del i
    for n in sizes:
        torch.full((n,), 7.0, device=_dev())
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_copy_keeps_its_tensors():
    src, dst = torch.randn(5000, device=_dev()), torch.zeros(5000, device=_dev())
    want = src.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    X.copy(dst, src, stream=side)
    del src
    torch.full((5000,), 7.0, device=_dev())
    torch.cuda.synchronize()
    assert torch.equal(dst, want)


def test_a_stream_by_its_handle():
    i = _inputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, call in CALLS.items():
        got = call(i, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
        side.synchronize()
        assert torch.equal(got, call(i)), name
