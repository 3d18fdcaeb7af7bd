"""The FP8 linear layer's operators with the ``stream`` argument: whose memory
they use, what they wait for, and what they refuse."""
import types

import numpy as np
import pytest

from xpose_testlib import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")

F32, BF16 = torch.float32, torch.bfloat16
SPIN = 5_000_000  # cycles that queued work waits for


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


def _inputs(m):
    gen = torch.Generator(device=_dev()).manual_seed(m)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    x = r(m, 1000).to(BF16)
    w, b = r(1000), r(1000)
    q, s = X.fp8_quantize(x)
    wq, ws = X.fp8_quantize(r(300, 1000), block_rows=128)
    long_a, long_b = X.fp8_quantize(r(m, 8200)), X.fp8_quantize(r(90, 8200))
    _, mean, rstd = X.layer_norm(x, w, b, stats=True)
    grads = [r(m, 100).to(BF16), r(77), r(0)]
    return types.SimpleNamespace(x=x, w=w, b=b, q=q, s=s, wq=wq, ws=ws, long_a=long_a, long_b=long_b, mean=mean,
                                 rstd=rstd, grads=grads)


CALLS = {
    "fp8_gemm": lambda i, **k: [X.fp8_gemm(i.q, i.s, i.wq, i.ws, **k)],
    "fp8_gemm in slices": lambda i, **k: [X.fp8_gemm(*i.long_a, *i.long_b, out_dtype=F32, **k)],
    "fp8_quantize": lambda i, **k: X.fp8_quantize(i.x, transposed=True, **k),
    "fp8_quantize tiles": lambda i, **k: X.fp8_quantize(i.x, block_rows=128, **k),
    "layer_norm": lambda i, **k: X.layer_norm(i.x, i.w, i.b, stats=True, **k),
    "layer_norm_quantize": lambda i, **k: X.layer_norm_quantize(i.x, i.w, i.b, stats=True, **k),
    "layer_norm_backward": lambda i, **k: X.layer_norm_backward(i.x, i.x, i.mean, i.rstd, i.w, **k),
    "clip_grad_norm": lambda i, **k: (lambda n, g: [n, *g])(*X.clip_grad_norm(i.grads, 0.1, **k)),
}


def _bytes(t):
    return t.contiguous().reshape(-1).view(torch.uint8)


def _same(a, b):
    return all(np.array_equal(_bytes(p).cpu().numpy(), _bytes(q).cpu().numpy()) for p, q in zip(a, b))


def _pool(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("m", [4, 300])
def test_memory_comes_from_the_given_stream(name, m):
    i = _inputs(m)
    torch.cuda.synchronize()
    say(f"pool {name} {m}")
    side = torch.cuda.Stream()
    got = CALLS[name](i, stream=side)
    torch.cuda.synchronize()
    assert {_pool(t) for t in got if t.numel()} == {side.cuda_stream}
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream  # and the caller's is current again


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("m", [4, 300])
def test_memory_that_queued_work_still_uses_is_not_written(name, m):
    """The current stream has work queued on blocks that were freed on the host:
    just the sizes that the call allocates, so its pool would hand them out."""
    i = _inputs(m)
    call = CALLS[name]
    want = call(i)
    torch.cuda.synchronize()
    say(f"queued work {name} {m}")
    side = torch.cuda.Stream()
    torch.cuda._sleep(SPIN)
    blocks = [torch.empty(t.untyped_storage().nbytes(), dtype=torch.uint8, device=_dev()) for t in want]
    blocks += [torch.empty(n, dtype=torch.uint8, device=_dev()) for n in (4096, 1 << 16, 1 << 20, 1 << 22)]
    sums = []
    for fill, t in enumerate(blocks):
        t.fill_(fill + 1)
        sums.append((t.min().clone() if t.numel() else None, t.max().clone() if t.numel() else None))
    del blocks, t
    got = call(i, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert _same(got, want)
    for fill, (lo, hi) in enumerate(sums):
        assert lo is None or (lo.item() == fill + 1 and hi.item() == fill + 1)


@pytest.mark.parametrize("name", CALLS)
def test_results_outlive_their_use_on_the_callers_stream(name):
    """A result that is read on the current stream and then dropped is not
    given out again before that reading: the given stream's next call would
    overwrite it."""
    i = _inputs(300)
    call = CALLS[name]
    want = call(i)
    torch.cuda.synchronize()
    say(f"outlive {name}")
    side = torch.cuda.Stream()
    got = call(i, stream=side)
    side.synchronize()
    torch.cuda._sleep(SPIN)
    kept = [_bytes(t).clone() for t in got]
    sizes = [t.untyped_storage().nbytes() for t in got]
    del got
    with torch.cuda.stream(side):
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=_dev()).fill_(0x55)
    torch.cuda.synchronize()
    assert _same(kept, want)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("m", [4, 300])
def test_every_function_runs_on_the_given_stream(name, m):
    """What the given stream does before the call is done when the call's work
    runs: inputs that are only written there."""
    i = _inputs(m)
    call = CALLS[name]
    want = call(i)
    torch.cuda.synchronize()
    say(f"given stream {name} {m}")
    side = torch.cuda.Stream()
    clear = [t for t in (i.x, i.q.view(torch.uint8), i.long_a[0].view(torch.uint8), i.grads[0])]
    values = [t.clone() for t in clear]
    for t in clear:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
        for t, v in zip(clear, values):
            t.copy_(v)
    got = call(i, stream=side)
    side.synchronize()
    assert _same(got, want)


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_by_name_is_the_default(name):
    i = _inputs(40)
    assert _same(CALLS[name](i, stream=torch.cuda.current_stream()), CALLS[name](i))


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name):
    i = _inputs(4)
    s = torch.cuda.current_stream()
    other = types.SimpleNamespace(cuda_stream=s.cuda_stream, stream_id=s.stream_id, device_index=1,
                                  device_type=s.device_type)
    with pytest.raises(ValueError):
        CALLS[name](i, stream=other)
