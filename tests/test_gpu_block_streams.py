"""A residual block's operators with the ``stream`` argument, in what autograd
sees of them, captured, and in places far into large buffers."""
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


def _inputs(m, k=1000, n=300):
    gen = torch.Generator(device=_dev()).manual_seed(m)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    i = types.SimpleNamespace(x=r(m, k).to(BF16), res=r(m, k).to(BF16), w=r(k), a=(r(5, 16, k) * 0.03).to(BF16),
                              b=r(5, n, 16).to(BF16), scale=r(5), base=r(m, n).to(BF16), dout=r(m, n).to(BF16),
                              ids=(torch.arange(m, device=_dev()) * 5 // 3 % 6).int(),
                              seed=torch.tensor([m], device=_dev()))
    i.h, i.rstd = X.rms_norm(i.x, i.w, residual=i.res, stats=True)[1:]
    i.q, i.s = X.fp8_quantize(i.x)
    i.hidden = X.adapters(i.x, i.a, i.b, i.ids, hidden=True)[1]
    return i


def _adapters(i, **k):
    return [X.adapters(i.x, i.a, i.b, i.ids, base=i.base, scale=i.scale, **k)]


CALLS = {
    "rms_norm": lambda i, **k: list(X.rms_norm(i.x, i.w, residual=i.res, stats=True, **k)),
    "rms_norm_quantize": lambda i, **k: list(X.rms_norm_quantize(i.x, i.w, residual=i.res, stats=True, **k)),
    "rms_norm_backward": lambda i, **k: list(X.rms_norm_backward(i.res, i.x, i.rstd, i.w, dresidual=i.res, **k)),
    "adapters": _adapters,
    "adapters of e4m3, hidden": lambda i, **k: list(X.adapters(i.q, i.a, i.b, i.ids, scale_x=i.s, hidden=True, **k)),
    "adapters_backward": lambda i, **k: list(X.adapters_backward(i.dout, i.x, i.a, i.b, i.ids, i.hidden, base=i.x,
                                                                 scale=i.scale, **k)),
    "adapters_backward, weights": lambda i, **k: list(X.adapters_backward(
        i.dout, i.x, i.a, i.b, i.ids, i.hidden, wanted=(False, True, True), **k))[1:],
    "dropout": lambda i, **k: [X.dropout(i.x, 0.3, i.seed, offset=7, residual=i.res, **k)],
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
@pytest.mark.parametrize("m", [4, 700])
def test_memory_comes_from_the_given_stream(name, m):
    i = _inputs(m)
    torch.cuda.synchronize()
    say(f"pool {name} {m}")
    side = torch.cuda.Stream()
    got = CALLS[name](i, stream=side)
    torch.cuda.synchronize()
    assert {_pool(t) for t in got if t.numel()} == {side.cuda_stream}
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("m", [4, 700])
def test_memory_that_queued_work_still_uses_is_not_written(name, m):
    """The current stream has work queued on blocks that were freed on the host,
    of the sizes that the call allocates."""
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
@pytest.mark.parametrize("m", [4, 700])
def test_every_function_runs_on_the_given_stream(name, m):
    """Inputs that the given stream has only written before the call, ids and
    seed among them."""
    i = _inputs(m)
    call = CALLS[name]
    want = call(i)
    torch.cuda.synchronize()
    say(f"given stream {name} {m}")
    side = torch.cuda.Stream()
    clear = [i.x, i.q.view(torch.uint8), i.dout, i.res, i.ids, i.seed, i.scale, i.hidden, i.rstd]
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
@pytest.mark.parametrize("m", [4, 700])
def test_calls_of_two_streams_at_once(name, m):
    """Both streams' calls queued behind a wait, several of each: nothing of the
    one's workspace is the other's."""
    cases = [_inputs(m), _inputs(m + 1)]
    call = CALLS[name]
    wants = [call(i) for i in cases]
    torch.cuda.synchronize()
    say(f"two streams {name} {m}")
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(SPIN)
    for _ in range(4):
        for s, i, g in zip(streams, cases, got):
            g.append(call(i, stream=s))
    torch.cuda.synchronize()
    for want, g in zip(wants, got):
        assert all(_same(v, want) for v in g)


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


# ----- what autograd sees -------------------------------------------------------------

def _out_case():
    gen = torch.Generator(device=_dev()).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    return r(2, 4, 30), r(2, 30, 4), torch.zeros(20, dtype=torch.int32, device=_dev())


def _out_adapters(out):
    a, b, ids = _out_case()
    X.adapters(torch.ones_like(out), a, b, ids, out=out)


def _out_adapters_in_place(out):
    a, b, ids = _out_case()
    X.adapters(torch.ones_like(out), a, b, ids, base=out, out=out)


def _out_backward(out):
    a, b, ids = _out_case()
    X.adapters_backward(torch.ones_like(out), torch.ones_like(out), a, b, ids, torch.ones(20, 4, device=_dev()), out=out)


WRITES = {
    "rms_norm": lambda out: X.rms_norm(torch.ones_like(out), out=out),
    "rms_norm in place": lambda out: X.rms_norm(out, out=out),
    "rms_norm residual_out": lambda out: X.rms_norm(torch.ones_like(out), residual=out, residual_out=out),
    "rms_norm_quantize residual_out": lambda out: X.rms_norm_quantize(out, residual=out.clone(), residual_out=out),
    "adapters": _out_adapters,
    "adapters in place": _out_adapters_in_place,
    "adapters_backward": _out_backward,
    "dropout": lambda out: X.dropout(out, 0.5, 1, out=out),
}


@pytest.mark.parametrize("name", WRITES)
def test_out_is_changed_in_place(name):
    x = torch.randn(20, 30, device=_dev(), requires_grad=True)
    y = x.exp()  # saves its result for the backward pass
    out = y.detach()
    before = out._version
    WRITES[name](out)
    assert out._version == y._version == before + 1
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


@pytest.mark.parametrize("name", WRITES)
def test_out_of_inference_mode(name):
    with torch.inference_mode():
        out = torch.ones(20, 30, device=_dev())
    WRITES[name](out)
    torch.cuda.synchronize()


def test_inputs_keep_their_version_and_results_have_no_graph():
    i = _inputs(20)
    for t in (i.x, i.res, i.w, i.a, i.b, i.base, i.dout, i.hidden, i.rstd):
        t.requires_grad_()
    tensors = [t for t in vars(i).values()]
    before = [t._version for t in tensors]
    for call in CALLS.values():
        assert not any(t.requires_grad for t in call(i))
    assert [t._version for t in tensors] == before


class _Adapted(torch.autograd.Function):
    """The adapters as a node of a graph, as a program would make one."""

    @staticmethod
    def forward(ctx, x, a, b, base, ids):
        out, hidden = X.adapters(x, a, b, ids, base=base, hidden=True)
        ctx.save_for_backward(x, a, b, ids, hidden)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, a, b, ids, hidden = ctx.saved_tensors
        dx, da, db = X.adapters_backward(dout.contiguous(), x, a, b, ids, hidden)
        return dx, da.to(a.dtype), db.to(b.dtype), dout, None


def _gradients(i, leaves):
    x, a, b, base = leaves
    return torch.autograd.grad(_Adapted.apply(x, a, b, base, i.ids), leaves, i.dout)


@pytest.mark.parametrize("m", [4, 700])
def test_a_step_in_a_graph(m):
    """Forward and backward of an autograd node captured and replayed, eager
    work of the same operators between."""
    i = _inputs(m)
    eager = [t.clone().requires_grad_() for t in (i.x, i.a, i.b, i.base)]
    leaves = [t.clone().requires_grad_() for t in (i.x, i.a, i.b, i.base)]
    say(f"step in a graph {m}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _gradients(i, leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _gradients(i, leaves)
    for turn in range(4):
        with torch.no_grad():
            for e, t in zip(eager, leaves):
                t.copy_(e)
            i.dout.mul_(-1 if turn % 2 else 1)
        graph.replay()
        want = _gradients(i, eager)
        torch.cuda.synchronize()
        assert _same(got, want)
        with torch.no_grad():
            eager[0].mul_(0.5)


def test_a_graph_of_other_sizes_than_were_called_before():
    """Nothing has to be called eagerly first: sizes, types and kernels that only
    the capture uses."""
    gen = torch.Generator(device=_dev()).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device=_dev())  # noqa: E731
    x, a, b = r(77, 96).half(), r(3, 24, 96).half(), r(3, 112, 24).half()
    ids = (torch.arange(77, device=_dev()) % 4).int()

    def run():
        y, rstd = X.rms_norm(x, stats=True)
        out, hidden = X.adapters(y, a, b, ids, hidden=True)
        dropped = X.dropout(out, 0.5, 3)
        dy, da, db = X.adapters_backward(dropped, y, a, b, ids, hidden)
        return [out, dropped, dy, da, db, *X.rms_norm_backward(dy, x, rstd)]

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(3):
        x.mul_(0.9)
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert _same(got, want)


# ----- places ---------------------------------------------------------------------------

def _far(t, pitch):
    """A matrix with rows so far apart that later ones begin over 2^31 elements in."""
    store = torch.empty((t.shape[0] - 1) * pitch + t.shape[1], dtype=t.dtype, device=_dev())
    view = torch.as_strided(store, t.shape, (pitch, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("name", ["adapters", "adapters_backward", "rms_norm", "rms_norm_quantize",
                                  "rms_norm_backward", "dropout"])
def test_far_rows(name):
    i, pitch = _inputs(40, 264, 300), 1 << 26
    far = lambda t: _far(t, pitch)  # noqa: E731
    empty = lambda t: far(torch.zeros_like(t))  # noqa: E731
    say(f"far rows {name}")
    if name == "adapters":
        want = _adapters(i)
        got = [X.adapters(i.x, i.a, i.b, i.ids, base=far(i.base), scale=i.scale, out=empty(i.base))]
    elif name == "adapters_backward":
        want = CALLS[name](i)
        got = X.adapters_backward(far(i.dout), i.x, i.a, i.b, i.ids, i.hidden, base=far(i.x), scale=i.scale,
                                  out=empty(i.x))
    elif name == "rms_norm":
        want = CALLS[name](i)
        got = X.rms_norm(far(i.x), i.w, residual=far(i.res), stats=True, out=empty(i.x), residual_out=empty(i.x))
    elif name == "rms_norm_quantize":
        want = CALLS[name](i)
        got = X.rms_norm_quantize(far(i.x), i.w, residual=far(i.res), stats=True, residual_out=empty(i.x))
    elif name == "rms_norm_backward":
        want = CALLS[name](i)
        got = X.rms_norm_backward(far(i.res), far(i.x), i.rstd, i.w, dresidual=far(i.res))
    else:
        want = CALLS[name](i)
        got = [X.dropout(far(i.x), 0.3, i.seed, offset=7, residual=far(i.res), out=empty(i.x))]
    torch.cuda.synchronize()
    assert _same(got, want)


def test_one_adapter_as_many_and_shared_weights():
    """Adapters that are the same memory (a pitch of zero between them), and a
    row that several results come from."""
    i = _inputs(300)
    a, b = i.a[1:2].expand(5, -1, -1), i.b[1:2].expand(5, -1, -1)
    want = X.adapters(i.x, a.contiguous(), b.contiguous(), i.ids, hidden=True)
    got = X.adapters(i.x, a, b, i.ids, hidden=True)
    assert _same(got, want)
    p = X.adapters_backward(i.dout, i.x, a, b, i.ids, got[1])
    q = X.adapters_backward(i.dout, i.x, a.contiguous(), b.contiguous(), i.ids, got[1])
    assert _same(p, q)
    assert torch.equal(X.rms_norm(i.x, residual=i.x)[1], (i.x.float() * 2).to(BF16))


@pytest.mark.parametrize("shift", [1, 3, 7])
def test_places_of_any_alignment(shift):
    """Inputs and outputs that begin at any element."""
    i = _inputs(100)
    want = {name: CALLS[name](i) for name in CALLS if name != "adapters of e4m3, hidden"}
    for name in ("x", "res", "w", "a", "b", "base", "dout", "hidden", "scale", "ids", "rstd"):
        t = getattr(i, name)
        store = torch.empty(t.numel() + 8, dtype=t.dtype, device=_dev())
        view = store[shift:shift + t.numel()].view(t.shape)
        view.copy_(t)
        setattr(i, name, view)
    for name, values in want.items():
        say(f"shift {shift} {name}")
        assert _same(CALLS[name](i), values)
