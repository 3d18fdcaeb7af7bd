"""What autograd sees of the linear operators: results without a graph, and
tensors given as ``out`` as changed in place."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
X = pytest.importorskip("lds_tiled_matrix_amd")


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda", 0)


def _clip(out):
    X.clip_grad_norm([torch.ones_like(out)], 1.0, out=[out])


def _clip_in_place(out):
    X.clip_grad_norm([out], 1.0, out=[out])


def _gemm(out):
    q, s = X.fp8_quantize(torch.ones(out.shape[0], 64, device=_dev()))
    p, t = X.fp8_quantize(torch.ones(out.shape[1], 64, device=_dev()))
    X.fp8_gemm(q, s, p, t, out=out)


WRITES = {
    "layer_norm": lambda out: X.layer_norm(torch.ones_like(out), out=out),
    "layer_norm in place": lambda out: X.layer_norm(out, out=out),
    "fp8_gemm": _gemm,
    "clip_grad_norm": _clip,
    "clip_grad_norm in place": _clip_in_place,
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
    x = torch.randn(20, 30, device=_dev(), requires_grad=True)
    w = torch.randn(30, device=_dev(), requires_grad=True)
    y, mean, rstd = X.layer_norm(x, w, stats=True)
    q, s = X.fp8_quantize(x)
    norm, out = X.clip_grad_norm([x], 1.0)
    got = [y, mean, rstd, s, norm, *out, *X.layer_norm_backward(x, x, mean, rstd, w), X.fp8_gemm(q, s, q, s)]
    assert not any(t.requires_grad for t in got)
    assert x._version == 0 and w._version == 0
