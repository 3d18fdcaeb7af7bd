"""A normalised linear layer trained and served in 8-bit floating point.

    python examples/fp8_linear.py [--tokens 4096] [--width 2048] [--outputs 2048] [--steps 20]

The layer is layer norm and a weight, y = norm(x) W^T.  A training step
quantises activations, weight and gradients in blocks of 128, takes the three
products of the layer in 8 bits, goes back through the norm and clips all
gradients by their global norm; serving takes one token through norm,
quantisation and product in two launches.  The data are synthetic: a fixed
layer of the same form whose outputs are to be learned.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lds_tiled_matrix_amd as X  # noqa: E402


class Fp8Linear:
    """Parameters in float32, products in e4m3."""

    def __init__(self, width, outputs, device, seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.gain = torch.ones(width, device=device)
        self.bias = torch.zeros(width, device=device)
        self.weight = torch.randn(outputs, width, generator=gen, device=device) * width ** -0.5

    def parameters(self):
        return [self.gain, self.bias, self.weight]

    def quantized_weight(self):
        """The weight for the forward product and its transpose for the
        backward one, a scale for each 128 x 128 tile: once an update."""
        return X.fp8_quantize(self.weight, block_rows=128, transposed=True)

    def forward(self, x, weight_q):
        y, mean, rstd = X.layer_norm(x, self.gain, self.bias, stats=True)
        y_q, y_s, y_qt, y_st = X.fp8_quantize(y, transposed=True)
        out = X.fp8_gemm(y_q, y_s, weight_q[0], weight_q[1])
        return out, (x, mean, rstd, y_qt, y_st)

    def backward(self, grad, saved, weight_q):
        """(grad of x, [grads of gain, bias, weight])."""
        x, mean, rstd, y_qt, y_st = saved
        g_q, g_s, g_qt, g_st = X.fp8_quantize(grad, transposed=True)
        grad_y = X.fp8_gemm(g_q, g_s, weight_q[2], weight_q[3], out_dtype=x.dtype)
        grad_weight = X.fp8_gemm(g_qt, g_st, y_qt, y_st, out_dtype=torch.float32)
        grad_x, grad_gain, grad_bias = X.layer_norm_backward(grad_y, x, mean, rstd, self.gain)
        return grad_x, [grad_gain, grad_bias, grad_weight]

    def serve(self, x, weight_q):
        """Few tokens: the norm goes straight to e4m3."""
        q, s = X.layer_norm_quantize(x, self.gain, self.bias)
        return X.fp8_gemm(q, s, weight_q[0], weight_q[1])


def train(tokens=4096, width=2048, outputs=2048, steps=20, rate=0.1, max_norm=1.0, device="cuda", log=print):
    """Learns a fixed layer's outputs; returns the losses."""
    teacher, student = Fp8Linear(width, outputs, device, seed=1), Fp8Linear(width, outputs, device, seed=2)
    gen = torch.Generator(device=device)
    gen.manual_seed(3)
    x = torch.randn(tokens, width, generator=gen, device=device).bfloat16()
    want = teacher.serve(x, teacher.quantized_weight()).float()
    losses = []
    for step in range(steps):
        weight_q = student.quantized_weight()
        out, saved = student.forward(x, weight_q)
        off = out.float() - want
        loss = off.square().mean()
        grad = (off * (2 / tokens)).bfloat16()  # of the loss summed over outputs
        _, grads = student.backward(grad, saved, weight_q)
        norm, grads = X.clip_grad_norm(grads, max_norm * outputs ** 0.5, out=grads)
        for p, g in zip(student.parameters(), grads):
            p.sub_(g, alpha=rate)
        losses.append(loss)
        if log and (step % 5 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {loss.item():.5f}  gradient norm {norm.item():.4f}")
    token = student.serve(x[:1], student.quantized_weight())
    if log:
        log(f"one token served: output {tuple(token.shape)}, "
            f"off by {(token.float() - want[:1]).square().mean().item():.5f}")
    return [v.item() for v in losses]


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("width", 2048), ("outputs", 2048), ("steps", 20)):
        parser.add_argument(f"--{name}", type=int, default=value)
    train(**vars(parser.parse_args()))
