"""The operators of an FP8 training and serving step of one normalised linear layer, as measured work.

A pre-normalised linear layer in 8-bit floating point goes layer norm -> quantisation in blocks of 128 -> matrix
product with block scales; its training step goes back through the same operators (products of transposed,
re-quantised operands, the norm's backward pass) and ends in the clipping of all gradients by their global norm.

    product   c = a b^T, a (m x k) and b (n x k) in e4m3 with one scale for each 128 columns of a row (or, for a
              weight, for each 128 x 128 tile)
    quantize  x -> e4m3 values and block scales, of x and of its transpose
    norm      layer norm, as a tensor or straight as e4m3 values and block scales
    norm_bwd  the gradients of layer norm's input, weight and bias
    clip      the global norm of many gradients, and the gradients scaled to a largest norm

A quantised matrix of `rows` x `cols` has its scales as a (ceil(cols / 128), rows) float32 tensor (tile of 128 rows:
(ceil(cols / 128), ceil(rows / 128))).  A scale is max(amax / 448, 2^-126), amax the block's largest magnitude; with
`pow2` the next power of two at or above that.  A value is x / scale, rounded to float32 and then to e4m3.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -126
EPS = 1e-5
CLIP_EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LARGEST_PRODUCT = 8192 ** 3
LARGEST_MATRIX = 12345 * 6789


def listed():
    return [
        # One token through a 4096 x 4096 weight while serving: the smallest call, bound by reading the weight.
        {"name": "product decode", "op": "product", "m": 1, "n": 4096, "k": 4096, "tile": 128, "pow2": False, "out": "bf16"},
        # The gradient of a weight: every operand quantised along an odd number of tokens, few blocks and a long sum.
        {"name": "product weight gradient", "op": "product", "m": 1000, "n": 2999, "k": 12345, "tile": 1, "pow2": False,
         "out": "fp32"},
        # A linear layer's forward pass over a prompt of 4096 tokens.
        {"name": "product prompt", "op": "product", "m": 4096, "n": 4096, "k": 4096, "tile": 128, "pow2": False,
         "out": "bf16"},
        # The same in a large training batch, with the power-of-two scales that the matrix cores take directly.
        {"name": "product large pow2", "op": "product", "m": 8192, "n": 8192, "k": 8192, "tile": 128, "pow2": True,
         "out": "bf16"},
        # Activations kept for both products of a training step: rows for the forward, columns for the weight gradient.
        {"name": "quantize activations", "op": "quantize", "rows": 8192, "cols": 8192, "tile": 1, "pow2": False, "in": "bf16"},
        # A float32 master weight of odd sizes, requantised after each update: one scale for each tile of 128 x 128.
        {"name": "quantize weight", "op": "quantize", "rows": 12345, "cols": 6789, "tile": 128, "pow2": True, "in": "fp32"},
        # Four sequences that each get one token: the norm before a decode product, straight to e4m3.
        {"name": "norm decode", "op": "norm", "rows": 4, "cols": 4096, "in": "bf16", "quantized": True},
        # The norm of a training batch, with the statistics that the backward pass needs.
        {"name": "norm train", "op": "norm", "rows": 8192, "cols": 8192, "in": "bf16", "quantized": False},
        # Its backward pass, with the weight's gradient summed over all tokens.
        {"name": "norm backward", "op": "norm_bwd", "rows": 8192, "cols": 4096, "in": "bf16"},
        # The same in float32 with odd sizes, rows that start off every vector boundary.
        {"name": "norm backward odd", "op": "norm_bwd", "rows": 3001, "cols": 2999, "in": "fp32"},
        # The small tensors of a model (biases, norms): latency and launches are what counts.
        {"name": "clip small", "op": "clip", "tensors": 24, "side": 64, "in": "fp32"},
        # All gradients of a stack of layers, matrices in bf16 and vectors in float32.
        {"name": "clip layers", "op": "clip", "tensors": 32, "side": 4096, "in": "bf16"},
    ]


def _log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "quantize", "norm", "norm_bwd", "clip"])
    if op == "product":
        case = {"op": op, "m": _log_size(rng, 1, 8192), "n": _log_size(rng, 16, 8192), "k": _log_size(rng, 16, 12345),
                "tile": rng.choice([1, 128]), "pow2": rng.random() < 0.5, "out": rng.choice(["bf16", "fp16", "fp32"])}
        if rng.random() < 0.5:  # half of the products are of whole vectors
            case["k"] = -(-case["k"] // 16) * 16
        while case["m"] * case["n"] * case["k"] > LARGEST_PRODUCT:
            case["m"] = max(1, case["m"] // 2)
        return case
    if op == "clip":
        return {"op": op, "tensors": rng.randint(1, 60), "side": _log_size(rng, 2, 3000), "in": rng.choice(list(TYPES))}
    rows, cols = _log_size(rng, 1, 16384), _log_size(rng, 64, 16384)
    if rng.random() < 0.5:
        cols = -(-cols // 8) * 8
    while rows * cols > LARGEST_MATRIX // 2:
        rows = max(1, rows // 2)
    case = {"op": op, "rows": rows, "cols": cols, "in": rng.choice(list(TYPES))}
    if op == "quantize":
        case.update(tile=rng.choice([1, 128]), pow2=rng.random() < 0.5)
    if op == "norm":
        case.update(quantized=rng.random() < 0.5)
    return case


# ----- inputs ----------------------------------------------------------------

def _activations(rows, cols, gen, dtype):
    """Normal values with a few loud channels and a few silent tokens."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.005
    x *= torch.where(loud, 20.0, 1.0)
    x *= (torch.rand(rows, 1, generator=gen, device="cuda") >= 0.002).float()
    return x.to(dtype)


def _gradients(rows, cols, gen, dtype):
    """Small values whose size differs from token to token."""
    size = torch.exp(torch.randn(rows, 1, generator=gen, device="cuda")) * 1e-3
    return (torch.randn(rows, cols, generator=gen, device="cuda") * size).to(dtype)


def _pitched(q):
    """The same matrix with rows that start at multiples of 16 elements, as a quantised matrix is stored."""
    rows, cols = q.shape
    store = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=q.device)
    store[:, :cols] = q.view(torch.uint8)
    return store.view(torch.float8_e4m3fn)[:, :cols]


def _clip_shapes(case):
    """Three matrices of different form for each vector; one tensor of every 16 is empty."""
    side = case["side"]
    forms = [(side, side), (side, 4 * side // 3 + 1), (side // 2 + 1, side), (4 * side + 1,)]
    return [(0,) if i % 16 == 13 else forms[i % 4] for i in range(case["tensors"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "product":
        a = _activations(case["m"], case["k"], gen, torch.float32)
        b = torch.randn(case["n"], case["k"], generator=gen, device="cuda") * 0.02
        a, scale_a = _quantize(a, 1, case["pow2"])
        b, scale_b = _quantize(b, case["tile"], case["pow2"])
        return {"case": case, "a": _pitched(a), "scale_a": scale_a, "b": _pitched(b), "scale_b": scale_b}
    dtype = TYPES[case["in"]]
    if op == "clip":
        grads = [torch.randn(s, generator=gen, device="cuda") * 1e-2 for s in _clip_shapes(case)]
        grads = [g if g.dim() == 1 else g.to(dtype) for g in grads]
        # A user's program has the scaled gradients go to buffers that it keeps.
        return {"case": case, "grads": grads, "out": [torch.empty_like(g) for g in grads], "max_norm": 1.0}
    x = _activations(case["rows"], case["cols"], gen, dtype)
    state = {"case": case, "x": x}
    if op != "quantize":
        state["x"] = (x.float() + 0.5).to(dtype)
        state["weight"] = 1 + 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")
        state["bias"] = 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")
    if op == "norm_bwd":
        state["dy"] = _gradients(case["rows"], case["cols"], gen, dtype)
        _, state["mean"], state["rstd"] = _norm(state["x"].float(), state["weight"], state["bias"])
    return state


# ----- the plain forms -------------------------------------------------------

def _blocks(x, tile):
    """x padded with zeros to whole blocks, as (row blocks, tile, column blocks, 128)."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % tile))
    return x.view(x.shape[0] // tile, tile, x.shape[1] // BLOCK, BLOCK)


def _quantize(x, tile, pow2):
    rows, cols = x.shape
    blocks = _blocks(x.float(), tile)
    amax = blocks.abs().amax(dim=(1, 3))
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=SMALLEST)  # by a scalar, torch multiplies by 1 / 448
    if pow2:
        bits = scale.view(torch.int32)
        scale = ((bits + 0x7FFFFF) & 0x7F800000).view(torch.float32)
    q = (blocks / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(blocks.shape[0] * tile, -1)[:rows, :cols].contiguous()
    return q.view(torch.float8_e4m3fn), scale.t().contiguous()


def _spread(scale, tile, rows, cols):
    """One scale for each value of a rows x cols matrix."""
    scale = scale.t().repeat_interleave(tile, dim=0).repeat_interleave(BLOCK, dim=1)
    return scale[:rows, :cols]


def _norm(x, weight, bias):
    mean = x.mean(dim=1, keepdim=True)
    centred = x - mean
    rstd = 1 / torch.sqrt((centred * centred).mean(dim=1, keepdim=True) + EPS)
    return centred * rstd * weight + bias, mean.squeeze(1), rstd.squeeze(1)


def _norm_backward(dy, x, mean, rstd, weight):
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dx = (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True)) * rstd[:, None]
    return dx, (dy * xhat).sum(dim=0), dy.sum(dim=0)


def _clip(grads, max_norm):
    """Squares are summed in 64 bits: a model has more gradients than 32 bits tell apart."""
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()
    factor = (max_norm / (norm + CLIP_EPS)).clamp(max=1.0)
    return norm.float(), [(g.float() * factor.float()).to(g.dtype) for g in grads]


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = s["a"].float() * _spread(s["scale_a"], 1, m, k)
        b = s["b"].float() * _spread(s["scale_b"], case["tile"], n, k)
        return (a @ b.t()).to(TYPES[case["out"]])
    if op == "quantize":
        q, scale = _quantize(s["x"], case["tile"], case["pow2"])
        qt, scale_t = _quantize(s["x"].t().contiguous(), case["tile"], case["pow2"])
        return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
    if op == "norm":
        y, mean, rstd = _norm(s["x"].float(), s["weight"], s["bias"])
        if case["quantized"]:
            q, scale = _quantize(y, 1, False)
            return {"q": q, "scale": scale}
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dweight, dbias = _norm_backward(s["dy"].float(), s["x"].float(), s["mean"], s["rstd"], s["weight"])
        return {"dx": dx.to(s["x"].dtype), "dweight": dweight, "dbias": dbias}
    norm, out = _clip(s["grads"], s["max_norm"])
    return {"norm": norm, "grads": out}


def _run_own(s):
    import lds_tiled_matrix_amd as X
    case, op = s["case"], s["case"]["op"]
    if op == "product":
        return X.fp8_gemm(s["a"], s["scale_a"], s["b"], s["scale_b"], out_dtype=TYPES[case["out"]], pow2=case["pow2"])
    if op == "quantize":
        q, scale, qt, scale_t = X.fp8_quantize(s["x"], block_rows=case["tile"], pow2=case["pow2"], transposed=True)
        return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
    if op == "norm":
        if case["quantized"]:
            q, scale = X.layer_norm_quantize(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"q": q, "scale": scale}
        y, mean, rstd = X.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dweight, dbias = X.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    norm, out = X.clip_grad_norm(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["out"])
    return {"norm": norm, "grads": out}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----- what a pass cannot do without -----------------------------------------

def _scales(rows, cols, tile):
    return -(-cols // BLOCK) * -(-rows // tile)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        read = m * k + n * k + 4 * (_scales(m, k, 1) + _scales(n, k, case["tile"]))
        return {"bytes": read + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if op == "clip":
        count = [(math.prod(s), 4 if len(s) == 1 else size[case["in"]]) for s in _clip_shapes(case)]
        return {"bytes": 2 * sum(n * b for n, b in count) + 4, "flops": 3 * sum(n for n, _ in count)}
    rows, cols = case["rows"], case["cols"]
    values = rows * cols
    if op == "quantize":
        scales = _scales(rows, cols, case["tile"]) + _scales(cols, rows, case["tile"])
        return {"bytes": values * (size[case["in"]] + 2) + 4 * scales, "flops": 4 * values}
    if op == "norm":
        if case["quantized"]:
            return {"bytes": values * (size[case["in"]] + 1) + 4 * _scales(rows, cols, 1) + 8 * cols, "flops": 10 * values}
        return {"bytes": 2 * values * size[case["in"]] + 8 * (rows + cols), "flops": 8 * values}
    return {"bytes": 3 * values * size[case["in"]] + 8 * rows + 12 * cols, "flops": 14 * values}


# ----- the definitions in 64 bits --------------------------------------------

def _exact_quantize(x, tile, pow2):
    """As the definition at the top says it: x in 64 bits; the scale and each quotient are numbers of 32 bits by definition."""
    rows, cols = x.shape
    row_blocks, col_blocks = -(-rows // tile), -(-cols // BLOCK)
    whole = torch.zeros(row_blocks * tile, col_blocks * BLOCK, dtype=torch.float64, device=x.device)
    whole[:rows, :cols] = x
    amax = whole.abs().reshape(row_blocks, tile, col_blocks, BLOCK).amax(dim=3).amax(dim=1)
    scale = torch.maximum((amax / E4M3_MAX).float(), torch.tensor(SMALLEST, device=x.device)).double()
    if pow2:
        fraction, exponent = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), torch.where(fraction == 0.5, exponent - 1, exponent))
    each = scale.repeat_interleave(tile, 0).repeat_interleave(BLOCK, 1)
    value = (whole / each).float().double()[:rows, :cols]
    # e4m3: four significant bits down to 2^-6, then steps of 2^-9, ties to even
    _, exponent = torch.frexp(value)
    step = torch.ldexp(torch.ones_like(value), exponent.clamp(min=-5) - 4)
    return torch.round(value / step) * step, scale.t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        row = torch.arange(n, device="cuda") // case["tile"]
        col = torch.arange(k, device="cuda") // BLOCK
        a = s["a"].double() * s["scale_a"].double()[col].t()
        b = s["b"].double() * s["scale_b"].double()[col][:, row].t()
        return torch.matmul(a, b.t().contiguous())
    if op == "quantize":
        x = s["x"].double()
        q, scale = _exact_quantize(x, case["tile"], case["pow2"])
        qt, scale_t = _exact_quantize(x.t().contiguous(), case["tile"], case["pow2"])
        return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}
    if op == "clip":
        grads = [g.double() for g in s["grads"]]
        norm = math.sqrt(math.fsum(float((g * g).sum()) for g in grads))
        factor = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [g * factor for g in grads]}
    x, weight = s["x"].double(), s["weight"].double()
    cols = case["cols"]
    if op == "norm":
        mean = x.sum(dim=1) / cols
        variance = ((x - mean[:, None]) ** 2).sum(dim=1) / cols
        rstd = (variance + EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * weight + s["bias"].double()
        if case["quantized"]:
            q, scale = _exact_quantize(y, 1, False)
            return {"q": q, "scale": scale}
        return {"y": y, "mean": mean, "rstd": rstd}
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xhat = (x - mean) * rstd
    g = dy * weight
    along = (g.sum(dim=1, keepdim=True) + xhat * (g * xhat).sum(dim=1, keepdim=True)) / cols
    return {"dx": rstd * (g - along), "dweight": (dy * xhat).sum(dim=0), "dbias": dy.sum(dim=0)}
