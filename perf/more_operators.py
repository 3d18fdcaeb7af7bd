"""The operators that fine-tune and serve low-rank adapters beside an 8-bit linear layer, as measured work.

A block of a residual stream goes root-mean-square norm (with the residual's addition before it) -> the shared 8-bit
product -> the adapters of each token's request added to that -> dropout on the way back to the residual stream.

    norm          h = x + residual, y = h / rms(h) * weight, as a tensor
    norm_q        the same straight to e4m3 values and block scales
    norm_bwd      the gradients of h and weight, with the gradient that comes down the residual stream added
    adapters      out = base + scale (x A^T) B^T with the A and B of each row's adapter, rows without one as they are
    adapters_bwd  the gradients of x (added to the shared product's), of every A and of every B
    dropout       residual + dropped x, the mask a function of a seed and the element's place

A quantised matrix is as in perf/operators.py: e4m3 values, a float32 scale for each row and 128 columns as a
(ceil(cols / 128), rows) tensor, scale max(amax / 448, 2^-126), value x / scale rounded to float32 and then to e4m3.

The dropout's mask.  Element (row, col) takes the 16 bits number col % 8 (the first word's low half first) of the
Philox4x32-10 block with the counter (col / 8, row, offset's low word, offset's high word) and the key (seed's low word,
seed's high word), and stays where they are at least t = round(65536 p); what stays is multiplied by 65536 / (65536 - t).
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -126
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LARGEST_MATRIX = 8192 * 8192
LARGEST_ADAPTERS = 8192 * (4096 + 4096)
NO_ADAPTER = -1


def listed():
    return [
        # One token of a request being served: the norm before an 8-bit product, bound by latency.
        {"name": "norm_q decode", "op": "norm_q", "rows": 1, "cols": 4096, "in": "bf16", "residual": True},
        # The same norm over a prompt.
        {"name": "norm_q prompt", "op": "norm_q", "rows": 4096, "cols": 8192, "in": "bf16", "residual": True},
        # The norm of a training batch with what its backward pass needs.
        {"name": "norm train", "op": "norm", "rows": 8192, "cols": 8192, "in": "bf16", "residual": True},
        # A float32 stream of odd sizes, rows that start off every vector boundary.
        {"name": "norm odd", "op": "norm", "rows": 3001, "cols": 2999, "in": "fp32", "residual": True},
        # The backward pass of a training batch, the residual stream's gradient added.
        {"name": "norm_bwd train", "op": "norm_bwd", "rows": 8192, "cols": 4096, "in": "bf16", "residual": True},
        # The same in float32 with odd sizes and no residual (a model's last norm).
        {"name": "norm_bwd odd", "op": "norm_bwd", "rows": 3001, "cols": 2999, "in": "fp32", "residual": False},
        # Sixteen requests that get one token each, most of them with an adapter of their own, beside an 8-bit product.
        {"name": "adapters decode", "op": "adapters", "rows": 16, "requests": 16, "k": 4096, "n": 4096, "rank": 16,
         "count": 32, "type": "bf16", "x": "e4m3", "out": "bf16"},
        # Prompts of different lengths in one batch, an odd number of tokens, into a wider layer.
        {"name": "adapters prompts", "op": "adapters", "rows": 4001, "requests": 7, "k": 4096, "n": 8192, "rank": 16,
         "count": 32, "type": "bf16", "x": "bf16", "out": "bf16"},
        # Fine-tuning of four adapters at once, every gradient.
        {"name": "adapters_bwd train", "op": "adapters_bwd", "rows": 8192, "requests": 8, "k": 4096, "n": 4096,
         "rank": 16, "count": 4, "type": "bf16", "out": "bf16"},
        # One adapter in float32 on a small batch of odd sizes.
        {"name": "adapters_bwd small", "op": "adapters_bwd", "rows": 300, "requests": 3, "k": 1222, "n": 2999,
         "rank": 12, "count": 1, "type": "fp32", "out": "fp32"},
        # A training batch's block output, dropped and added to the residual stream.
        {"name": "dropout train", "op": "dropout", "rows": 8192, "cols": 8192, "in": "bf16", "p": 0.1, "residual": True},
        # The input of one adapter in a small batch of odd rows.
        {"name": "dropout small", "op": "dropout", "rows": 64, "cols": 4519, "in": "fp16", "p": 0.05, "residual": False},
    ]


def _log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_q", "norm_bwd", "adapters", "adapters", "adapters_bwd", "dropout"])
    if op in ("adapters", "adapters_bwd"):
        rows = _log_size(rng, 1, 8192)
        k, n = _log_size(rng, 16, 8192), _log_size(rng, 16, 8192)
        if rng.random() < 0.5:  # half of them of whole vectors
            k, n = -(-k // 16) * 16, -(-n // 16) * 16
        kind = rng.choice(list(TYPES))
        case = {"op": op, "rows": rows, "k": k, "n": n, "rank": rng.choice([4, 8, 12, 16, 16, 24, 32, 64]),
                "count": _log_size(rng, 1, 64), "type": kind, "out": rng.choice([kind, "fp32"])}
        if op == "adapters":
            case["x"] = rng.choice([kind, "e4m3"])
        else:
            case["out"] = kind
        while case["rows"] * (k + n) * case["rank"] > LARGEST_ADAPTERS * 16:
            case["rows"] = max(1, case["rows"] // 2)
        rows = case["rows"]
        # few rows are tokens of as many requests, many are prompts
        case["requests"] = rows if rows <= 64 else _log_size(rng, 1, 32)
        return case
    rows, cols = _log_size(rng, 1, 16384), _log_size(rng, 64, 16384)
    if rng.random() < 0.5:
        cols = -(-cols // 8) * 8
    while rows * cols > LARGEST_MATRIX // 2:
        rows = max(1, rows // 2)
    case = {"op": op, "rows": rows, "cols": cols, "in": rng.choice(list(TYPES)), "residual": rng.random() < 0.7}
    if op == "dropout":
        case["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
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


def _row_adapters(case, seed):
    """Requests one after the other, each with its adapter for all of its rows; one in ten has none."""
    gen = torch.Generator()
    gen.manual_seed(seed + 1)
    rows, requests = case["rows"], case["requests"]
    if requests >= rows:
        of_row = torch.arange(rows)
    else:
        ends = torch.sort(torch.randperm(rows - 1, generator=gen)[:requests - 1] + 1).values
        of_row = torch.searchsorted(ends, torch.arange(rows), right=True)
    adapter = torch.randint(0, case["count"], (requests,), generator=gen)
    adapter[torch.rand(requests, generator=gen) < 0.1] = NO_ADAPTER
    return adapter[of_row].to(torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    op = case["op"]
    state = {"case": case}
    if op in ("adapters", "adapters_bwd"):
        rows, k, n, rank, count = (case[v] for v in ("rows", "k", "n", "rank", "count"))
        kind = TYPES[case["type"]]
        x = _activations(rows, k, gen, kind)
        state["a"] = (randn(count, rank, k) * k ** -0.5).to(kind)
        state["b"] = (randn(count, n, rank) * 0.02).to(kind)
        state["ids"] = _row_adapters(case, seed)
        state["scale"] = torch.rand(count, generator=gen, device="cuda") + 0.5  # each adapter's own
        if op == "adapters":
            state["base"] = randn(rows, n).to(TYPES[case["out"]])
            if case["x"] == "e4m3":
                x, state["scale_x"] = _quantize(x.float())
                x = _pitched(x)
        else:
            # The step's forward pass kept x A^T; the shared product's backward pass has given its gradient of x.
            state["hidden"] = _hidden(x.float(), state["a"].float(), state["ids"]).sum(dim=1)
            state["dout"] = _gradients(rows, n, gen, kind)
            state["base"] = _gradients(rows, k, gen, TYPES[case["out"]])
        state["x"] = x
        return state
    rows, cols, dtype = case["rows"], case["cols"], TYPES[case["in"]]
    state["x"] = _activations(rows, cols, gen, dtype)
    if case["residual"] and op != "norm_bwd":
        state["residual"] = (randn(rows, cols) * 2).to(dtype)
    if op == "dropout":
        # A training program's seed, and a number of its own for each dropout of a step.
        state["seed"], state["offset"] = 0x1234567 * (seed + 1), (seed << 33) + 5
        return state
    state["weight"] = 1 + 0.1 * randn(cols)
    if op == "norm_bwd":
        state["rstd"] = _rstd(state["x"].float())
        state["dy"] = _gradients(rows, cols, gen, dtype)
        if case["residual"]:
            state["dresidual"] = _gradients(rows, cols, gen, dtype)
    return state


# ----- the plain forms -------------------------------------------------------

def _quantize(x):
    rows, cols = x.shape
    blocks = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    amax = blocks.abs().amax(dim=2)
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp(min=SMALLEST)  # by a scalar, torch multiplies by 1 / 448
    q = (blocks / scale[:, :, None]).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(rows, -1)[:, :cols].contiguous()
    return q.view(torch.float8_e4m3fn), scale.t().contiguous()


def _rstd(h):
    return 1 / torch.sqrt((h * h).mean(dim=1) + EPS)


def _norm(s):
    """(y, h, rstd): h is rounded to its type, as the stream holds it, and that is what is normalised."""
    h = s["x"]
    if "residual" in s:
        h = (h.float() + s["residual"].float()).to(h.dtype)
    rstd = _rstd(h.float())
    return h.float() * rstd[:, None] * s["weight"], h, rstd


def _hidden(x, a, ids):
    """x A^T of every adapter, zeros but for each row's own: (rows, count, rank)."""
    count, rank, k = a.shape
    each = (x @ a.reshape(count * rank, k).t()).view(-1, count, rank)
    mine = ids[:, None] == torch.arange(count, device=ids.device)
    return torch.where(mine[:, :, None], each, 0.0)


def _adapters(s):
    x = s["x"].float()
    if "scale_x" in s:
        x = x * s["scale_x"].t().repeat_interleave(BLOCK, dim=1)[:, :x.shape[1]]
    h = _hidden(x, s["a"].float(), s["ids"]) * s["scale"][:, None]
    b = s["b"].float().transpose(1, 2).reshape(-1, s["b"].shape[1])
    return s["base"].float() + h.view(h.shape[0], -1) @ b


def _adapters_backward(s):
    dout, x, a, b, ids = s["dout"].float(), s["x"].float(), s["a"].float(), s["b"].float(), s["ids"]
    count, rank, k = a.shape
    bt = b.transpose(1, 2).contiguous()
    dh = (_hidden(dout, bt, ids) * s["scale"][:, None]).view(-1, count * rank)
    mine = ids[:, None] == torch.arange(count, device=ids.device)
    h = torch.where(mine, s["scale"], 0.0)[:, :, None] * s["hidden"][:, None, :]
    dx = s["base"].float() + dh @ a.view(count * rank, k)
    da = (dh.t() @ x).view(count, rank, k)
    db = (h.view(-1, count * rank).t() @ dout).view(count, rank, -1).transpose(1, 2).contiguous()
    return dx, da, db


def _philox(counter, key):
    """Philox4x32-10 on 32-bit words held in int64: products wrap, which leaves both halves in place."""
    low = 0xFFFFFFFF
    c0, c1, c2, c3 = counter
    k0, k1 = key
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & low) ^ c1 ^ k0, p1 & low, (p0 >> 32 & low) ^ c3 ^ k1, p0 & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return c0, c1, c2, c3


def _threshold(p):
    return int(p * 65536 + 0.5)


def _dropout(s):
    x, p, seed, offset = s["x"], s["case"]["p"], s["seed"], s["offset"]
    rows, cols = x.shape
    row = torch.arange(rows, device=x.device)[:, None]
    block = torch.arange(-(-cols // 8), device=x.device)[None, :]
    low = 0xFFFFFFFF
    zero = torch.zeros_like(row * block)
    words = _philox((block + zero, row + zero, zero + (offset & low), zero + (offset >> 32 & low)),
                    (seed & low, seed >> 32 & low))
    bits = torch.stack([w >> shift & 0xFFFF for w in words for shift in (0, 16)], dim=2).view(rows, -1)[:, :cols]
    t = _threshold(p)
    y = torch.where(bits >= t, x.float() * (65536 / (65536 - t)), 0.0)
    return y + s["residual"].float() if "residual" in s else y


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "adapters":
        return _adapters(s).to(TYPES[case["out"]])
    if op == "adapters_bwd":
        dx, da, db = _adapters_backward(s)
        return {"dx": dx.to(TYPES[case["out"]]), "da": da, "db": db}
    if op == "dropout":
        return _dropout(s).to(s["x"].dtype)
    if op == "norm_bwd":
        xhat = s["x"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["weight"]
        dx = (g - xhat * (g * xhat).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
        if "dresidual" in s:
            dx = dx + s["dresidual"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(dim=0)}
    y, h, rstd = _norm(s)
    out = {"h": h} if "residual" in s else {}
    if op == "norm":
        return {**out, "y": y.to(h.dtype), "rstd": rstd}
    q, scale = _quantize(y)
    return {**out, "q": q, "scale": scale}


def _run_own(s):
    import lds_tiled_matrix_amd as X
    case, op = s["case"], s["case"]["op"]
    if op == "adapters":
        return X.adapters(s["x"], s["a"], s["b"], s["ids"], base=s["base"], scale=s["scale"], scale_x=s.get("scale_x"))
    if op == "adapters_bwd":
        dx, da, db = X.adapters_backward(s["dout"], s["x"], s["a"], s["b"], s["ids"], s["hidden"], base=s["base"],
                                         scale=s["scale"])
        return {"dx": dx, "da": da, "db": db}
    if op == "dropout":
        return X.dropout(s["x"], case["p"], s["seed"], offset=s["offset"], residual=s.get("residual"))
    if op == "norm_bwd":
        dx, dweight = X.rms_norm_backward(s["dy"], s["x"], s["rstd"], s["weight"], dresidual=s.get("dresidual"))
        return {"dx": dx, "dweight": dweight}
    if op == "norm":
        got = X.rms_norm(s["x"], s["weight"], residual=s.get("residual"), eps=EPS, stats=True)
        return dict(zip(("y", "h", "rstd") if "residual" in s else ("y", "rstd"), got))
    got = X.rms_norm_quantize(s["x"], s["weight"], residual=s.get("residual"), eps=EPS)
    return dict(zip(("q", "scale", "h"), got))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----- what a pass cannot do without -----------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
    if op in ("adapters", "adapters_bwd"):
        m, k, n, rank = case["rows"], case["k"], case["n"], case["rank"]
        used = min(case["requests"], case["count"])
        weights, outs = used * rank * (k + n) * size[case["type"]], size[case["out"]]
        if op == "adapters":
            read = m * k * size[case["x"]] + (4 * m * -(-k // BLOCK) if case["x"] == "e4m3" else 0)
            return {"bytes": read + weights + 2 * m * n * outs + 4 * m, "flops": 2 * m * rank * (k + n)}
        read = m * (k + n) * size[case["type"]] + weights + 4 * m * (rank + 1)
        return {"bytes": read + 2 * m * k * outs + 4 * case["count"] * rank * (k + n), "flops": 4 * m * rank * (k + n)}
    rows, cols = case["rows"], case["cols"]
    values, each = rows * cols, size[case["in"]]
    if op == "dropout":
        # ten rounds of four products and six other operations for eight elements, and three for each element
        return {"bytes": values * each * (3 if case["residual"] else 2), "flops": 16 * values}
    if op == "norm_bwd":
        return {"bytes": values * each * (4 if case["residual"] else 3) + 4 * rows + 8 * cols, "flops": 10 * values}
    more = 3 if case["residual"] else 1  # x, the residual and their sum, or x
    if op == "norm":
        return {"bytes": values * each * (more + 1) + 4 * (rows + cols), "flops": 6 * values}
    return {"bytes": values * (each * more + 1) + 4 * (rows * -(-cols // BLOCK) + cols), "flops": 8 * values}


# ----- the definitions in 64 bits --------------------------------------------

def _exact_quantize(y):
    """The scale and each quotient are numbers of 32 bits by definition."""
    rows, cols = y.shape
    whole = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=y.device)
    whole[:, :cols] = y
    amax = whole.abs().reshape(rows, -1, BLOCK).amax(dim=2)
    scale = torch.maximum((amax / E4M3_MAX).float(), torch.tensor(SMALLEST, device=y.device)).double()
    value = (whole / scale.repeat_interleave(BLOCK, 1)).float().double()[:, :cols]
    # e4m3: four significant bits down to 2^-6, then steps of 2^-9, ties to even
    _, exponent = torch.frexp(value)
    step = torch.ldexp(torch.ones_like(value), exponent.clamp(min=-5) - 4)
    return torch.round(value / step) * step, scale.t()


def _exact_mask(rows, cols, p, seed, offset):
    """The mask from the definition, each product put together from 16-bit halves, for all eight places of a block."""
    col = torch.arange(cols, device="cuda")
    words = [(col // 8).expand(rows, cols), torch.arange(rows, device="cuda")[:, None].expand(rows, cols),
             offset % 2 ** 32, offset // 2 ** 32 % 2 ** 32]

    def multiply(word, by):
        high, low = word // 65536, word % 65536
        under = low * (by % 65536)
        middle = high * (by % 65536) + low * (by // 65536) + under // 65536
        return high * (by // 65536) + middle // 65536, middle % 65536 * 65536 + under % 65536

    for turn in range(10):
        keys = [(seed + turn * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + turn * 0xBB67AE85) % 2 ** 32]
        first, second = multiply(words[0], 0xD2511F53), multiply(words[2], 0xCD9E8D57)
        words = [second[0] ^ words[1] ^ keys[0], second[1], first[0] ^ words[3] ^ keys[1], first[1]]
    half = torch.zeros(rows, cols, dtype=torch.int64, device="cuda")
    for place in range(8):
        half[:, place::8] = words[place // 2][:, place::8] // 65536 ** (place % 2) % 65536
    return half >= _threshold(p)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("adapters", "adapters_bwd"):
        x, a, b, scale = (s[v].double() for v in ("x", "a", "b", "scale"))
        out = s["base"].double()
        if op == "adapters":
            if "scale_x" in s:
                x = x * s["scale_x"].double()[torch.arange(case["k"], device="cuda") // BLOCK].t()
            for l in range(case["count"]):
                at = torch.nonzero(s["ids"] == l).flatten()
                out[at] += scale[l] * (x[at] @ a[l].t()) @ b[l].t()
            return out
        dout, hidden = s["dout"].double(), s["hidden"].double()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for l in range(case["count"]):
            at = torch.nonzero(s["ids"] == l).flatten()
            dh = scale[l] * (dout[at] @ b[l])
            out[at] += dh @ a[l]
            da[l] = dh.t() @ x[at]
            db[l] = scale[l] * (dout[at].t() @ hidden[at])
        return {"dx": out, "da": da, "db": db}
    x = s["x"].double()
    if op == "dropout":
        t = _threshold(case["p"])
        kept = _exact_mask(*x.shape, case["p"], s["seed"], s["offset"])
        x = x * kept.double() * 65536 / (65536 - t)
        return x + s["residual"].double() if "residual" in s else x
    weight, cols = s["weight"].double(), case["cols"]
    if op == "norm_bwd":
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        g = dy * weight
        dx = rstd * g - x * rstd ** 3 * (g * x).sum(dim=1, keepdim=True) / cols
        if "dresidual" in s:
            dx += s["dresidual"].double()
        return {"dx": dx, "dweight": (dy * x * rstd).sum(dim=0)}
    out = {}
    if "residual" in s:
        x = (x + s["residual"].double()).to(s["x"].dtype).double()  # the stream holds it in its own type
        out["h"] = x
    rstd = ((x ** 2).sum(dim=1) / cols + EPS) ** -0.5
    y = x * rstd[:, None] * weight
    if op == "norm":
        return {**out, "y": y, "rstd": rstd}
    q, scale = _exact_quantize(y)
    return {**out, "q": q, "scale": scale}
