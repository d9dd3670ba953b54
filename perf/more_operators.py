"""Performance cases of what stands around a linear layer: its product in 8-bit
integers with a scale for each token and channel, the layer norm before it with
its gradient, and the clipping of the gradients after it.

``run`` computes a case either with the library's calls (``own = True``) or in
plain form: elementary torch operations in 32 bits (in 64 where a value lies next
to a border), rounded once at the end.  ``exact`` is the operators' definition in
64 bits.

Definitions:
  quantize   for each row: ac = max(max |x|, 2^-96), r = 127 / ac and scale = ac / 127,
             both 32-bit numbers, q = x r (the exact product) rounded to the nearest
             whole number, ties to even.
  product    C[m, n] = sa[m] sb[n] sum over k of a[m, k] b[n, k].
  linear     the product of x quantised by rows (tokens) and W kept quantised by
             its rows (output channels).
  norm       y = (x - mean) rstd w + b by rows, rstd = 1 / sqrt(var + eps), var the
             mean square of x - mean.
  norm train also dx = rstd (g - mean(g) - xhat mean(g xhat)) with g = dy w and
             xhat = (x - mean) rstd, dw = sum of dy xhat and db = sum of dy over rows.
  clip       norm = sqrt(sum of the squares of all gradients), each gradient times
             min(1, max_norm / (norm + eps)).
"""
import math

import torch

own = False

AC_MIN = 2.0 ** -96
TOP = 127.0
NORM_EPS = 1e-5
CLIP_EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # activations of a long prompt, quantised once for the layers that read them
        {"name": "quant prompt", "op": "quantize", "M": 8192, "K": 4096, "dtype": "bf16"},
        # a short ragged prompt
        {"name": "quant ragged", "op": "quantize", "M": 77, "K": 1000, "dtype": "f32"},
        # one token of one sequence through a layer: latency
        {"name": "linear 1 token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # a short prompt, odd everywhere
        {"name": "linear ragged", "op": "linear", "M": 333, "N": 1111, "K": 1999, "dtype": "f16"},
        # a decoding batch, quantised before, through a wide layer
        {"name": "product 13 tokens", "op": "product", "M": 13, "N": 10240, "K": 4096, "dtype": "bf16"},
        # a long prompt, quantised before
        {"name": "product long", "op": "product", "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16"},
        # one token: latency
        {"name": "norm 1 token", "op": "norm", "M": 1, "N": 4096, "dtype": "bf16", "wtype": "bf16"},
        # a prompt with an odd width
        {"name": "norm ragged", "op": "norm", "M": 1001, "N": 1999, "dtype": "f16", "wtype": "f32"},
        # forward and backward in a training step
        {"name": "norm train", "op": "norm train", "M": 8192, "N": 4096, "dtype": "bf16", "wtype": "f32"},
        # a small network on a ragged number of tokens, all in 32 bits
        {"name": "norm train ragged", "op": "norm train", "M": 1001, "N": 600, "dtype": "f32", "wtype": "f32"},
        # the gradients of a network of eight blocks, clipped into the 32-bit buffers that its update reads
        {"name": "clip network", "op": "clip", "layers": 8, "width": 4096, "hidden": 10240, "dtype": "bf16",
         "out": "f32"},
        # those of one small block: latency
        {"name": "clip small", "op": "clip", "layers": 1, "width": 600, "hidden": 1024, "dtype": "f32", "out": "f32"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A size spread over its logarithm: half of them any whole number, half a multiple of 64."""
    v = _log_int(rng, low, high)
    return max(low, v // 64 * 64) if v >= 128 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "product", "norm", "norm train", "clip"])
    if op in ("linear", "product"):
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 256, 8192), "K": _size(rng, 256, 8192),
                "dtype": rng.choice(["bf16", "f16"])}
    if op == "clip":
        return {"op": op, "layers": rng.randint(1, 8), "width": _size(rng, 64, 4096), "hidden": _size(rng, 64, 10240),
                "dtype": rng.choice(["bf16", "f32"]), "out": rng.choice(["f32", "same"])}
    n = _size(rng, 64, 10240)
    m = _size(rng, 1, min(16384, (1 << 25) // n))
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "M": m, "K": n, "dtype": dtype}
    return {"op": op, "M": m, "N": n, "dtype": dtype, "wtype": rng.choice(["f32", dtype])}


def _activations(g, rows, cols, dtype):
    """Normal values whose rows differ in size, with a few columns far larger."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    x *= 1.0 + 30.0 * (torch.rand((1, cols), generator=g, device="cuda") < 0.01)
    return x.to(dtype)


def _kept(q):
    """8-bit values in rows of a multiple of 16 bytes, as a program keeps them."""
    m, k = q.shape
    kept = torch.zeros((m, (k + 15) // 16 * 16), dtype=torch.int8, device="cuda")
    kept[:, :k] = q
    return kept[:, :k]


def _shapes(case):
    """(shape, type) of the gradients: two weights, and the norm's weight and bias, a block."""
    w, h = case["width"], case["hidden"]
    return [((h, w), case["dtype"]), ((w, h), case["dtype"]), ((w,), "f32"), ((w,), "f32")] * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    op, dtype = case["op"], TYPES[case["dtype"]]
    if op == "clip":
        state["grads"] = []
        kinds = sorted({t if case["out"] == "same" else case["out"] for _, t in _shapes(case)})
        total = {t: 0 for t in kinds}
        at = []
        for shape, t in _shapes(case):
            n = math.prod(shape)
            x = torch.randn(n, generator=g, device="cuda", dtype=TYPES[t]).view(shape)
            state["grads"].append(x.mul_(0.02 * math.exp(torch.randn(1, generator=g, device="cuda").item())))
            t = t if case["out"] == "same" else case["out"]
            at.append((t, total[t], n, shape))
            total[t] += n
        # the buffers that the clipped gradients go to, one after another in one piece of memory for each type
        flat = {t: torch.zeros(total[t], dtype=TYPES[t], device="cuda") for t in kinds}
        state["flat"] = [flat[t] for t in kinds]
        state["out"] = [flat[t][o:o + n].view(shape) for t, o, n, shape in at]
        return state
    if op == "quantize":
        state["x"] = _activations(g, case["M"], case["K"], dtype)
        return state
    if op in ("norm", "norm train"):
        m, n = case["M"], case["N"]
        state["x"] = _activations(g, m, n, dtype)
        state["w"] = (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(TYPES[case["wtype"]])
        state["b"] = (0.2 * torch.randn(n, generator=g, device="cuda")).to(TYPES[case["wtype"]])
        if op == "norm train":
            state["dy"] = (1e-2 * torch.randn((m, n), generator=g, device="cuda")).to(dtype)
        return state
    m, n, k = case["M"], case["N"], case["K"]
    x = _activations(g, m, k, dtype)
    # the weights a serving program keeps
    q, state["sw"] = _quantize(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k))
    state["qw"] = _kept(q)
    if op == "linear":
        state["x"] = x
    else:
        q, state["sx"] = _quantize(x)
        state["qx"] = _kept(q)
    return state


# ---- the plain form -----------------------------------------------------------
def _quantize(x):
    ac = x.float().abs().amax(1).clamp_min(AC_MIN)
    top = torch.full_like(ac, TOP)  # a tensor: torch divides by a plain number through its rounded reciprocal
    # next to a border between two whole numbers 32 bits would go the wrong way
    q = (x.double() * (top / ac).double().unsqueeze(1)).round().to(torch.int8)
    return q, ac / top


def _product(qa, sa, qb, sb, dtype):
    return ((qa.float() @ qb.float().t()) * (sa.unsqueeze(1) * sb.unsqueeze(0))).to(dtype)


def _norm(x, w, b):
    x = x.float()
    d = x - x.mean(1, keepdim=True)
    rstd = 1.0 / (d.square().mean(1, keepdim=True) + NORM_EPS).sqrt()
    xhat = d * rstd
    return xhat * w.float() + b.float(), xhat, rstd


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        return list(_quantize(state["x"]))
    if op == "linear":
        return [_product(*_quantize(state["x"]), state["qw"], state["sw"], state["x"].dtype)]
    if op == "product":
        return [_product(state["qx"], state["sx"], state["qw"], state["sw"], TYPES[case["dtype"]])]
    if op == "clip":
        norm = torch.stack([x.float().square().sum() for x in state["grads"]]).sum().sqrt()
        factor = (1.0 / (norm + CLIP_EPS)).clamp_max(1.0)
        [o.copy_(x.float() * factor) for x, o in zip(state["grads"], state["out"])]
        return [norm, *state["flat"]]
    x, w = state["x"], state["w"]
    y, xhat, rstd = _norm(x, w, state["b"])
    if op == "norm":
        return [y.to(x.dtype)]
    dy = state["dy"].float()
    g = dy * w.float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return [y.to(x.dtype), dx.to(x.dtype), (dy * xhat).sum(0), dy.sum(0)]


def run(state):
    if not own:
        return _plain(state)
    import thread_block_smem_gb300 as swz
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        return list(swz.quantize_int8(state["x"]))
    if op == "linear":
        return [swz.linear_int8(state["x"], state["qw"], state["sw"])]
    if op == "product":
        return [swz.gemm_int8(state["qx"], state["sx"], state["qw"], state["sw"], out_dtype=TYPES[case["dtype"]])]
    if op == "clip":
        norm = swz.clip_grad_norm(state["grads"], 1.0, eps=CLIP_EPS, out=state["out"])
        return [norm, *state["flat"]]
    x, w = state["x"], state["w"]
    y, mean, rstd = swz.layer_norm_forward(x, w, state["b"], NORM_EPS)
    if op == "norm":
        return [y]
    return [y, *swz.layer_norm_backward(state["dy"], x, w, mean, rstd)]


# ---- the definition in 64 bits --------------------------------------------------
def _exact_rows(x):
    v = x.double()
    big = torch.maximum(v.max(1).values, -v.min(1).values).clamp(min=AC_MIN).unsqueeze(1)
    q = torch.round(v * (TOP / big).float().double())
    return q, (big / TOP).float()


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, s = _exact_rows(state["x"])
        return [q.to(torch.int8), s.flatten()]
    if op in ("linear", "product"):
        if op == "linear":
            q, s = _exact_rows(state["x"])
        else:
            q, s = state["qx"].double(), state["sx"].unsqueeze(1)
        return [torch.matmul(s.double() * q, state["qw"].double().t()) * state["sw"].double()]
    if op == "clip":
        norm = math.sqrt(sum(torch.linalg.vector_norm(x.double()).item() ** 2 for x in state["grads"]))
        factor = min(1.0, 1.0 / (norm + CLIP_EPS))
        kinds = [f.dtype for f in state["flat"]]
        return [torch.tensor(norm, dtype=torch.float64, device="cuda"),
                *(torch.cat([x.double().flatten() * factor for x, o in zip(state["grads"], state["out"])
                             if o.dtype == t]) for t in kinds)]
    x, w = state["x"].double(), state["w"].double()
    m = x.shape[1]
    mean = x.sum(1, keepdim=True) / m
    sigma = torch.sqrt(torch.var(x, 1, unbiased=False, keepdim=True) + NORM_EPS)
    xhat = (x - mean) / sigma
    y = torch.addcmul(state["b"].double(), xhat, w)
    if op == "norm":
        return [y]
    dy = state["dy"].double()
    g = dy * w
    along = torch.linalg.vecdot(g, xhat).unsqueeze(1) / m
    return [y, (g - g.sum(1, keepdim=True) / m - along * xhat) / sigma, torch.einsum("mn,mn->n", dy, xhat),
            torch.einsum("mn->n", dy)]


def work(case):
    """Bytes and operations that a pass cannot do without: each input read once, each output written once."""
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "clip":
        shapes = [(math.prod(s), SIZE[t]) for s, t in _shapes(case)]
        return {"bytes": sum(n * (e + (e if case["out"] == "same" else SIZE[case["out"]])) for n, e in shapes) + 4,
                "flops": 3 * sum(n for n, _ in shapes)}
    m = case["M"]
    if op == "quantize":
        return {"bytes": m * case["K"] * (size + 1) + 4 * m, "flops": 2 * m * case["K"]}
    n = case["N"]
    if op in ("linear", "product"):
        k = case["K"]
        return {"bytes": m * k * (size if op == "linear" else 1) + n * k + size * m * n
                + 4 * (n if op == "linear" else n + m), "flops": 2 * m * n * k}
    params = n * SIZE[case["wtype"]]
    if op == "norm":
        return {"bytes": 2 * m * n * size + 2 * params, "flops": 7 * m * n}
    return {"bytes": 5 * m * n * size + 2 * params + 8 * n, "flops": 18 * m * n}
