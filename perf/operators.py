"""Performance cases of the linear-layer operators: block quantisation to 8
bits, the 8-bit linear layer (forward, and with its gradient) and the
orthogonalised update.

``run`` computes a case either with the library's calls (``own = True``) or in
plain form: elementary torch operations in 32 bits, rounded once at the end.
``exact`` is the operators' definition in 64 bits.

Definitions (F = 448 for e4m3, 57344 for e5m2; a block that the edge cuts is
shorter):
  quantize   ac = max(max |x| over the block, 2^-96), r = F / ac and scale = ac / F,
             both 32-bit numbers, q = x r rounded to nearest even in 8 bits (r is
             part of the definition: with its rounding left out, values that lie
             between two 8-bit ones would go the other way).  "row" blocks are 1 x 128
             along a row, "square" ones 128 x 128; the transposed operand is x^T
             with blocks of its own rows, or with the same square ones.
             Scales of row blocks are stored (ceil(K / 128), M), of square
             ones (ceil(M / 128), ceil(K / 128)).
  linear     y = x W^T: x quantised in row blocks, W given in square ones.
  training   y as above from W unquantised; dx = dy W with dy in row blocks and
             W in square ones; dW = dy^T x with both quantised along the tokens.
  update     X = G / (|G|_F + eps), then `steps` times, with A = X X^T (X^T X when
             G is tall): X = a X + (b A + c A^2) X.
"""
import math

import torch

own = False

BLOCK = 128
AC_MIN = 2.0 ** -96
F_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
F_TYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # activations of a training step, read by the forward product and, transposed, by the weight's gradient
        {"name": "quant activations", "op": "quantize", "M": 8192, "K": 4096, "dtype": "bf16", "block": "row",
         "fmt": "e4m3", "both": True},
        # weights after an optimiser step, for the forward and the data gradient
        {"name": "quant weights", "op": "quantize", "M": 10240, "K": 4096, "dtype": "f32", "block": "square",
         "fmt": "e4m3", "both": True},
        # a short ragged prompt
        {"name": "quant ragged", "op": "quantize", "M": 77, "K": 1000, "dtype": "bf16", "block": "row",
         "fmt": "e5m2", "both": False},
        # one token of one sequence: latency
        {"name": "linear 1 token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # a decoding batch through a wide layer
        {"name": "linear 13 tokens", "op": "linear", "M": 13, "N": 10240, "K": 4096, "dtype": "bf16"},
        # a short prompt, odd everywhere
        {"name": "linear ragged", "op": "linear", "M": 333, "N": 1111, "K": 1999, "dtype": "f16"},
        # a long prompt
        {"name": "linear long", "op": "linear", "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16"},
        # forward and backward of a layer in a training step
        {"name": "train layer", "op": "train", "M": 8192, "N": 10240, "K": 4096, "dtype": "bf16"},
        # a small layer on a ragged number of tokens
        {"name": "train ragged", "op": "train", "M": 1001, "N": 1024, "K": 600, "dtype": "bf16"},
        # the update of a large square weight from its 32-bit gradient
        {"name": "update square", "op": "update", "batch": 1, "M": 4096, "N": 4096, "dtype": "f32", "steps": 5},
        # a stack of tall matrices of one shape
        {"name": "update stack", "op": "update", "batch": 6, "M": 2048, "N": 512, "dtype": "bf16", "steps": 5},
        # one small odd matrix: latency
        {"name": "update small", "op": "update", "batch": 1, "M": 100, "N": 333, "dtype": "bf16", "steps": 5},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A size spread over its logarithm: half of them any whole number, half a multiple of 64."""
    v = _log_int(rng, low, high)
    v = max(low, v // 64 * 64) if v >= 128 and rng.random() < 0.5 else v
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "train", "update"])
    if op == "quantize":
        return {"op": op, "M": _size(rng, 1, 8192), "K": _size(rng, 64, 4096),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "block": rng.choice(["row", "square"]),
                "fmt": rng.choice(["e4m3", "e5m2"]), "both": rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 256, 8192), "K": _size(rng, 256, 8192),
                "dtype": rng.choice(["bf16", "f16"])}
    if op == "train":
        return {"op": op, "M": _size(rng, 64, 8192), "N": _size(rng, 128, 8192), "K": _size(rng, 128, 4096),
                "dtype": "bf16"}
    m, n = _size(rng, 32, 4096), _size(rng, 32, 4096)
    batch = max(1, min(_log_int(rng, 1, 16), (1 << 24) // (m * n)))
    return {"op": op, "batch": batch, "M": m, "N": n, "dtype": rng.choice(["bf16", "f32"]), "steps": 5}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _spread(g, rows, cols, heavy):
    """Normal values whose rows and columns differ in size, as activations (a few columns far larger) and gradients do."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    if heavy:
        x *= 1.0 + 30.0 * (torch.rand((1, cols), generator=g, device="cuda") < 0.01)
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    op, dtype = case["op"], TYPES[case["dtype"]]
    if op == "quantize":
        state["x"] = _spread(g, case["M"], case["K"], case["block"] == "row").to(dtype)
        return state
    if op == "update":
        b, m, n = case["batch"], case["M"], case["N"]
        # a gradient: full-rank noise and a few strong directions
        k = max(1, min(m, n) // 16)
        u = torch.randn((b, m, k), generator=g, device="cuda") * torch.exp(-0.2 * torch.arange(k, device="cuda"))
        x = torch.randn((b, m, n), generator=g, device="cuda")
        x += 3.0 * u @ torch.randn((b, k, n), generator=g, device="cuda") / math.sqrt(k)
        state["x"] = (1e-3 * x if b > 1 else 1e-3 * x[0]).to(dtype)
        return state
    m, n, k = case["M"], case["N"], case["K"]
    state["x"] = _spread(g, m, k, True).to(dtype)
    w = torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)
    if op == "train":
        state["w"] = w.to(dtype)
        state["dy"] = (1e-2 * _spread(g, m, n, False)).to(dtype)
        return state
    # the weights a serving program keeps: 8 bits in rows of a multiple of 16 bytes, square blocks
    q, s = _quantize(w, "square", "e4m3")
    kept = torch.zeros((n, (k + 15) // 16 * 16), dtype=q.dtype, device="cuda")
    kept[:, :k] = q
    state["qw"], state["sw"] = kept[:, :k], s
    return state


# ---- the plain form -----------------------------------------------------------
def _per_element(scales, block, m, k):
    """One value an element from the scales of an m x k matrix."""
    if block == "row":
        return scales.t().repeat_interleave(BLOCK, 1)[:, :k]
    return scales.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:m, :k]


def _quantize(x, block, fmt):
    m, k = x.shape
    kb, mb = _blocks(k), _blocks(m)
    a = torch.nn.functional.pad(x.float().abs(), (0, kb * BLOCK - k, 0, mb * BLOCK - m if block == "square" else 0))
    if block == "row":
        ac = a.view(m, kb, BLOCK).amax(2).t().contiguous()
    else:
        ac = a.view(mb, BLOCK, kb, BLOCK).amax((1, 3))
    ac = ac.clamp_min(AC_MIN)
    f = F_MAX[fmt]
    top = torch.full_like(ac, f)  # a tensor: torch divides by a plain number through its rounded reciprocal
    q = (x.float() * _per_element(top / ac, block, m, k)).clamp(-f, f).to(F_TYPE[fmt])
    return q, ac / top


def _values(q, scales, block):
    return q.float() * _per_element(scales, block, *q.shape)


def _rounded(x, block):
    """x as 8 bits hold it."""
    return _values(*_quantize(x, block, "e4m3"), block)


def _update(g, steps):
    a, b, c = COEFFICIENTS
    x = g.float()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    for _ in range(steps):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.mT if tall else x).to(torch.bfloat16)


def _plain(state):
    case, x = state["case"], state["x"]
    if case["op"] == "quantize":
        out = list(_quantize(x, case["block"], case["fmt"]))
        if case["both"]:
            out += _quantize(x.t(), case["block"], case["fmt"])
        return out
    if case["op"] == "linear":
        y = _rounded(x, "row") @ _values(state["qw"], state["sw"], "square").t()
        return [y.to(x.dtype)]
    if case["op"] == "train":
        w, dy = state["w"], state["dy"]
        w8 = _rounded(w, "square")
        y = _rounded(x, "row") @ w8.t()
        dx = _rounded(dy, "row") @ w8
        dw = _rounded(dy.t(), "row") @ _rounded(x.t(), "row").t()
        return [y.to(x.dtype), dx.to(x.dtype), dw]
    return [_update(x, case["steps"])]


def run(state):
    if not own:
        return _plain(state)
    import thread_block_smem_gb300 as swz
    case, x = state["case"], state["x"]
    if case["op"] == "quantize":
        out = swz.quantize_fp8(x, block=case["block"], fmt=case["fmt"], transposed=case["both"])
        return list(out)
    if case["op"] == "linear":
        return [swz.linear_fp8(x, state["qw"], state["sw"])]
    if case["op"] == "train":
        y, saved = swz.linear_fp8_forward(x, state["w"])
        dx, dw = swz.linear_fp8_backward(state["dy"], saved)
        return [y, dx, dw]
    return [swz.newton_schulz(x, steps=case["steps"], coefficients=COEFFICIENTS, eps=EPS)]


# ---- the definition in 64 bits --------------------------------------------------
def _exact_q(x, square, fmt):
    """The 8-bit values (as 64-bit numbers) and scales, block by block along K, as (M, KB) or (MB, KB)."""
    x = x.double()
    m, k = x.shape
    top = torch.tensor(F_MAX[fmt], dtype=x.dtype, device=x.device)
    q, scales = torch.empty_like(x), []
    for k0 in range(0, k, BLOCK):
        part = x[:, k0:k0 + BLOCK]
        big = part.abs().max(1, keepdim=True).values
        if square:
            big = torch.cat([rows.max().expand(rows.shape[0], 1) for rows in big.split(BLOCK)])
        big = big.clamp(min=AC_MIN)
        r = (top / big).float().double()
        q[:, k0:k0 + BLOCK] = (part * r).clamp(-F_MAX[fmt], F_MAX[fmt]).to(F_TYPE[fmt]).double()
        scales.append((big / top).float().double())
    return q, torch.cat(scales, 1)


def _exact_values(x, square):
    q, s = _exact_q(x, square, "e4m3")
    return torch.cat([q[:, i * BLOCK:(i + 1) * BLOCK] * s[:, i:i + 1] for i in range(s.shape[1])], 1)


def exact(case, seed):
    state = prepare(case, seed)
    x = state["x"]
    if case["op"] == "quantize":
        out = []
        for v in ([x, x.t()] if case["both"] else [x]):
            q, s = _exact_q(v, case["block"] == "square", case["fmt"])
            out += [q, s[::BLOCK].contiguous() if case["block"] == "square" else s.t().contiguous()]
        return out
    if case["op"] == "linear":
        q, s = state["qw"].double(), state["sw"].double()
        x8 = _exact_values(x, False)
        y = torch.zeros((x.shape[0], q.shape[0]), dtype=torch.float64, device=x.device)
        for i in range(s.shape[1]):
            cols = slice(i * BLOCK, (i + 1) * BLOCK)
            rows = s[:, i:i + 1].expand(-1, BLOCK).reshape(-1, 1)[: q.shape[0]]
            y += x8[:, cols] @ (q[:, cols] * rows).t()
        return [y]
    if case["op"] == "train":
        w8 = _exact_values(state["w"], True)
        dy = state["dy"]
        y = _exact_values(x, False) @ w8.t()
        dx = _exact_values(dy, False) @ w8
        return [y, dx, _exact_values(dy.t(), False) @ _exact_values(x.t(), False).t()]
    v = x.double()
    v = v / (torch.linalg.matrix_norm(v, keepdim=True) + EPS)
    side = min(v.shape[-2:])
    a, b, c = COEFFICIENTS
    eye = torch.eye(side, dtype=v.dtype, device=v.device)
    for _ in range(case["steps"]):
        if v.shape[-2] <= v.shape[-1]:
            p = torch.matmul(v, v.mT)
            v = torch.matmul(a * eye + torch.matmul(p, b * eye + c * p), v)
        else:
            p = torch.matmul(v.mT, v)
            v = torch.matmul(v, a * eye + torch.matmul(p, b * eye + c * p))
    return [v]


def work(case):
    """Bytes and operations that a pass cannot do without: each operand once;
    symmetric products by half; 8-bit products counted as they are."""
    op, m = case["op"], case["M"]
    size = SIZE[case["dtype"]]
    if op == "quantize":
        k = case["K"]
        square = case["block"] == "square"
        sides = [(m, k), (k, m)] if case["both"] else [(m, k)]
        scales = sum(4 * _blocks(c) * (_blocks(r) if square else r) for r, c in sides)
        return {"bytes": m * k * (size + len(sides)) + scales, "flops": 2 * m * k * len(sides)}
    n = case["N"]
    if op == "linear":
        k = case["K"]
        return {"bytes": size * m * (k + n) + n * k + 4 * _blocks(n) * _blocks(k), "flops": 2 * m * n * k}
    if op == "train":
        k = case["K"]
        return {"bytes": size * (2 * m * k + 2 * m * n + n * k) + 4 * n * k, "flops": 6 * m * n * k}
    b, s, t = case["batch"], min(m, n), max(m, n)
    return {"bytes": b * m * n * (size + 2), "flops": b * case["steps"] * (s * s * t + s ** 3 + 2 * s * s * t)}
