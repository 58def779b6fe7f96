"""The operators of a linear layer's training and serving in 8 bits, as they are measured.

Three operators, each reached through the package's public functions where
``own`` is true and computed here in elementary 32-bit torch operations where
it is false:

* ``quantize``: blocks of 128 values of a matrix to 8-bit floating point with
  one fp32 scale each, along the rows, and in the same pass along the columns
  (the transposed matrix) for the products of the backward pass.
* ``gemm_scaled``: ``C = A @ B.T`` of two such matrices, every block of 128
  along K weighted with its scales.
* ``orthogonalize``: the Newton-Schulz iteration that replaces a matrix's
  singular values by values near one (the update of the Muon optimiser).
"""
import math

import torch

own = False

BLOCK = 128
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOAT8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SMALLEST_AMAX = 2.0 ** -100  # a block with nothing larger is scaled as if it held this
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ------------------------------------------------------------------ the cases
def _quantize(name, rows, cols, dtype="bf16", blocks="row", transposed=False, pow2=False, kind="e4m3"):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype, "blocks": blocks,
            "transposed": transposed, "pow2": pow2, "kind": kind}


def _gemm(name, M, N, K, out="bf16", a_blocks="row", b_blocks="square", a_kind="e4m3", pow2=False):
    return {"name": name, "op": "gemm_scaled", "M": M, "N": N, "K": K, "out": out, "a_blocks": a_blocks,
            "b_blocks": b_blocks, "a_kind": a_kind, "pow2": pow2}


def _ortho(name, batch, rows, cols, dtype="bf16"):
    return {"name": name, "op": "orthogonalize", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # the activations of one generated token before a layer's product: latency
        _quantize("quantize token", 1, 8192),
        # the activations of a training step: rows for the forward product, columns for the weight's gradient
        _quantize("quantize activations", 8192, 8192, transposed=True),
        # the largest weight after an optimiser step: one set of scales serves it and its transpose
        _quantize("quantize weight", 28672, 8192, blocks="square", transposed=True),
        # one token through an attention output projection: the weight's bytes are the time
        _gemm("gemm token", 1, 8192, 8192),
        # a decode batch through the MLP's up projection
        _gemm("gemm decode", 64, 28672, 8192, pow2=True),
        # a prompt, or a training step's forward product
        _gemm("gemm prefill", 8192, 28672, 8192),
        # the weight's gradient: both operands scaled along the tokens, fp32 out for the optimiser
        _gemm("gemm weight gradient", 8192, 8192, 8192, out="fp32", b_blocks="row", a_kind="e5m2"),
        # no size a multiple of anything: a last partial batch on an odd layer
        _gemm("gemm ragged", 333, 1000, 5005, out="fp16"),
        # one small fp32 momentum of odd size: latency of fifteen dependent products
        _ortho("ortho odd", 1, 300, 1000, dtype="fp32"),
        # a stack of equal small matrices (heads or experts)
        _ortho("ortho stack", 16, 512, 1344),
        # a square weight's momentum
        _ortho("ortho square", 1, 4096, 4096),
        # an MLP weight's momentum, more rows than columns
        _ortho("ortho tall", 1, 28672, 4096),
    ]


def _size(rng, low, high):
    """A size from low to high, spread over the logarithm; half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["quantize", "gemm_scaled", "orthogonalize"])
    if op == "quantize":
        while True:
            rows, cols = _size(rng, 1, 28672), _size(rng, 32, 28672)
            if rows * cols <= 28672 * 8192:
                break
        case = _quantize("", rows, cols, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["row", "row", "square"]),
                         rng.random() < 0.5, rng.random() < 0.5, rng.choice(["e4m3", "e4m3", "e5m2"]))
    elif op == "gemm_scaled":
        while True:
            M, N, K = _size(rng, 1, 8192), _size(rng, 64, 28672), _size(rng, 128, 28672)
            if M * N * K <= 8192 * 28672 * 8192 and N * K <= 28672 * 8192:
                break
        case = _gemm("", M, N, K, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["row", "row", "square"]),
                     rng.choice(["square", "square", "row"]), rng.choice(["e4m3", "e4m3", "e5m2"]), rng.random() < 0.5)
    else:
        while True:
            batch = rng.choice([1, 1, 1, 2, 5, 16, 32])
            rows, cols = _size(rng, 16, 8192), _size(rng, 16, 28672)
            if rng.random() < 0.5:
                rows, cols = cols, rows
            m, n = min(rows, cols), max(rows, cols)
            if m <= 4096 and batch * (3 * m * m * n + m ** 3) <= 3 * 4096 * 4096 * 28672 + 4096 ** 3 and batch * m * n <= 28672 * 4096:
                break
        case = _ortho("", batch, rows, cols, rng.choice(["bf16", "bf16", "fp32"]))
    del case["name"]
    return case


def work(case):
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        kb, rb = -(-C // BLOCK), -(-R // BLOCK)
        scales = kb * R if case["blocks"] == "row" else kb * rb
        if case["transposed"]:
            scales += rb * C if case["blocks"] == "row" else kb * rb
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": R * C * (size + 1 + case["transposed"]) + 4 * scales, "flops": 2 * R * C}
    if case["op"] == "gemm_scaled":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        scales = kb * (M if case["a_blocks"] == "row" else -(-M // BLOCK))
        scales += kb * (N if case["b_blocks"] == "row" else -(-N // BLOCK))
        return {"bytes": M * K + N * K + M * N * (4 if case["out"] == "fp32" else 2) + 4 * scales, "flops": 2 * M * N * K}
    m, n = sorted((case["rows"], case["cols"]))
    # a step: X X^T and its square, symmetric (half each), and the product with X
    flops = case["batch"] * STEPS * (m * m * n + m ** 3 + 2 * m * m * n)
    return {"bytes": case["batch"] * m * n * ((4 if case["dtype"] == "fp32" else 2) + 2), "flops": flops}


# ----------------------------------------------------------------- the inputs
def _padded(t, multiple):
    """t's values in rows that lie a multiple of `multiple` elements apart."""
    cols = t.shape[1]
    wide = torch.zeros(t.shape[0], -(-cols // multiple) * multiple, dtype=t.dtype, device=t.device)
    wide[:, :cols] = t
    return wide[:, :cols]


def _activations(rows, cols, gen):
    """N(0, 1), with a few columns tens of times larger, as activations have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.002
    return x * torch.where(loud, 30.0, 1.0)


def _weights(rows, cols, gen):
    return 0.02 * torch.randn(rows, cols, generator=gen, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "quantize":
        make = _weights if case["blocks"] == "square" else _activations
        return {"case": case, "x": _padded(make(case["rows"], case["cols"], gen).to(DTYPES[case["dtype"]]), 8)}
    if case["op"] == "gemm_scaled":
        a = _activations(case["M"], case["K"], gen)
        b = (_weights if case["b_blocks"] == "square" else _activations)(case["N"], case["K"], gen)
        qa, sa = _plain_blocks(a, case["a_blocks"], case["pow2"], case["a_kind"])
        del a
        qb, sb = _plain_blocks(b, case["b_blocks"], case["pow2"], "e4m3")
        del b
        return {"case": case, "a": _padded(qa.view(torch.uint8), 16).view(qa.dtype), "sa": _padded(sa, 4),
                "b": _padded(qb.view(torch.uint8), 16).view(qb.dtype), "sb": _padded(sb, 4)}
    B, R, C = case["batch"], case["rows"], case["cols"]
    # a momentum: noise, and a few directions that stand out of it
    g = torch.randn(B, R, C, generator=gen, device="cuda")
    u = torch.randn(B, R, 8, generator=gen, device="cuda")
    v = torch.randn(B, 8, C, generator=gen, device="cuda")
    g = 1e-3 * (g + 0.25 * torch.matmul(u, v))
    return {"case": case, "g": g.to(DTYPES[case["dtype"]])}


# ------------------------------------------------------------ the plain forms
def _blocked(x, along_rows):
    """x padded with zeros to whole blocks, as (row blocks, rows, column blocks, columns) of a block."""
    rows, cols = x.shape
    rb = BLOCK if along_rows else 1
    r, c = -(-rows // rb) * rb, -(-cols // BLOCK) * BLOCK
    full = torch.zeros(r, c, dtype=x.dtype, device=x.device)
    full[:rows, :cols] = x
    return full.view(r // rb, rb, c // BLOCK, BLOCK)


def _plain_blocks(x, blocks, pow2, kind):
    """(values in 8 bits, scales (column blocks, rows or row blocks)) of a matrix."""
    rows, cols = x.shape
    x4 = _blocked(x.float(), blocks == "square")
    amax = x4.abs().amax(dim=(1, 3)).clamp_min(SMALLEST_AMAX)
    limit = torch.full_like(amax, FLOAT8_MAX[kind])
    scale = amax / limit
    if pow2:  # the next power of two: any mantissa bits carry into the exponent
        bits = (scale.view(torch.int32) + 0x7FFFFF) & 0x7F800000
        scale = bits.view(torch.float32)
        factor = 1.0 / scale
    else:
        factor = limit / amax
    q = (x4 * factor[:, None, :, None]).to(FLOAT8[kind])
    q = q.view(torch.uint8).reshape(x4.shape[0] * x4.shape[1], -1)[:rows, :cols].view(FLOAT8[kind])
    return q, scale.t().contiguous()


def _plain_values(q, scale):
    """The fp32 values that 8-bit values and their scales stand for."""
    rows, cols = q.shape
    full = scale if scale.shape[1] == rows else scale.repeat_interleave(BLOCK, dim=1)[:, :rows]
    return q.float() * full.t().repeat_interleave(BLOCK, dim=1)[:, :cols]


def _plain_orthogonalize(g):
    x = g.float()
    wide = x.shape[-2] <= x.shape[-1]
    if not wide:
        x = x.mT
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        s = torch.matmul(x, x.mT)
        x = a * x + torch.matmul(b * s + c * torch.matmul(s, s), x)
    return (x if wide else x.mT).to(torch.bfloat16)


def run(state):
    case = state["case"]
    if own:
        import dense_gemm_blackwell_03_gb300 as bwgemm

        if case["op"] == "quantize":
            return list(bwgemm.quantize(state["x"], blocks=case["blocks"], transposed=case["transposed"], pow2=case["pow2"],
                                        dtype=FLOAT8[case["kind"]]))
        if case["op"] == "gemm_scaled":
            return bwgemm.gemm_scaled(state["a"], state["sa"], state["b"], state["sb"], out_dtype=DTYPES[case["out"]])
        return bwgemm.orthogonalize(state["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    if case["op"] == "quantize":
        x = state["x"]
        q, s = _plain_blocks(x, case["blocks"], case["pow2"], case["kind"])
        if not case["transposed"]:
            return [q, s]
        if case["blocks"] == "square":
            return [q, s, q.view(torch.uint8).t().contiguous().view(q.dtype), s.t().contiguous()]
        qt, st = _plain_blocks(x.t(), "row", case["pow2"], case["kind"])
        return [q, s, qt, st]
    if case["op"] == "gemm_scaled":
        c = torch.matmul(_plain_values(state["a"], state["sa"]), _plain_values(state["b"], state["sb"]).t())
        return c.to(DTYPES[case["out"]])
    return _plain_orthogonalize(state["g"])


# ----------------------------------------------------------------- in 64 bits
def _exact_round(v, kind):
    """The nearest 8-bit value, ties to the even one, by the format's definition."""
    mantissa, least = (3, -6) if kind == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(least).double() - mantissa)
    return torch.round(v / step) * step


def _exact_blocks(x, blocks, pow2, kind):
    rows, cols = x.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    scales = []
    for c in range(0, cols, BLOCK):
        part = x[:, c:c + BLOCK].double()
        amax = part.abs().amax(dim=1)
        if blocks == "square":
            amax = torch.stack([v.max() for v in amax.split(BLOCK)])
        scale = amax.clamp_min(SMALLEST_AMAX) / FLOAT8_MAX[kind]
        if pow2:
            part_of, e = torch.frexp(scale)
            scale = torch.exp2(e.double() - (part_of == 0.5).double())
        each = scale.repeat_interleave(BLOCK)[:rows] if blocks == "square" else scale
        out[:, c:c + BLOCK] = _exact_round(part / each[:, None], kind)
        scales.append(scale)
    return out, torch.stack(scales)


def _exact_values(q, scale):
    rows, cols = q.shape
    i = torch.arange(rows, device=q.device) // (1 if scale.shape[1] == rows else BLOCK)
    j = torch.arange(cols, device=q.device) // BLOCK
    return q.double() * scale.double()[j][:, i].t()


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        q, s = _exact_blocks(state["x"], case["blocks"], case["pow2"], case["kind"])
        if not case["transposed"]:
            return [q, s]
        if case["blocks"] == "square":
            return [q, s, q.t(), s.t()]
        return [q, s, *_exact_blocks(state["x"].t(), "row", case["pow2"], case["kind"])]
    if case["op"] == "gemm_scaled":
        return _exact_values(state["a"], state["sa"]) @ _exact_values(state["b"], state["sb"]).t()
    g = state["g"].double()
    m, n = sorted(g.shape[1:])
    if case["batch"] * STEPS * (4 * m * m * n + 2 * m ** 3) > 1.5e13:
        return None
    a, b, c = COEFFICIENTS
    done = []
    for x in g:
        x = x if x.shape[0] <= x.shape[1] else x.t()
        x = x / (torch.linalg.vector_norm(x) + EPS)
        for _ in range(STEPS):
            s = x @ x.t()
            x = a * x + b * (s @ x) + c * (s @ (s @ x))
        done.append(x if x.shape == g.shape[1:] else x.t())
    return torch.stack(done)
