"""The operators of a gated feed-forward layer and of its serving in 8-bit integers, as they are measured.

Four operators, each reached through the package's public functions where
``own`` is true and computed here in elementary 32-bit torch operations where
it is false:

* ``gated_linear``: ``act(x @ w_gate.T) * (x @ w_up.T)``, both projections, the
  activation and the product of a gated feed-forward layer.
* ``gated_linear_backward``: the gradients of its input and of both weights.
* ``quantize_int8``: the rows of a matrix (tokens, or a weight's output
  channels) to 8-bit integers with one fp32 scale each.
* ``gemm_int8``: ``C = A @ B.T`` of two such matrices.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SMALLEST_AMAX = 2.0 ** -100  # a row with nothing larger is scaled as if it held this


# ------------------------------------------------------------------ the cases
def _gated(name, M, N, K, dtype="bf16", act="silu"):
    return {"name": name, "op": "gated_linear", "M": M, "N": N, "K": K, "dtype": dtype, "act": act}


def _backward(name, M, N, K, dtype="bf16", act="silu"):
    return {"name": name, "op": "gated_linear_backward", "M": M, "N": N, "K": K, "dtype": dtype, "act": act}


def _quantize(name, rows, cols, dtype="bf16"):
    return {"name": name, "op": "quantize_int8", "rows": rows, "cols": cols, "dtype": dtype}


def _gemm(name, M, N, K, out="bf16"):
    return {"name": name, "op": "gemm_int8", "M": M, "N": N, "K": K, "out": out}


def listed():
    return [
        # a few tokens through a small layer of odd size: the latency of the call
        _gated("gated small", 5, 1000, 520, dtype="fp16", act="gelu"),
        # one generated token: two weights' bytes are the time
        _gated("gated token", 1, 10240, 8192),
        # a decode batch through the largest feed-forward layer
        _gated("gated decode", 64, 28672, 8192),
        # a prompt, or a training step's forward pass
        _gated("gated prefill", 8192, 28672, 8192),
        # a training step's backward pass
        _backward("gated backward", 4096, 28672, 8192),
        # a last partial batch, no size a multiple of anything
        _backward("gated backward ragged", 333, 1000, 5005, dtype="fp16", act="gelu_tanh"),
        # the activations of one generated token before a layer's product: latency
        _quantize("int8 quantize token", 1, 8192),
        # the activations of a prompt
        _quantize("int8 quantize activations", 8192, 8192),
        # one token through an attention output projection
        _gemm("int8 token", 1, 8192, 8192),
        # a decode batch through the MLP's up projection
        _gemm("int8 decode", 64, 28672, 8192),
        # a prompt
        _gemm("int8 prefill", 8192, 28672, 8192),
        # a last partial batch on an odd layer
        _gemm("int8 ragged", 333, 1000, 5005, out="fp32"),
    ]


def _size(rng, low, high):
    """A size from low to high, spread over the logarithm; half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["gated_linear", "gated_linear", "gated_linear_backward", "quantize_int8", "gemm_int8", "gemm_int8"])
    if op == "quantize_int8":
        while True:
            rows, cols = _size(rng, 1, 28672), _size(rng, 32, 28672)
            if rows * cols <= 28672 * 8192:
                break
        case = _quantize("", rows, cols, rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    else:
        most = 8192 if op != "gated_linear_backward" else 4096
        while True:
            M, N, K = _size(rng, 1, most), _size(rng, 64, 28672), _size(rng, 64, 28672 if op == "gemm_int8" else 8192)
            if M * N * K <= most * 28672 * 8192 and N * K <= 28672 * 8192:
                break
        if op == "gemm_int8":
            case = _gemm("", M, N, K, rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        else:
            make = _gated if op == "gated_linear" else _backward
            case = make("", M, N, K, rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    del case["name"]
    return case


def work(case):
    if case["op"] == "quantize_int8":
        R, C = case["rows"], case["cols"]
        return {"bytes": R * C * ((4 if case["dtype"] == "fp32" else 2) + 1) + 4 * R, "flops": 2 * R * C}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gemm_int8":
        return {"bytes": M * K + N * K + M * N * (4 if case["out"] == "fp32" else 2) + 4 * (M + N), "flops": 2 * M * N * K}
    if case["op"] == "gated_linear":
        return {"bytes": 2 * (M * K + 2 * N * K + M * N), "flops": 4 * M * N * K}
    # dh, gate, up, x and both weights in; dx and both weights' gradients out
    return {"bytes": 2 * (3 * M * N + 2 * M * K + 4 * N * K), "flops": 8 * M * N * K}


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
    state = {"case": case}
    if case["op"] == "quantize_int8":
        state["x"] = _padded(_activations(case["rows"], case["cols"], gen).to(DTYPES[case["dtype"]]), 8)
        return state
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gemm_int8":
        a, state["sa"] = _plain_int8(_activations(M, K, gen))
        b, state["sb"] = _plain_int8(_weights(N, K, gen))
        state["a"], state["b"] = _padded(a, 16), _padded(b, 16)
        return state
    dtype = DTYPES[case["dtype"]]
    state["x"] = _padded(torch.randn(M, K, generator=gen, device="cuda").to(dtype), 8)  # what a norm gives
    state["wg"] = _padded(_weights(N, K, gen).to(dtype), 8)
    state["wu"] = _padded(_weights(N, K, gen).to(dtype), 8)
    if case["op"] == "gated_linear_backward":
        # what the forward pass kept, with the spread that such weights give, and the
        # gradient as a scaled loss has it
        spread = 0.02 * math.sqrt(K)
        state["gate"] = _padded((spread * torch.randn(M, N, generator=gen, device="cuda")).to(dtype), 8)
        state["up"] = _padded((spread * torch.randn(M, N, generator=gen, device="cuda")).to(dtype), 8)
        state["dh"] = _padded((0.1 * torch.randn(M, N, generator=gen, device="cuda")).to(dtype), 8)
    return state


# ------------------------------------------------------------ the plain forms
def _plain_int8(x):
    """(values, scales) of a matrix's rows.  In 64 bits: whether a value lies below or above
    the middle of two integers, or on it, is lost in 32."""
    amax = x.float().abs().amax(dim=1).clamp_min(SMALLEST_AMAX)
    q = torch.round(x.double() * 127.0 / amax.double()[:, None])
    return q.to(torch.int8), amax / 127.0


def _plain_act(act, g):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_slope(act, g):
    """The activation's derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def run(state):
    case = state["case"]
    if own:
        import dense_gemm_blackwell_03_gb300 as bwgemm

        if case["op"] == "quantize_int8":
            return list(bwgemm.quantize_int8(state["x"]))
        if case["op"] == "gemm_int8":
            return bwgemm.gemm_int8(state["a"], state["sa"], state["b"], state["sb"], out_dtype=DTYPES[case["out"]])
        if case["op"] == "gated_linear":
            return bwgemm.gated_linear(state["x"], state["wg"], state["wu"], activation=case["act"])
        return list(bwgemm.gated_linear_backward(state["dh"], state["gate"], state["up"], state["x"], state["wg"], state["wu"],
                                                 activation=case["act"]))
    if case["op"] == "quantize_int8":
        return list(_plain_int8(state["x"]))
    if case["op"] == "gemm_int8":
        sums = torch.matmul(state["a"].float(), state["b"].float().t())
        return (sums * state["sa"][:, None] * state["sb"]).to(DTYPES[case["out"]])
    x, wg, wu = state["x"].float(), state["wg"].float(), state["wu"].float()
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "gated_linear":
        return (_plain_act(case["act"], torch.matmul(x, wg.t())) * torch.matmul(x, wu.t())).to(dtype)
    g, dh = state["gate"].float(), state["dh"].float()
    dg = dh * state["up"].float() * _plain_slope(case["act"], g)
    du = dh * _plain_act(case["act"], g)
    return [(torch.matmul(dg, wg) + torch.matmul(du, wu)).to(dtype), torch.matmul(dg.t(), x).to(dtype),
            torch.matmul(du.t(), x).to(dtype)]


# ----------------------------------------------------------------- in 64 bits
def _exact_act(act, g):
    """The activation and its derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if act == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    # x (1 + tanh z) / 2 = x sigmoid(2 z)
    z2 = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(z2)
    return g * s, s + g * s * (1 - s) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize_int8":
        x = state["x"].double()
        scale = x.abs().amax(dim=1).clamp_min(SMALLEST_AMAX) / 127
        amax = scale.new_tensor(SMALLEST_AMAX).maximum(x.abs().amax(dim=1))[:, None]
        # below |x| * 127 / amax, and one more past the middle (on it where that is even)
        low = torch.floor(x.abs() * 127 / amax)
        over = 2 * (127 * x.abs() - low * amax) - amax
        up = (over > 0) | ((over == 0) & (low % 2 == 1))
        return [(torch.sign(x) * (low + up)).to(torch.int8), scale]
    if case["op"] == "gemm_int8":
        c = state["a"].double() @ state["b"].double().t()
        return c * (state["sa"].double()[:, None] * state["sb"].double())
    x, wg, wu = state["x"].double(), state["wg"].double(), state["wu"].double()
    if case["op"] == "gated_linear":
        act, _ = _exact_act(case["act"], x @ wg.t())
        return act * (x @ wu.t())
    act, slope = _exact_act(case["act"], state["gate"].double())
    dh = state["dh"].double()
    dg, du = dh * slope * state["up"].double(), dh * act
    return [dg @ wg + du @ wu, dg.t() @ x, du.t() @ x]
