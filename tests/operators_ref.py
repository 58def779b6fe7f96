"""What the operators' GPU tests compare with: random 8-bit operands, and the
formulas in 64 bits on the GPU (torch's double precision)."""
from __future__ import annotations

import torch

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# relative rounding of the result, as unit roundoff
OWN = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def operand(rows, K, square=False, kind="e4m3", seed=0):
    """(values in padded rows, scales, what they stand for in fp64), all on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    v = (4 * torch.randn(rows, K, generator=gen, device="cuda")).to(F8[kind])
    wide = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")
    wide[:, :K] = v.view(torch.uint8)
    s = torch.exp2(10 * torch.rand(-(-K // 128), -(-rows // 128) if square else rows, generator=gen, device="cuda") - 9)
    return wide.view(F8[kind])[:, :K], s, dequantized(v, s)


def dequantized(v, s):
    """The fp64 values that 8-bit values and their scales stand for."""
    rows, K = v.shape
    r = torch.arange(rows, device=v.device) // (1 if s.shape[1] == rows else 128)
    k = torch.arange(K, device=v.device) // 128
    return v.double() * s.double()[k][:, r].t()


def product(a, b, out):
    """The exact product and a bound of each element's error: the 128 products of a block are
    exact in fp32 and summed in fp32 (any order and rounding mode: 128 steps of at most
    2^-23 of the sum of magnitudes), then weighted and added over the K blocks and, where
    K is cut, over its pieces (3 roundings of 2^-24 each), and the result's own rounding."""
    exact = a @ b.t()
    blocks = -(-a.shape[1] // 128)
    bound = (128 + 3 * blocks + 4) * 2.0 ** -23 * (a.abs() @ b.abs().t())
    return exact, bound + OWN[out] * exact.abs() + 2.0 ** -24


def orthogonalized(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    x = g.double()
    wide = x.shape[-2] <= x.shape[-1]
    x = x if wide else x.mT
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    a, b, c = coefficients
    for _ in range(steps):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x if wide else x.mT


def off(got, want):
    """Relative 2-norm of the error, the largest of a stack."""
    d = torch.linalg.vector_norm(got.double() - want, dim=(-2, -1)) / torch.linalg.vector_norm(want, dim=(-2, -1))
    return float(d.max())
