"""What the tests of the gated feed-forward layer and of the 8-bit integers compare with: the
formulas in 64 bits, with a bound of each element's error.

Bounds, from the arithmetic (r = half a step of the type, relative: bf16 2^-8, fp16 2^-11,
fp32 2^-24; results below fp16's normal numbers are off by 2^-25 at most):

* a sum of K products that are exact in fp32, in any order and rounding mode: K steps of at
  most 2^-23 of the sum of magnitudes.
* activation and slope: exp is off by 2 + 1.2 |t| ulp, |t| < 88 before it over- or
  underflows, so each factor by 2^-16.2 of it at most, the few operations around it by
  2^-21: EVAL = 2^-16 of the terms' magnitudes, which an activation's value and 2 |g| + 1 of a
  slope bound.  Slopes of all three lie within 1.13.
* dG and dU are rounded to the type before the products.
"""
from __future__ import annotations

import math

import torch

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
R = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
STEP = 2.0 ** -23
EVAL = 2.0 ** -16


def act(name, g):
    """(activation, its slope) of float64 g."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        cdf = torch.special.erfc(-g / math.sqrt(2)) / 2  # (torch's ndtr is 0 below -8.3)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(8 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * c * (1 + 0.134145 * g * g)


def padded(t, multiple, extra=0, fill=float("nan")):
    """t's values in rows `multiple` elements (and `extra` times that) apart, the rest filled."""
    rows, cols = t.shape
    wide = torch.full((rows, -(-cols // multiple) * multiple + extra * multiple), fill, dtype=torch.float32, device=t.device)
    wide[:, :cols] = t
    return wide.to(t.dtype)[:, :cols]


def layer(M, N, K, dtype=torch.bfloat16, seed=0, device="cuda", spread=1.5):
    """x, w_gate, w_up with projections of the given spread, rows padded with NaN."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=gen).to(dtype)
    w = [(spread / math.sqrt(max(K, 1)) * torch.randn(N, K, generator=gen)).to(dtype) for _ in range(2)]
    return [padded(t.to(device), 8) for t in (x, *w)]


def gated(x, wg, wu, name):
    """((h, g, u) in float64, their error bounds)."""
    dtype, K = x.dtype, x.shape[1]
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = K * STEP * (x.abs() @ wg.abs().t()), K * STEP * (x.abs() @ wu.abs().t())
    a, _ = act(name, g)
    h = a * u
    eh = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + EVAL * h.abs()
    r, least = R[dtype], LEAST[dtype]
    return (h, g, u), [e + r * (v.abs() + e) + least for v, e in ((h, eh), (g, eg), (u, eu))]


def backward(dh, g, u, x, wg, wu, name):
    """((dx, dwg, dwu) in float64, their error bounds)."""
    dtype = dh.dtype
    r, least = R[dtype], LEAST[dtype]
    dh, g, u, x, wg, wu = (t.double() for t in (dh, g, u, x, wg, wu))
    a, slope = act(name, g)
    dg, du = dh * u * slope, dh * a
    edg = (dh * u).abs() * (EVAL * (2 * g.abs().clamp(max=60) + 1)) + r * dg.abs() * 1.01 + least
    edu = (EVAL + 1.01 * r) * du.abs() + least
    M, N = dh.shape

    def total(terms):
        exact = sum(p @ q for p, _, q in terms)
        n = sum(p.shape[1] for p, _, _ in terms)
        off = sum(e @ q.abs() + n * STEP * ((p.abs() + e) @ q.abs()) for p, e, q in terms)
        return exact, off + r * (exact.abs() + off) + least

    out = [total([(dg, edg, wg), (du, edu, wu)]), total([(dg.t(), edg.t(), x)]), total([(du.t(), edu.t(), x)])]
    return [v for v, _ in out], [e for _, e in out]


def rows_int8(x):
    """(q, scales in float64) of a finite matrix: the quotient against the middle of two
    integers, both sides exact in 64 bits."""
    x = x.double()
    a = x.abs().amax(dim=1, keepdim=True).clamp_min(2.0 ** -100)
    low = torch.floor(x.abs() * 127 / a)
    over = 254 * x.abs() - (2 * low + 1) * a
    q = low + ((over > 0) | ((over == 0) & (low % 2 == 1)))
    return (torch.sign(x) * q).to(torch.int8), a[:, 0] / 127


def integers(rows, K, seed, device="cuda", low=-128):
    """(int8 values in rows padded with ones, fp32 scales)."""
    gen = torch.Generator().manual_seed(seed)
    q = torch.randint(low, 128, (rows, K), generator=gen, dtype=torch.int8)
    wide = torch.ones(rows, -(-K // 16) * 16, dtype=torch.int8)
    wide[:, :K] = q
    s = torch.exp2(8 * torch.rand(rows, generator=gen) - 10)
    return wide.to(device)[:, :K], s.to(device)


def product_int8(a, sa, b, sb, dtype):
    """(C in float64, its error bound): the sum exact up to 2^24, two products of 2^-24 each."""
    K = a.shape[1]
    a, b = a.double(), b.double()
    scale = sa.double()[:, None] * sb.double()
    exact = (a @ b.t()) * scale
    mags = a.abs() @ b.abs().t()
    off = torch.where(mags <= 2.0 ** 24, 0.0, K * STEP * mags) * scale + 3 * 2.0 ** -24 * exact.abs()
    return exact, off + R[dtype] * (exact.abs() + off) + LEAST[dtype]


def check(got, want, bound):
    assert got.shape == want.shape
    off = (got.double() - want).abs() - bound
    if got.dtype == torch.float16:
        # from 65520 on, the middle of the largest value 65504 and 2^16, fp16 rounds to infinity
        infinite = got.isinf() & (got.double().sign() == want.sign()) & (want.abs() + bound >= 65520)
        off = torch.where(infinite, torch.zeros_like(off), off)
    assert bool((off <= 0).all()), f"{int((~(off <= 0)).sum())} of {off.numel()} values past their bound, worst by {float(off.max()):.3g}"
