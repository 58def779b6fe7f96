"""GPU tests of the gated layer's activations where their values are tiny, but not nothing: a large U or
gradient brings them back among the results."""
from __future__ import annotations

import math

import pytest
import torch

import feed_forward_ref as ref
from dense_gemm_blackwell_03_gb300 import binding
from feed_forward_ref import check

pytestmark = pytest.mark.gpu

# of an activation's value or slope, relative: exp is off by 2 + 1.2 |t| ulp, 2^-16.2 at |t| = 88 and
# 2^-15.9 at 104, gelu_tanh's t by four roundings, 4 * 2^-24 * 104 = 2^-15.3; the rest is below 2^-21
EVAL = 2.0 ** -14
LEAST = 2.0 ** -149  # of fp32: values below its normal numbers are multiples of it
POINTS = {"silu": torch.arange(-103.5, -70.0, 0.5), "gelu_tanh": -torch.arange(8.0, 10.75, 0.0625),
          "gelu": -torch.arange(8.0, 13.0, 0.125)}


@pytest.fixture(scope="module")
def plan():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library(build_if_missing=True)
    p = binding.Plan(0)
    yield p
    assert p.status() == 0
    p.close()


def tail(act, g):
    """(activation, slope, bound of either's error) of far negative g, in 64 bits."""
    a, slope = ref.act(act, g)
    if act == "gelu":  # (1 - erfc would lose the slope's terms one against the other)
        cdf = torch.special.erfc(-g / math.sqrt(2)) / 2
        s = cdf.abs() + (g * torch.exp(-g * g / 2)).abs()  # magnitudes of the slope's terms
        c = g.abs()
    else:
        t = g if act == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
        c = g.abs() if act == "silu" else (g * math.sqrt(8 / math.pi) * (1 + 0.134145 * g * g)).abs()
        s = torch.exp(t) * (1 + c)
    # the factor that may be subnormal is off by a step, and weighed with g or c
    return a, slope, EVAL * a.abs() + 2 * LEAST * (1 + g.abs()), EVAL * s + 2 * LEAST * (1 + c)


@pytest.mark.parametrize("act", sorted(POINTS))
@pytest.mark.parametrize("M", [1, 40, 300])
def test_small_activations_times_a_large_factor(plan, act, M):
    g = POINTS[act].bfloat16().cuda()
    N = len(g)
    x = torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    wg, wu = (torch.zeros(N, 16, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wg[:, 0] = g
    wu[:, 0] = 2.0 ** 120
    h = plan.gated_linear(x, wg, wu, act)
    a, _, ea, _ = tail(act, g.double())
    want = (a * 2.0 ** 120).expand(M, N)
    bound = ea * 2.0 ** 120
    check(h, want, (bound + 2.0 ** -8 * (want.abs() + bound)).expand(M, N))
    # most of them far above what their bound allows to be missing
    assert int((want[0].abs() > 100 * bound).sum()) > N // 2


@pytest.mark.parametrize("act", sorted(POINTS))
@pytest.mark.parametrize("M", [1, 200])
def test_small_slopes_times_a_large_gradient(plan, act, M):
    g = POINTS[act].bfloat16().cuda()
    N = len(g)
    gate = torch.zeros(M, -(-N // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :N]
    gate[:] = g
    up = torch.ones(M, -(-N // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :N]
    dh = torch.zeros(M, -(-N // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :N]
    dh[0] = 2.0 ** 120  # one token's, so that the sums over tokens have one term
    x = torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 1
    _, dwg, dwu = plan.gated_linear_backward(dh, gate, up, x, None, None, act, input_grad=False)
    a, slope, ea, es = tail(act, g.double())
    for got, v, e in ((dwg, slope, es), (dwu, a, ea)):
        want, bound = v * 2.0 ** 120, e * 2.0 ** 120
        # dG and dU are rounded, the result is not rounded again: it is one of them
        check(got[:, 3], want, bound + 2.0 ** -8 * (want.abs() + bound))
        assert not got[:, :3].any() and not got[:, 4:].any()
        assert int((want.abs() > 100 * bound).sum()) > N // 2


@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("act", sorted(POINTS))
def test_a_gradient_and_a_factor_whose_product_passes_fp32(plan, act, swap):
    # dH U is 2^150, the slope brings dH U act'(G) back
    points = {"silu": torch.arange(-100.0, -30.0, 0.5), "gelu_tanh": -torch.arange(6.0, 10.0, 0.0625), "gelu": -torch.arange(7.0, 13.0, 0.125)}
    g = points[act].bfloat16().cuda()
    N = len(g)
    g = torch.cat([g, torch.full((-N % 8,), -300.0, dtype=torch.bfloat16, device="cuda")])[None]
    dh, up = torch.full_like(g, 2.0 ** (50 if swap else 100)), torch.full_like(g, 2.0 ** (100 if swap else 50))
    x = torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 1
    _, dwg, _ = plan.gated_linear_backward(dh, g, up, x, None, None, act, input_grad=False)
    _, slope, _, es = tail(act, g[0].double())
    want, bound = slope * 2.0 ** 150, es * 2.0 ** 150
    bound = bound + 2.0 ** -8 * (want.abs() + bound)
    far = want.abs() - bound >= 3.3961775292304e38
    assert int(far.sum()) < N // 2 and bool(dwg[:, 3][far].isinf().all())
    near = ~far & (want.abs() + bound >= 3.38e38)
    fine = ~far & ~near
    check(dwg[:, 3][fine], want[fine], bound[fine])
    assert not dwg[:, 3].isnan().any() and not dwg[N:].any()
