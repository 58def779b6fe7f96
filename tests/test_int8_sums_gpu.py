"""GPU tests of what the product of 8-bit integers does with its sums: scales at the ends of fp32."""
from __future__ import annotations

import pytest
import torch

import feed_forward_ref as ref
from dense_gemm_blackwell_03_gb300 import binding
from feed_forward_ref import T, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def plan():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library(build_if_missing=True)
    p = binding.Plan(0)
    yield p
    assert p.status() == 0
    p.close()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# few rows (dot products, then matrix instructions); weights in the lanes, whole tiles and
# pieces of every width, pairs; A in the lanes
FORMS = [(1, 200, 300), (2, 200, 300), (7, 200, 300), (16, 200, 300), (24, 200, 300), (40, 130, 9000), (64, 9000, 300), (300, 520, 300),
         (700, 1300, 600), (300, 65, 5000), (3000, 1400, 300), (3000, 260, 300)]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_scales_at_the_ends_of_fp32(plan, M, N, K, out):
    # results in range come out right whatever the scales are, and whichever of them is large
    a, _ = ref.integers(M, K, M)
    b, _ = ref.integers(N, K, N + 1)
    ends = [1e33, -2e36, 2.0 ** 80, 1.5 * 2.0 ** 80, 1.0, 3e-5, 1e-30, 2.0 ** -126, 2e-42, 0.0]
    sa = torch.tensor(ends, device="cuda").repeat(-(-M // len(ends)))[:M]
    sb = torch.tensor(ends[::-1] + [7e-33], device="cuda").repeat(-(-N // 11))[:N]
    got = plan.gemm_int8(a, sa, b, sb, out_dtype=T[out])
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    most = {"bf16": 3.3961775292304e38, "fp16": 65520.0, "fp32": 3.4028235677973366e38}[out]  # from here on infinity
    # the two products and the result are rounded
    bound = 2.01 * 2.0 ** -24 * want.abs() + 2.0 ** -149
    bound = bound + ref.R[T[out]] * (want.abs() + bound) + ref.LEAST[T[out]]
    far = want.abs() >= most * (1 + 2.0 ** -20)
    near = (want.abs() < most * (1 + 2.0 ** -20)) & (want.abs() > most * (1 - 2.0 ** -20))
    assert not near.any() and far.any() and not far.all()
    assert torch.equal(got.isinf() & (got.double().sign() == want.sign()), far)
    assert not got.isnan().any()
    check(torch.where(far, torch.zeros_like(got), got), torch.where(far, torch.zeros_like(want), want), bound)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_rows_of_huge_values_times_weights_of_tiny_ones(plan, M):
    # as quantize_int8 scales them: 8 bits, and nothing lost at fp32's ends
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, 256, generator=gen, device="cuda") * 1e37
    w = torch.randn(520, 256, generator=gen, device="cuda") * 1e-30
    qx, sx = plan.quantize_int8(x)
    qw, sw = plan.quantize_int8(w)
    got = plan.gemm_int8(qx, sx, qw, sw, out_dtype=torch.float32)
    check(got, *ref.product_int8(qx, sx, qw, sw, torch.float32))
