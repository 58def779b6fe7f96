"""GPU tests of what the product of 8-bit integers does with its sums: scales at the ends of fp32, sums that
are exact in every form, and sums past 2^24."""
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


# ------------------------------------------------------------------------ sums
# every form that a plan takes on 152 SMs: (size, kernel, rows of X a tile, whole tiles or tiles in
# pieces); kernel 1: the weights in the lanes, 2: few rows, 3: A in the lanes
DEEP = [
    ((1, 512, 30000), 2, 8, "few"), ((2, 700, 20000), 2, 8, "few"), ((5, 2500, 20001), 2, 8, "few"), ((16, 690, 28671), 2, 16, "few"),
    ((8, 24, 131071), 2, 8, "few"), ((17, 33, 100), 1, 16, "whole"), ((17, 33, 5000), 1, 16, "pieces"), ((24, 512, 60001), 1, 16, "pieces"),
    ((17, 12000, 100), 1, 32, "whole"), ((17, 200, 9000), 1, 32, "pieces"), ((17, 20000, 9000), 1, 32, "both"),
    ((200, 3000, 2100), 1, 64, "whole"), ((100, 3000, 9000), 1, 64, "pieces"), ((33, 20000, 9000), 1, 64, "both"),
    ((200, 9000, 700), 1, 128, "whole"), ((100, 4096, 9000), 1, 128, "pieces"), ((520, 9000, 2100), 1, 128, "both"),
    ((1500, 3000, 300), 1, 256, "whole"), ((160, 12000, 9000), 1, 256, "pieces"), ((160, 28672, 5000), 1, 256, "both"),
    ((40, 33, 100), 3, 16, "whole"), ((40, 33, 5000), 3, 16, "pieces"), ((1500, 200, 100), 3, 32, "whole"), ((64, 33, 28700), 3, 32, "pieces"),
    ((3000, 200, 2100), 3, 64, "whole"), ((3000, 130, 9000), 3, 64, "pieces"), ((3000, 700, 700), 3, 128, "whole"),
    ((3000, 65, 20000), 3, 128, "pieces"), ((3000, 1000, 5000), 3, 128, "both"), ((3000, 1000, 700), 3, 256, "whole"),
    ((3000, 1000, 9000), 3, 256, "pieces"), ((3000, 2048, 5000), 3, 256, "both")]


def check_form(M, N, K, lanes, width, work):
    if sms() != 152:
        return
    s = binding.select_int8(152, M, N, K)
    got = "few" if s["lanes"] == 2 else "both" if s["dp_tiles"] and s["sk_tiles"] else "pieces" if s["sk_tiles"] else "whole"
    assert (s["lanes"], s["tile_x"], got) == (lanes, width, work)


def draw(rows, K, low, high, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.full((rows, -(-K // 16) * 16), 99, dtype=torch.int8, device="cuda")
    wide[:, :K] = torch.randint(low, high, (rows, K), generator=gen, device="cuda", dtype=torch.int8)
    return wide[:, :K]


@pytest.mark.parametrize("size,lanes,width,work", DEEP)
def test_sums_up_to_2_24_are_exact(plan, size, lanes, width, work):
    # no sum of any part of the products passes 2^24 (16 * 16 * 60001, 8 * 8 * 131071), scales are powers of two: a
    # result is the exact value, rounded once to its type
    M, N, K = size
    check_form(M, N, K, lanes, width, work)
    most = 16 if K < 65536 else 8
    a, b = draw(M, K, -most, most + 1, M), draw(N, K, -most, most + 1, N + 1)
    sa, sb = (torch.exp2((torch.arange(n, device="cuda") % 9 - 4).float()) for n in (M, N))
    exact = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
    assert float(exact.abs().max()) > 0
    assert torch.equal(plan.gemm_int8(a, sa, b, sb, out_dtype=torch.float32).double(), exact)
    assert torch.equal(plan.gemm_int8(a, sa, b, sb), exact.bfloat16())


@pytest.mark.parametrize("low", [0, 127, -128])
@pytest.mark.parametrize("size,lanes,width,work", [d for d in DEEP if d[0][2] >= 2100])
def test_sums_past_2_24(plan, size, lanes, width, work, low):
    # operands of one sign.  Few rows: 32-bit integers, rounded once.  Elsewhere the tensor cores' fp32
    # sums, cut toward zero: never too large but by the pieces' roundings, too small by K 2^-24 at most
    M, N, K = size
    check_form(M, N, K, lanes, width, work)
    a, b = (draw(n, K, low, low + 1 if low else 128, n) for n in (M, N))
    ones = [torch.ones(n, device="cuda") for n in (M, N)]
    got = plan.gemm_int8(a, ones[0], b, ones[1], out_dtype=torch.float32)
    exact = a.double() @ b.double().t()
    if lanes == 2:
        assert torch.equal(got, exact.float())
        return
    off = got.double() - exact
    pieces = 2 * 152 * 2.0 ** -24  # a tile's pieces: at most as many as there are CTAs, each added and rounded
    assert bool((off <= pieces * exact).all()) and bool((off >= -(K * 2.0 ** -24 + pieces) * exact).all())
    if float(exact.max()) <= 2.0 ** 24:
        assert not off.any()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("M,N,K", [(64, 9000, 16384), (200, 300, 65536), (512, 512, 65537), (3000, 200, 16384)])
def test_small_products_after_a_large_sum(plan, M, N, K, sign):
    # what is added to a sum past 2^24 loses its last bits
    a = torch.full((M, -(-K // 16) * 16), 127, dtype=torch.int8, device="cuda")[:, :K]
    b = torch.full((N, -(-K // 16) * 16), 127, dtype=torch.int8, device="cuda")[:, :K]
    a[:, K // 2:] = 3 * sign
    b[:, K // 2:] = 5
    ones = [torch.ones(n, device="cuda") for n in (M, N)]
    got = plan.gemm_int8(a, ones[0], b, ones[1], out_dtype=torch.float32).double()
    exact = a.double() @ b.double().t()
    mags = a.double().abs() @ b.double().abs().t()
    assert bool(((got - exact).abs() <= (K + 304) * 2.0 ** -24 * mags).all())
