"""GPU parity of the scaled product in every compiled form and division of the
work, each asserted from the plan: tiles in order of 256 and 128 columns with a
scale per column or per 128, swapped tiles of 64, 32 and 16 rows; whole tiles,
tiles cut along K, and both in one launch.  A cap of five CTAs brings the large
forms to small sizes; some sizes run on the whole GPU as well.  The bound of an
element's error is derived in operators_ref.product."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding
from operators_ref import F8, T, operand, product

pytestmark = pytest.mark.gpu

TIMEOUT = 6
CAP = 5
SMS = 152

# (columns per tile, swapped, scale per column, division): M, N, K, blocks of B; rows of C
# on 16-byte boundaries and off them
CAPPED = [
    ((256, 0, 0, "whole"), 473, 432, 662, "square"), ((256, 0, 0, "whole"), 193, 945, 625, "square"),
    ((256, 0, 0, "mixed"), 463, 392, 3706, "square"), ((256, 0, 0, "mixed"), 500, 387, 3487, "square"),
    ((256, 0, 0, "cut"), 322, 192, 4403, "square"), ((256, 0, 0, "cut"), 338, 171, 4484, "square"),
    ((256, 0, 1, "whole"), 521, 400, 618, "row"), ((256, 0, 1, "whole"), 1015, 133, 690, "row"),
    ((256, 0, 1, "mixed"), 492, 448, 3524, "row"), ((256, 0, 1, "mixed"), 474, 426, 3657, "row"),
    ((256, 0, 1, "cut"), 323, 152, 4822, "row"), ((256, 0, 1, "cut"), 370, 130, 4758, "row"),
    ((128, 0, 0, "whole"), 335, 272, 639, "square"), ((128, 0, 0, "whole"), 324, 265, 632, "square"),
    ((128, 0, 0, "mixed"), 963, 32, 5125, "square"), ((128, 0, 0, "mixed"), 234, 265, 7435, "square"),
    ((128, 0, 0, "cut"), 322, 24, 6143, "square"), ((128, 0, 0, "cut"), 327, 19, 6075, "square"),
    ((128, 0, 1, "whole"), 973, 24, 613, "row"), ((128, 0, 1, "whole"), 338, 261, 645, "row"),
    ((128, 0, 1, "mixed"), 213, 328, 7500, "row"), ((128, 0, 1, "mixed"), 195, 334, 7321, "row"),
    ((128, 0, 1, "cut"), 329, 24, 6046, "row"), ((128, 0, 1, "cut"), 97, 266, 5001, "row"),
    ((64, 1, 1, "whole"), 267, 152, 610, "row"), ((64, 1, 1, "whole"), 261, 130, 632, "row"),
    ((64, 1, 1, "mixed"), 174, 168, 6146, "row"), ((64, 1, 1, "mixed"), 176, 187, 5535, "row"),
    ((32, 1, 1, "whole"), 129, 144, 620, "square"), ((32, 1, 1, "whole"), 145, 138, 616, "row"),
]
FULL = [
    ((256, 0, 0, "whole"), 7348, 389, 200, "square"), ((256, 0, 0, "mixed"), 4181, 1669, 2862, "square"),
    ((256, 0, 0, "cut"), 775, 2969, 3985, "square"), ((256, 0, 1, "whole"), 7431, 394, 200, "row"),
    ((256, 0, 1, "mixed"), 5844, 1221, 3126, "row"), ((256, 0, 1, "cut"), 1606, 1498, 4158, "row"),
    ((128, 0, 0, "whole"), 4913, 179, 200, "square"), ((128, 0, 0, "mixed"), 3550, 779, 7853, "square"),
    ((128, 0, 0, "cut"), 1652, 700, 4541, "square"), ((128, 0, 1, "whole"), 5024, 184, 200, "row"),
    ((128, 0, 1, "mixed"), 4643, 1094, 5159, "row"), ((128, 0, 1, "cut"), 1929, 522, 4816, "row"),
    ((64, 1, 1, "whole"), 4987, 16, 200, "square"), ((64, 1, 1, "mixed"), 950, 1491, 5497, "row"),
    ((64, 1, 1, "cut"), 360, 270, 11296, "square"), ((32, 1, 1, "whole"), 17, 48, 200, "row"),
    ((32, 1, 1, "mixed"), 17, 20554, 13101, "square"), ((32, 1, 1, "cut"), 247, 140, 7294, "row"),
    ((16, 1, 1, "whole"), 9, 18939, 553, "row"), ((16, 1, 1, "mixed"), 3, 20898, 8871, "square"),
    ((16, 1, 1, "cut"), 17, 17, 6886, "square"),
]
IN_ORDER = [c for c in CAPPED if not c[0][1]]


def form(M, N, K, blocks, **opts):
    c = binding.select_scaled(SMS, M, N, K, blocks, **opts)
    assert not c["few_rows"]
    division = "whole" if not c["sk_tiles"] else "mixed" if c["dp_tiles"] else "cut"
    return c["tile_c"], c["swap_ab"], c["column_scales"], division


@pytest.fixture(scope="module")
def capped():
    binding.load_library(build_if_missing=True)
    with binding.Plan(0, max_ctas=CAP) as p:
        yield p
        assert p.status() == 0


@pytest.fixture(scope="module")
def full():
    binding.load_library(build_if_missing=True)
    with binding.Plan(0, max_ctas=SMS) as p:
        yield p
        assert p.status() == 0


def check(plan, M, N, K, blocks, out, a_square=False, kinds=("e4m3", "e4m3")):
    a, sa, av = operand(M, K, a_square, kinds[0], seed=M)
    b, sb, bv = operand(N, K, blocks == "square", kinds[1], seed=N)
    exact, bound = product(av, bv, out)
    c = plan.gemm_scaled(a, sa, b, sb, out_dtype=T[out])
    assert plan.status() == 0
    assert ((c.double() - exact).abs() <= bound).all()
    for _ in range(2):
        assert torch.equal(plan.gemm_scaled(a, sa, b, sb, out_dtype=T[out]), c)


def ids(cases):
    return ["%d%s%s-%s-%dx%dx%d" % (f[0], "s" * f[1], "c" * f[2], f[3], *rest[:3]) for f, *rest in cases]


@pytest.mark.parametrize("want,M,N,K,blocks", CAPPED, ids=ids(CAPPED))
@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
def test_capped(capped, want, M, N, K, blocks, out):
    assert form(M, N, K, blocks, max_ctas=CAP) == want
    check(capped, M, N, K, blocks, out)


@pytest.mark.parametrize("want,M,N,K,blocks", FULL, ids=ids(FULL))
def test_full(full, want, M, N, K, blocks):
    assert form(M, N, K, blocks, max_ctas=SMS) == want
    check(full, M, N, K, blocks, "fp32")
    check(full, M, N, K, blocks, "bf16")


@pytest.mark.parametrize("want,M,N,K,blocks", IN_ORDER[::3], ids=ids(IN_ORDER[::3]))
@pytest.mark.parametrize("a_square", [False, True])
@pytest.mark.parametrize("kinds", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_types_in_order(capped, want, M, N, K, blocks, a_square, kinds):
    assert form(M, N, K, blocks, max_ctas=CAP) == want
    check(capped, M, N, K, blocks, "fp32", a_square, kinds)


@pytest.mark.parametrize("want,M,N,K,blocks", CAPPED, ids=ids(CAPPED))
def test_adding_to_a_result(capped, want, M, N, K, blocks):
    # i products added to 3; the padding and the rows around stay
    a, sa, av = operand(M, K, seed=M)
    b, sb, bv = operand(N, K, blocks == "square", seed=N)
    exact, bound = product(av, bv, "fp32")
    wide = torch.full((M + 2, -(-N // 4) * 4 + 8), 3.0, device="cuda")
    out = wide[1:M + 1, :N]
    for i in range(1, 4):
        capped.gemm_scaled(a, sa, b, sb, out=out, accumulate=True)
        # i products, and i additions of one rounding each
        assert ((out.double() - 3 - i * exact).abs() <= i * bound + i * 2.0 ** -23 * (3 + i * exact.abs())).all()
    assert (wide[0] == 3).all() and (wide[M + 1] == 3).all() and (wide[:, N:] == 3).all()
    half = torch.full((M + 2, -(-N // 8) * 8 + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    capped.gemm_scaled(a, sa, b, sb, out=half[1:M + 1, :N])
    assert (half[0] == 3).all() and (half[M + 1] == 3).all() and (half[:, N:] == 3).all()
    assert torch.equal(half[1:M + 1, :N], capped.gemm_scaled(a, sa, b, sb))


@pytest.mark.parametrize("want,M,N,K,blocks", CAPPED[::2], ids=ids(CAPPED[::2]))
def test_nans_infinities_and_zeros_stay_where_they_are(capped, want, M, N, K, blocks):
    # a NaN in A, a row of scales of zero, an infinite scale of B
    a, sa, av = operand(M, K, seed=M)
    b, sb, bv = operand(N, K, blocks == "square", seed=N)
    sa[:, 3] = 0
    a.view(torch.uint8)[9, 200] = 0x7F  # of either type a NaN
    sb[1, 0] = float("inf")
    av[3] = 0
    c = capped.gemm_scaled(a, sa, b, sb, out_dtype=torch.float32)
    touched = min(N, 128) if blocks == "square" else 1  # columns of the infinite scale
    assert torch.isnan(c[9]).all() and not torch.isfinite(c[:, :touched]).any()
    rows = torch.tensor([i for i in range(M) if i != 9], device="cuda")
    exact, bound = product(av[rows], bv[touched:], "fp32")
    got = c[rows][:, touched:]
    assert ((got.double() - exact).abs() <= bound).all() and (c[3, touched:] == 0).all()


@pytest.mark.parametrize("M,N,K,blocks", [(300, 128, 20000, "square"), (48, 300, 9000, "row"), (463, 392, 3706, "square")])
def test_without_room_for_partial_tiles(M, N, K, blocks):
    # cut along K with the default workspace (the last one on five CTAs), whole without
    cap = CAP if M == 463 else SMS
    small = (1 << 20) + 4096
    assert form(M, N, K, blocks, max_ctas=cap)[3] != "whole"
    assert form(M, N, K, blocks, max_ctas=cap, workspace_bytes=small)[3] == "whole"
    for room in (0, small):
        with binding.Plan(0, max_ctas=cap, workspace_bytes=room) as p:
            check(p, M, N, K, blocks, "fp32")


@pytest.mark.parametrize("want,M,N,K,blocks", IN_ORDER[::2], ids=ids(IN_ORDER[::2]))
def test_a_timeout_in_order_is_reported(want, M, N, K, blocks):
    # the producer of CTA 0 never fills its second stage: the bounded waits run out
    a, sa, _ = operand(M, K, seed=M)
    b, sb, _ = operand(N, K, blocks == "square", seed=N)
    with binding.Plan(0, max_ctas=CAP, stall_kblock=1, timeout_ns=20_000_000) as p:
        p.gemm_scaled(a, sa, b, sb)
        assert p.status() == TIMEOUT and p.last_device_status() != 0
        assert p.status() == 0


def test_the_formats_used_here():
    assert set(F8) == {"e4m3", "e5m2"} and {f[0] for f in CAPPED + FULL} == {
        (n, s, c, d) for n, s, c in ((256, 0, 0), (256, 0, 1), (128, 0, 0), (128, 0, 1), (64, 1, 1), (32, 1, 1), (16, 1, 1))
        for d in ("whole", "mixed", "cut")}
