"""Products whose last tiles are cut into pieces of K: every worker that a tile's sums are taken from
has computed one (a worker without a step of K leaves in its place what an earlier call put there)."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
from dense_gemm_blackwell_03_gb300 import binding

# one tile more than workers, and a K of about as many blocks as there are workers
SIZES = [(cap, 128 * (cap + 1), 128 * kb) for cap in (118, 130, 152) for kb in range(cap - 14, cap + 2)]


def blocks(n):
    return -(-n // 128)


@pytest.fixture(scope="module", autouse=True)
def lib():
    return binding.load_library(build_if_missing=True)


@pytest.mark.parametrize("M", [9, 16, 24, 100])
def test_every_worker_of_a_scaled_product_has_a_step(M):
    for cap, N, K in SIZES:
        for kind in ("row", "square"):
            c = binding.select_scaled(152, M, N, K, kind, max_ctas=cap)
            assert c["sk_tiles"] == 0 or c["workers"] <= c["sk_tiles"] * blocks(K), (cap, M, N, K)


@pytest.mark.parametrize("select,rows", [(binding.select_gated, 64), (binding.select_int8, 128), (binding.select_int8, 256)])
def test_every_worker_of_a_product_with_the_weights_in_the_lanes_has_a_step(select, rows):
    # (with joins as dear as they are no plan comes near to it)
    for cap in (2, 5, 20, 80, 152):
        for more in {1, 2, cap // 2, cap - 1} - {0, cap}:
            for M in (17, 64, 200):
                for kb in range(1, cap // more + 2):
                    c = select(152, M, rows * (cap + more), 128 * kb, max_ctas=cap)
                    assert c["sk_tiles"] == 0 or c["workers"] <= c["sk_tiles"] * kb, (cap, more, M, kb)


@pytest.mark.gpu
@pytest.mark.parametrize("blocks_k", [-3, -1, 0])
def test_a_scaled_product_takes_nothing_from_an_earlier_call(blocks_k):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    M, N, K = 9, 128 * (sms + 1), 128 * (sms + blocks_k)
    gen = torch.Generator(device="cuda").manual_seed(sms)

    def operand(rows, cols):
        return torch.randn(rows, cols, generator=gen, device="cuda").bfloat16()
    with binding.Plan(0) as p:
        # all workers leave a piece that is NaN in the plan's workspace
        wide = 128 * 4 * sms
        c = binding.select_scaled(sms, M, 512, wide)
        assert c["workers"] == sms and c["sk_tiles"] > 0 == c["dp_tiles"] and c["tile_c"] == 16
        a, w = p.quantize(operand(M, wide)), p.quantize(operand(512, wide), blocks="square")
        a[1].fill_(float("nan"))
        assert bool(torch.isnan(p.gemm_scaled(*a, *w)).all())
        a, w = p.quantize(operand(M, K)), p.quantize(operand(N, K), blocks="square")
        got = p.gemm_scaled(*a, *w, out_dtype=torch.float32)
        assert p.status() == 0
    want, bound = ref.product(ref.dequantized(*a), ref.dequantized(*w), "fp32")
    assert bool(((got.double() - want).abs() <= bound).all())
