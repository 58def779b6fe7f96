"""GPU tests of the gated layer in every form that a plan takes on a whole GPU, each asserted to be the one
that its size takes there: the kernel for few rows, the weights in the lanes at every width with whole
tiles and tiles in pieces, and CTA pairs."""
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


# (size, kernel, rows of X a tile, whole tiles or tiles in pieces); kernel 0: pairs, 1: the weights in
# the lanes, 2: few rows
FORMS = [((2, 200, 1000), 2, 8, "few"), ((16, 200, 1000), 2, 16, "few"), ((17, 33, 700), 1, 16, "whole"), ((17, 33, 2100), 1, 16, "pieces"),
         ((17, 12000, 300), 1, 32, "whole"), ((520, 65, 9000), 1, 32, "pieces"), ((33, 20000, 300), 1, 64, "whole"),
         ((700, 130, 20000), 1, 64, "pieces"), ((1500, 130, 20000), 1, 128, "pieces"), ((96, 12000, 20000), 1, 128, "both"),
         ((17, 33, 100), 0, 256, "whole"), ((700, 520, 200), 0, 256, "whole")]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu_tanh")])
@pytest.mark.parametrize("size,lanes,width,work", FORMS)
def test_gated_layer_in_every_form(plan, size, lanes, width, work, dtype, act, keep):
    M, N, K = size
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        s = binding.select_gated(152, M, N, K)
        got = "few" if s["lanes"] == 2 else "both" if s["dp_tiles"] and s["sk_tiles"] else "pieces" if s["sk_tiles"] else "whole"
        assert (s["lanes"], s["tile_x"], got) == (lanes, width, work)
    x, wg, wu = ref.layer(M, N, K, T[dtype], M)
    got = plan.gated_linear(x, wg, wu, act, keep=keep)
    want, bound = ref.gated(x, wg, wu, act)
    for t, w, e in zip(got if keep else (got,), want, bound):
        check(t, w, e)
