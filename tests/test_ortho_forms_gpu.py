"""GPU parity of the orthogonalisation in every form of its products, asserted from
the plan: S and B on single CTAs and on CTA pairs, S in slices of K on both, X on
both, for matrices wider and taller, alone and in stacks.  A cap on the grid brings
the pairs, which large matrices take, to small sizes.

Tolerance, relative 2-norm: rounding the result to bf16 gives 1.7e-3, the fp16
roundings of the operands up to 1.7e-3 where all singular values are close and
1.4e-3 elsewhere (simulated in numpy), together 2.4e-3; a quarter more is allowed:
3.1e-3.  In fp16, only where they are not close, the result's own rounding is 2.1e-4:
1.42e-3 and two fifths, 2.0e-3.
"""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding
from operators_ref import T, off, orthogonalized

pytestmark = pytest.mark.gpu

TIMEOUT = 6
SMS = 152
TOLERANCE = {torch.bfloat16: 3.1e-3, torch.float16: 2.0e-3}

# (tile of S, S in slices, tile of B, tile of X): cap, batch, rows, cols, dtype
CASES = [
    ((128, 0, 128, 128), 8, 1, 135, 131, "fp32"), ((128, 0, 128, 256), 6, 2, 135, 131, "fp32"),
    ((128, 1, 128, 128), 16, 1, 909, 131, "bf16"), ((128, 1, 128, 256), 16, 1, 1047, 130, "fp32"),
    ((256, 0, 256, 128), 8, 3, 260, 131, "fp32"), ((256, 0, 256, 256), 8, 3, 141, 132, "bf16"),
    ((256, 1, 128, 128), 8, 1, 1227, 133, "fp32"), ((256, 1, 128, 256), 8, 1, 959, 133, "fp32"),
    ((128, 0, 128, 128), 16, 1, 130, 130, "fp32"), ((128, 0, 128, 256), 6, 2, 138, 144, "fp32"),
    ((128, 1, 128, 128), 16, 1, 131, 932, "bf16"), ((128, 1, 128, 256), 16, 1, 130, 1049, "bf16"),
    ((256, 0, 256, 128), 6, 3, 130, 263, "bf16"), ((256, 0, 256, 256), 6, 3, 130, 142, "fp32"),
    ((256, 1, 128, 128), 8, 1, 131, 1259, "fp32"), ((256, 1, 128, 256), 8, 1, 133, 912, "bf16"),
    # several tiles: mirrored boxes, the last tile row ragged
    ((256, 0, 256, 256), 12, 2, 515, 700, "bf16"), ((256, 0, 256, 256), 12, 2, 700, 515, "fp32"),
    ((256, 0, 256, 256), 4, 1, 777, 1300, "fp16"), ((256, 0, 256, 256), 4, 1, 1300, 777, "bf16"),
    ((256, 0, 256, 256), 12, 1, 600, 9000, "bf16"), ((256, 0, 256, 256), 12, 1, 9000, 600, "fp32"),
    ((256, 0, 256, 256), 12, 2, 390, 9000, "bf16"),
    # on the whole GPU
    ((256, 0, 256, 256), SMS, 16, 512, 1344, "bf16"), ((256, 0, 256, 256), SMS, 1, 3300, 3700, "bf16"),
    ((256, 0, 256, 256), SMS, 1, 3700, 3300, "fp32"), ((256, 1, 128, 256), SMS, 1, 1024, 24000, "bf16"),
    ((256, 1, 128, 256), SMS, 1, 24000, 1024, "bf16"), ((256, 1, 128, 256), SMS, 3, 900, 12000, "fp32"),
    ((128, 1, 128, 256), SMS, 1, 1100, 26000, "bf16"),
]
IDS = ["%d%s-%d-%d-cap%d-%dx%dx%d" % (f[0], "sliced" * f[1], f[2], f[3], *rest[:4]) for f, *rest in CASES]
ON_PAIRS = [c for c in CASES if c[0][0] == 256]
ON_PAIRS_IDS = [i for c, i in zip(CASES, IDS) if c[0][0] == 256]


def form(cap, batch, rows, cols, dtype):
    code = {"bf16": binding.BF16, "fp16": binding.FP16, "fp32": binding.FP32}[dtype]
    s, b, x = binding.select_orthogonalize(SMS, batch, rows, cols, code, step=1, max_ctas=cap)
    return s["tile"], int(s["splits"] > 1), b["tile"], x["tile"]


def matrices(batch, rows, cols, dtype, loud=0.25):
    """A momentum: noise, and a few directions that stand out of it."""
    gen = torch.Generator(device="cuda").manual_seed(rows * 31 + cols)
    u, v = (torch.randn(batch, *s, generator=gen, device="cuda") for s in ((rows, 4), (4, cols)))
    g = 1e-3 * (torch.randn(batch, rows, cols, generator=gen, device="cuda") + loud * u @ v)
    return g.to(T[dtype])


@pytest.fixture(scope="module", autouse=True)
def lib():
    return binding.load_library(build_if_missing=True)


@pytest.mark.parametrize("want,cap,batch,rows,cols,dtype", CASES, ids=IDS)
@pytest.mark.parametrize("loud", [0.25, 0.0])  # without: all singular values close, B close to a multiple of I
def test_forms(want, cap, batch, rows, cols, dtype, loud):
    assert form(cap, batch, rows, cols, dtype) == want
    g = matrices(batch, rows, cols, dtype, loud)
    with binding.Plan(0, max_ctas=cap) as p:
        # a workspace that held NaNs leaves no trace
        torch.full((1 << 24,), float("nan"), device="cuda")
        x = p.orthogonalize(g)
        assert p.status() == 0
        assert off(x, orthogonalized(g)) <= TOLERANCE[x.dtype]
        for _ in range(2):
            assert torch.equal(p.orthogonalize(g), x)


@pytest.mark.parametrize("want,cap,batch,rows,cols,dtype", ON_PAIRS, ids=ON_PAIRS_IDS)
def test_results_of_other_types_and_layouts(want, cap, batch, rows, cols, dtype):
    # fp16; rows off 16-byte boundaries (stored element by element), nothing written between
    assert form(cap, batch, rows, cols, dtype) == want
    g = matrices(batch, rows, cols, dtype)
    exact = orthogonalized(g)
    with binding.Plan(0, max_ctas=cap) as p:
        for out_dtype in (torch.float16, torch.bfloat16):
            hold = torch.full((batch, rows + 2, cols + 7), 9.0, dtype=out_dtype, device="cuda")
            out = hold[:, 1:rows + 1, 3:3 + cols]
            p.orthogonalize(g, out=out)
            assert off(out, exact) <= TOLERANCE[out_dtype]
            apart = torch.full((batch, rows + 1, -(-cols // 8) * 8 + 8), 9.0, dtype=out_dtype, device="cuda")
            p.orthogonalize(g, out=apart[:, :rows, :cols])
            assert torch.equal(apart[:, :rows, :cols], out)
            assert (apart[:, rows] == 9).all() and (apart[:, :, cols:] == 9).all()
            out.fill_(9.0)
            assert (hold == 9).all()
        assert p.status() == 0


@pytest.mark.parametrize("want,cap,batch,rows,cols,dtype", ON_PAIRS[::4], ids=ON_PAIRS_IDS[::4])
def test_a_matrix_of_a_stack_leaves_the_others_alone(want, cap, batch, rows, cols, dtype):
    g = matrices(3, rows, cols, dtype)
    g[0] = 0
    g[2, rows - 1, cols - 1] = float("nan")
    with binding.Plan(0, max_ctas=cap) as p:
        x = p.orthogonalize(g)
        assert (x[0] == 0).all() and torch.isnan(x[2]).all()
        assert off(x[1], orthogonalized(g[1])) <= TOLERANCE[x.dtype]
        assert p.status() == 0


@pytest.mark.parametrize("want,cap,batch,rows,cols,dtype", ON_PAIRS[::3], ids=ON_PAIRS_IDS[::3])
def test_a_timeout_on_pairs_is_reported(want, cap, batch, rows, cols, dtype):
    # the producer of CTA 0 never fills its second stage: the bounded waits run out
    g = matrices(batch, rows, cols, dtype)
    with binding.Plan(0, max_ctas=cap, stall_kblock=1, timeout_ns=20_000_000) as p:
        p.orthogonalize(g, steps=1)
        assert p.status() == TIMEOUT
        assert p.status() == 0


def test_every_combination_is_here():
    assert {(c[0], c[3] > c[4]) for c in CASES} >= {((s, k, b, x), tall) for s, k, b in ((128, 0, 128), (128, 1, 128), (256, 0, 256),
                                                                                      (256, 1, 128)) for x in (128, 256)
                                                    for tall in (False, True)}
