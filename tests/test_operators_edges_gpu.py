"""GPU tests of the operators at the edges of their arguments: layouts that are
refused, and forms that only some sizes take.  Plain forms in 64 bits."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding

pytestmark = pytest.mark.gpu

INVALID = 1


@pytest.fixture(scope="module")
def plan():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library(build_if_missing=True)
    p = binding.Plan(0)
    yield p
    assert p.status() == 0
    p.close()


# ------------------------------------------------------------ orthogonalise
@pytest.mark.parametrize("shape", [(64, 128), (3, 64, 128)])
def test_orthogonalize_refuses_rows_closer_than_their_length(plan, shape):
    dense = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    room = torch.ones(3 * 64 * 128, dtype=torch.bfloat16, device="cuda")
    expanded = torch.ones(shape[:-2] + (1, 128), dtype=torch.bfloat16, device="cuda").expand(shape)
    overlapping = room.as_strided(shape, (64 * 128, 120, 1)[-len(shape):])
    for bad in (expanded, overlapping):
        for kw in (dict(G=bad), dict(G=dense, out=bad)):
            with pytest.raises(binding.BwgemmError) as e:
                plan.orthogonalize(**kw)
            assert e.value.status == INVALID
    assert (room == 1).all() and (expanded == 1).all()


# ------------------------------------------------------------ scaled product
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [256, 0])
def test_scaled_product_refuses_a_strided_row_as_result(plan, dtype, K):
    a, sa = plan.quantize(torch.ones(1, 256, device="cuda"))
    b, sb = plan.quantize(torch.ones(32, 256, device="cuda"))
    operands = (a[:, :K], sa[:K // 128], b[:, :K], sb[:K // 128])
    held = torch.full((32, 8), 5.0, dtype=dtype, device="cuda")
    wide = torch.full((1, 64), 5.0, dtype=dtype, device="cuda")
    for out in (held[:, :1].t(), wide[:, ::2]):
        with pytest.raises(ValueError, match="unit stride"):
            plan.gemm_scaled(*operands, out=out)
    assert (held == 5).all() and (wide == 5).all()
    plan.gemm_scaled(*operands, out=wide[:, 32:])  # in place: 32 elements and nothing else
    assert (wide[:, :32] == 5).all() and torch.equal(wide[:, 32:], plan.gemm_scaled(*operands, out_dtype=dtype))


# ----------------------------------------------------------- a linear layer
@pytest.mark.parametrize("outer", [136, 61])
@pytest.mark.parametrize("loss", [lambda y, v: (y.sum(0) * v).sum(), lambda y, v: y.sum(), lambda y, v: (y.t() @ y).sum()])
def test_linear_gradients_of_expanded_and_transposed_gradients(plan, outer, loss):
    # the same bits as for the same gradient laid out densely
    from dense_gemm_blackwell_03_gb300.linear_training import scaled_linear
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, w, v = (torch.randn(*s, generator=gen, device="cuda") for s in ((96, 200), (outer, 200), (outer,)))
    x.requires_grad_()
    w.requires_grad_()
    y = scaled_linear(x, w)
    at = y.detach().requires_grad_()
    dy, = torch.autograd.grad(loss(at, v), at)
    want = torch.autograd.grad(y, (x, w), dy.clone(memory_format=torch.contiguous_format), retain_graph=True)
    got = torch.autograd.grad(loss(y, v), (x, w))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
