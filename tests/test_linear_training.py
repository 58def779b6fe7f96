"""The 8-bit linear layer's Python side on the CPU: plain forms stand in for the
two operators, so that what is asked of them, and what autograd does, is seen."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import linear_training


class Plain:
    """quantize and gemm_scaled without rounding: values pass through, scales are ones."""

    def __init__(self):
        self.quantized = []

    def quantize(self, x, blocks="row", transposed=False):
        per = 16 // x.element_size()
        rows, cols = x.shape
        assert cols <= 1 or x.stride(1) == 1
        assert rows <= 1 or (x.stride(0) >= cols and x.stride(0) % per == 0), "the library refuses this row stride"
        assert x.data_ptr() % 16 == 0
        self.quantized.append((blocks, transposed))
        out = (x.clone(), None)
        return out + (x.t().clone(), None) if transposed else out

    def gemm_scaled(self, a, scale_a, b, scale_b, out_dtype):
        return (a.double() @ b.double().t()).to(out_dtype)


@pytest.fixture
def plain(monkeypatch):
    p = Plain()
    monkeypatch.setattr(linear_training, "binding", p)
    return p


def leaves(tokens, inner, outer):
    gen = torch.Generator().manual_seed(tokens)
    return [torch.randn(*s, generator=gen, dtype=torch.float64).float().requires_grad_()
            for s in ((tokens, inner), (outer, inner))]


# what autograd hands to the backward pass: expanded by a sum over rows, over columns,
# over both, transposed, a slice of something wider, one row
@pytest.mark.parametrize("loss", [lambda y: (y.sum(0) * torch.arange(y.shape[1])).sum(), lambda y: y.sum(1).square().sum(),
                                  lambda y: y.sum(), lambda y: (y.t() @ torch.ones(y.shape[0], 3)).square().sum(),
                                  lambda y: torch.cat([y, y], 1)[:, 1:].square().sum(), lambda y: y.square().sum()])
@pytest.mark.parametrize("tokens,inner,outer", [(12, 16, 24), (7, 9, 13), (1, 16, 5), (6, 8, 1)])
def test_gradients_of_any_layout(plain, loss, tokens, inner, outer):
    x, w = leaves(tokens, inner, outer)
    loss(linear_training.scaled_linear(x, w)).backward()
    xr, wr = (t.detach().double().requires_grad_() for t in (x, w))
    torch.set_default_dtype(torch.float64)
    try:
        loss(xr @ wr.t()).backward()
    finally:
        torch.set_default_dtype(torch.float32)
    for got, want in ((x.grad, xr.grad), (w.grad, wr.grad)):
        assert (got - want).abs().max() <= 1e-5 * want.abs().max() + 1e-30


@pytest.mark.parametrize("make", [lambda: torch.ones(1, 8).expand(4, 8), lambda: torch.ones(20).as_strided((4, 8), (4, 1)),
                                  lambda: torch.ones(1, 1).expand(4, 8), lambda: torch.ones(8, 4).t(),
                                  lambda: torch.ones(4, 9)[:, 1:], lambda: torch.ones(4, 12)[:, 4:]])
def test_rows_are_copied_unless_the_quantiser_reads_them(make):
    t = make()
    got = linear_training._aligned_rows(t)
    assert torch.equal(got, t) and got.stride(1) == 1 and got.stride(0) >= 8 and got.stride(0) % 4 == 0
    assert got.data_ptr() % 16 == 0
    dense = torch.ones(4, 8)
    assert linear_training._aligned_rows(dense) is dense


def test_a_second_derivative_raises(plain):
    # the backward pass is computed in 8 bits outside the graph: a gradient penalty
    # through it would silently lose its terms
    x, w = leaves(12, 16, 24)
    y = linear_training.scaled_linear(x, w)
    gx, = torch.autograd.grad((y ** 3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        gx.square().sum().backward()


# ------------------------------------- each direction is quantised only where it is read
@pytest.mark.parametrize("of_x,of_w", [(True, True), (True, False), (False, True), (False, False)])
def test_only_the_directions_that_gradients_read(plain, of_x, of_w):
    x, w = leaves(12, 16, 24)
    x.requires_grad_(of_x)
    w.requires_grad_(of_w)
    y = linear_training.scaled_linear(x, w)
    # the weight's gradient reads x's columns, x's gradient the weight's
    assert plain.quantized == [("row", of_w), ("square", of_x)]
    if of_x or of_w:
        plain.quantized.clear()
        y.sum().backward()
        assert plain.quantized == [("row", of_w)]
        for t, want in ((x, of_x), (w, of_w)):
            assert (t.grad is not None) == want


def test_no_direction_for_gradients_without_a_graph(plain):
    x, w = leaves(12, 16, 24)
    with torch.no_grad():
        y = linear_training.scaled_linear(x, w)
    assert not y.requires_grad and plain.quantized == [("row", False), ("square", False)]


def test_a_gradient_of_one_operand_alone(plain):
    x, w = leaves(12, 16, 24)
    both = torch.autograd.grad(linear_training.scaled_linear(x, w).square().sum(), (x, w))
    for i, t in enumerate((x, w)):
        for of in (True, False):
            (w if t is x else x).requires_grad_(of)
            got, = torch.autograd.grad(linear_training.scaled_linear(x, w).square().sum(), t)
            assert torch.equal(got, both[i])
            (w if t is x else x).requires_grad_(True)


def test_weights_without_a_gradient_stay(plain):
    plain.orthogonalize = lambda g, steps, scale: scale * g
    a, b = torch.ones(4, 8, requires_grad=True), torch.ones(4, 8, requires_grad=True)
    opt = linear_training.OrthogonalMomentum([a, b], lr=0.5, beta=0.0)
    a.sum().backward()
    opt.step()
    assert (a == 0.5).all() and (b == 1).all() and a.grad is None and (opt.momentum[1] == 0).all()
