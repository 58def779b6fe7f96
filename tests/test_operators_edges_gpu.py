"""GPU tests of the operators at the edges of their arguments: layouts that are
refused, and forms that only some sizes take.  Plain forms in 64 bits."""
from __future__ import annotations

import threading

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding
from operators_ref import T, off, operand, orthogonalized, product

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


@pytest.mark.parametrize("shape", [(140, 200), (3, 64, 64), (2000, 16)])
@pytest.mark.parametrize("eps", [0.0, 1e-7])
def test_orthogonalize_zeros_give_zeros_with_any_eps(plan, shape, eps):
    g = torch.zeros(shape, device="cuda")
    assert (plan.orthogonalize(g, eps=eps) == 0).all()
    g.view(-1)[5] = float("nan")
    x = plan.orthogonalize(g, eps=eps)
    assert torch.isnan(x[0] if x.dim() == 3 else x).all() and (x.dim() == 2 or (x[1:] == 0).all())


# Tolerance: as in test_ortho_forms_gpu, 3.1e-3; where X stays small, the only operation
# is X <- a X.
TINY = 3.1e-3


@pytest.mark.parametrize("power", [-7, -8, -9, -10, -11, -12, -13, -15, -17])
@pytest.mark.parametrize("shape,dtype", [((300, 1000), "fp32"), ((64, 4096), "bf16"), ((700, 90), "fp32"), ((1, 40), "bf16")])
def test_orthogonalize_matrices_far_below_eps(plan, power, shape, dtype):
    # |G| = 10^power, eps = 1e-7: the result is small too, and right to the same relative error
    g = torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.float64)
    g = (g / g.norm() * 10.0 ** power).to(T[dtype])
    assert off(plan.orthogonalize(g), orthogonalized(g)) <= TINY


@pytest.mark.parametrize("table", [[(3.4445, -4.775, 2.0315)], [(0.3, -0.1, 0.2), (5.0, -4.0, 1.0)], [(2.0, -1.5, 0.5)] * 12,
                                   [(-2.5, 1.0, 0.0), (0.01, 1.0, 1.0), (60.0, 0.0, 0.0)]])
def test_orthogonalize_small_matrices_with_other_coefficients(plan, table):
    g = torch.randn(3, 150, 260, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=torch.float64)
    g = g / g.norm(dim=(1, 2), keepdim=True) * torch.tensor([1e-3, 1e-9, 1e-12], device="cuda")[:, None, None]
    g = g.float()
    want = g.double() / (g.double().norm(dim=(1, 2), keepdim=True) + 1e-5)
    for a, b, c in table:
        s = want @ want.mT
        want = a * want + (b * s + c * (s @ s)) @ want
    x = plan.orthogonalize(g, steps=len(table), coefficients=table, eps=1e-5, scale=0.5)
    assert off(x, 0.5 * want) <= TINY


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


# -------------------------------------------------- a cap on the persistent grids
@pytest.mark.parametrize("cap", [1, 2, 7])
def test_few_ctas_give_the_same_results(cap):
    a, sa, av = operand(300, 900, seed=cap)
    b, sb, bv = operand(200, 900, square=True, seed=cap + 1)
    g = torch.randn(3, 200, 700, device="cuda").to(torch.bfloat16)
    with binding.Plan(0, max_ctas=cap) as p:
        exact, bound = product(av, bv, "fp32")
        assert ((p.gemm_scaled(a, sa, b, sb, out_dtype=T["fp32"]) - exact).abs() <= bound).all()
        assert off(p.orthogonalize(g), orthogonalized(g)) <= 4.1e-3
        assert p.status() == 0


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


# -------------------------------------------------------------- default plans
def split_product(seed):
    """Operands whose product's tiles are cut along K (partial sums in the plan's workspace),
    a matrix whose orthogonalisation is, and what a plan of their own gives for both."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a, b = (torch.randn(n, 9000, generator=gen, device="cuda").to(torch.bfloat16) for n in (48, 300))
    g = torch.randn(200, 9000, generator=gen, device="cuda").to(torch.bfloat16)
    with binding.Plan(0) as p:
        operands = p.quantize(a) + p.quantize(b, blocks="square")
        want = (p.gemm_scaled(*operands, out_dtype=torch.float32), p.orthogonalize(g), p.gemm(a[:, :8000], b[:296, :8000]))
        assert p.status() == 0
    torch.cuda.synchronize()
    return operands, g, (a[:, :8000], b[:296, :8000]), want


def test_module_calls_on_two_streams_at_a_time(plan):
    work = [split_product(s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(40):
        for (operands, g, ab, want), st in zip(work, streams):
            got.append((binding.gemm_scaled(*operands, out_dtype=torch.float32, stream=st), binding.orthogonalize(g, stream=st),
                        want))
    torch.cuda.synchronize()
    for c, x, want in got:
        assert torch.equal(c, want[0]) and torch.equal(x, want[1])


def test_module_calls_of_two_threads(plan):
    work = [split_product(s) for s in (3, 4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]

    def run(i):
        operands, g, ab, want = work[i]
        with torch.cuda.stream(streams[i]):
            for _ in range(40):
                got[i].append((binding.gemm_scaled(*operands, out_dtype=torch.float32), binding.orthogonalize(g),
                               binding.gemm(*ab)))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 40
        for outputs in got[i]:
            assert all(torch.equal(o, w) for o, w in zip(outputs, work[i][3]))


def test_the_first_module_call_of_a_stream_inside_a_capture(plan):
    operands, g, ab, want = split_product(5)
    binding.gemm_scaled(*operands)  # the library's kernels are loaded
    fresh = torch.cuda.Stream()
    assert (0, threading.get_ident(), fresh.cuda_stream) not in binding._plans
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh):
        got = (binding.gemm_scaled(*operands, out_dtype=torch.float32), binding.orthogonalize(g), binding.gemm(*ab))
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(got, want))


@pytest.mark.parametrize("warm", [False, True])
def test_a_training_step_of_a_linear_layer_inside_a_capture(plan, warm):
    # forward here, backward on autograd's thread: both make their plans while this thread captures
    from dense_gemm_blackwell_03_gb300.linear_training import scaled_linear
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_() for s in ((48, 9000), (300, 9000)))

    def step():  # (detached: a graph that lives on keeps its leaves on the stream of its forward pass)
        y = scaled_linear(x, w)
        return [t.detach() for t in (y, *torch.autograd.grad(y.float().square().sum(), (x, w)))]

    stream = torch.cuda.Stream()
    want = step()
    torch.cuda.synchronize()
    if warm:
        with torch.cuda.stream(stream):
            step()
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
