"""GPU tests of the gated layer and the 8-bit integers at the edges of their arguments: refusals,
memory beside the operands, special values, every form of the kernels, streams and graphs, waits
that run out.  Bounds: feed_forward_ref.py."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import feed_forward_ref as ref
from dense_gemm_blackwell_03_gb300 import binding
from feed_forward_ref import T, check

pytestmark = pytest.mark.gpu

INVALID, ALIGN, UNSUP, TIMEOUT, WORKSPACE = 1, 2, 3, 6, 7


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


def gated_case(M, N, K, dtype="bf16", act="silu", seed=0):
    x, wg, wu = ref.layer(M, N, K, T[dtype], seed)
    want, bound = ref.gated(x, wg, wu, act)
    return (x, wg, wu, act), want, bound


def int8_case(M, N, K, out="bf16", seed=0):
    a, sa = ref.integers(M, K, seed)
    b, sb = ref.integers(N, K, seed + 1)
    return (a, sa, b, sb), ref.product_int8(a, sa, b, sb, T[out])


def backward_case(M, N, K, dtype="bf16", act="silu", seed=0):
    x, wg, wu = ref.layer(M, N, K, T[dtype], seed)
    gen = torch.Generator().manual_seed(seed + 5)
    dh, g, u = (ref.padded((f * torch.randn(M, N, generator=gen)).to(T[dtype]).cuda(), 8) for f in (0.3, 1.5, 1.5))
    want, bound = ref.backward(dh, g, u, x, wg, wu, act)
    return (dh, g, u, x, wg, wu, act), want, bound


# --------------------------------------------------- every form, whole and in pieces
# what a plan takes for these sizes on a GPU of 152 SMs is asserted, the results are checked
@pytest.mark.parametrize("M,N,K,form", [
    (2, 200, 1000, (2, 8)), (16, 200, 1000, (2, 16)), (16, 9000, 4096, (1, 16)), (30, 9000, 4096, (1, 32)), (64, 9000, 4096, (1, 64)),
    (700, 520, 200, (1, 128)), (300, 9000, 400, (0, 256))])
@pytest.mark.parametrize("keep", [False, True])
def test_gated_forms(plan, M, N, K, form, keep):
    args, want, bound = gated_case(M, N, K, seed=M)
    s = binding.select_gated(sms(), M, N, K)
    if sms() == 152 and form[0] != 1:
        assert (s["lanes"], s["tile_x"]) == form
    got = plan.gated_linear(*args, keep=keep)
    for t, w, e in zip(got if keep else (got,), want, bound):
        check(t, w, e)


@pytest.mark.parametrize("tile", [16, 32, 64, 128])
@pytest.mark.parametrize("mode", ["gated", "int8"])
def test_every_narrow_tile_whole_and_in_pieces(mode, tile):
    # a cap on the grid brings every width, with whole tiles and with tiles in pieces, to small
    # sizes: the sizes are searched by what the plan says it takes
    select = binding.select_gated if mode == "gated" else binding.select_int8
    found = {}
    for cap in (2, 3, 5, 9, 20, 60, 152):
        for M in (17, 30, 40, 64, 100, 128, 200, 400):
            for N in (64, 200, 333, 600, 1100):
                for K in (100, 1000, 3000, 9000):
                    s = select(sms(), M, N, K, max_ctas=cap)
                    if s["lanes"] == 1 and s["tile_x"] == tile:
                        found.setdefault(s["sk_tiles"] > 0, (cap, M, N, K))
                        if s["sk_tiles"] > 0 and s["dp_tiles"] > 0:
                            found.setdefault("both", (cap, M, N, K))
    assert found, "no size takes this form"
    for cap, M, N, K in found.values():
        with binding.Plan(0, max_ctas=cap) as p:
            if mode == "gated":
                args, want, bound = gated_case(M, N, K, seed=tile)
                for t, w, e in zip(p.gated_linear(*args, keep=True), want, bound):
                    check(t, w, e)
            else:
                args, (want, bound) = int8_case(M, N, K, seed=tile)
                check(p.gemm_int8(*args), want, bound)
            assert p.status() == 0


@pytest.mark.parametrize("M,N,K", [(1000, 1300, 600), (257, 9000, 300), (520, 700, 3000)])
def test_int8_pairs_whole_and_in_pieces(M, N, K):
    for cap in (4, 10, 152):
        s = binding.select_int8(sms(), M, N, K, max_ctas=cap)
        with binding.Plan(0, max_ctas=cap) as p:
            args, (want, bound) = int8_case(M, N, K, "fp32", seed=cap)
            check(p.gemm_int8(*args, out_dtype=torch.float32), want, bound)
            assert p.status() == 0, s


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cap", [0, 4, 152])
@pytest.mark.parametrize("M,N,K", [(700, 33, 300), (300, 65, 5000), (1001, 131, 1001), (3000, 260, 700), (513, 400, 1300),
                                   (3000, 1400, 1100)])
def test_int8_with_more_rows_than_columns(M, N, K, cap, out):
    # A's rows in the lanes: whole tiles and pieces, every width, odd ends
    assert binding.select_int8(sms(), M, N, K, max_ctas=cap)["lanes"] == 3
    (a, sa, b, sb), (want, bound) = int8_case(M, N, K, out, seed=cap)
    hold = torch.full((M + 2, -(-N // 8) * 8 + 24), 7.0, dtype=T[out], device="cuda")
    with binding.Plan(0, max_ctas=cap) as p:
        p.gemm_int8(a, sa, b, sb, out=hold[1:M + 1, 8:8 + N])
        assert p.status() == 0
    check(hold[1:M + 1, 8:8 + N], want, bound)
    hold[1:M + 1, 8:8 + N] = 7
    assert bool((hold == 7).all())


@pytest.mark.parametrize("cap", [1, 2, 7])
def test_few_ctas_give_right_results(cap):
    with binding.Plan(0, max_ctas=cap) as p:
        for M in (3, 40, 300):
            args, want, bound = gated_case(M, 333, 300, seed=cap)
            check(p.gated_linear(*args), want[0], bound[0])
            args, (c, e) = int8_case(M, 333, 300, seed=cap)
            check(p.gemm_int8(*args), c, e)
            args, want, bound = backward_case(M, 333, 300, seed=cap)
            for t, w, e in zip(p.gated_linear_backward(*args), want, bound):
                check(t, w, e)
        assert p.status() == 0


@pytest.mark.parametrize("K", [64, 129, 8192, 20000])
@pytest.mark.parametrize("N", [24, 700, 2500])
@pytest.mark.parametrize("M", [1, 5, 16])
def test_few_rows_with_any_number_of_warps(plan, M, N, K):
    args, want, bound = gated_case(M, N, K, "fp16", "gelu", seed=K)
    check(plan.gated_linear(*args), want[0], bound[0])
    args, (c, e) = int8_case(M, N, K, "fp32", seed=N)
    check(plan.gemm_int8(*args, out_dtype=torch.float32), c, e)


def test_small_workspace():
    with binding.Plan(0, workspace_bytes=(1 << 20) + 4096) as p:
        args, (c, e) = int8_case(40, 300, 9000)
        check(p.gemm_int8(*args), c, e)
        args, want, bound = gated_case(40, 300, 9000)
        check(p.gated_linear(*args), want[0], bound[0])
        args, want, bound = backward_case(40, 3000, 200)
        for t, w, e in zip(p.gated_linear_backward(*args), want, bound):
            check(t, w, e)
        assert p.status() == 0


def test_without_dependent_launch():
    with binding.Plan(0, pdl_off=1) as p:
        for _ in range(3):
            args, (c, e) = int8_case(40, 3000, 1000)
            check(p.gemm_int8(*args), c, e)
            args, want, bound = backward_case(40, 3000, 200)
            for t, w, e in zip(p.gated_linear_backward(*args), want, bound):
                check(t, w, e)


# ------------------------------------------------------------ memory beside the matrices
@pytest.mark.parametrize("M,N,K", [(5, 61, 200), (40, 61, 200), (700, 133, 136), (1300, 1001, 72)])
def test_gated_writes_its_results_and_nothing_else(plan, M, N, K):
    # results in the middle of wider matrices, operands that end with their last value
    args, want, bound = gated_case(M, N, K)
    tight, held = [], []
    for t in args[:3]:
        rows, cols = t.shape
        ld = -(-cols // 8) * 8 + 8
        y = torch.empty((rows - 1) * ld + cols, dtype=t.dtype, device="cuda").as_strided((rows, cols), (ld, 1))
        y.copy_(t)
        tight.append(binding._MATRIX.pack(y.data_ptr(), ld))
        held.append(y)
    hold = [torch.full((M + 2, -(-N // 8) * 8 + 24), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    records = [binding._MATRIX.pack(h[1:, 8:].data_ptr(), h.stride(0)) for h in hold]
    rc = plan.lib.bwgemm_gated(plan.handle, *tight, *records, M, N, K, 0, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for h, w, e in zip(hold, want, bound):
        check(h[1:M + 1, 8:8 + N], w, e)
        h[1:M + 1, 8:8 + N] = 7
        assert bool((h == 7).all())


@pytest.mark.parametrize("M,N,K", [(5, 61, 200), (40, 61, 201), (700, 133, 37), (300, 1001, 1001)])
def test_backward_writes_its_results_and_nothing_else(plan, M, N, K):
    args, want, bound = backward_case(M, N, K)
    records = [binding._MATRIX.pack(t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 1 << 12) for t in args[:6]]
    hold = [torch.full((r + 2, -(-K // 8) * 8 + 24), 7.0, dtype=torch.bfloat16, device="cuda") for r in (M, N, N)]
    records += [binding._MATRIX.pack(h[1:, 8:].data_ptr(), h.stride(0)) for h in hold]
    need = binding._workspace_bytes("bwgemm_gated_backward_workspace", M, N)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    rc = plan.lib.bwgemm_gated_backward(plan.handle, *records, M, N, K, 0, 0, ws.data_ptr(), need,
                                        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and bool((ws[need:] == 77).all())
    for h, w, e in zip(hold, want, bound):
        r = len(h) - 2
        check(h[1:r + 1, 8:8 + K], w, e)
        h[1:r + 1, 8:8 + K] = 7
        assert bool((h == 7).all())


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(5, 61, 200), (40, 61, 201), (700, 133, 37), (300, 1001, 1001)])
def test_int8_writes_its_result_and_nothing_else(plan, M, N, K, out):
    (a, sa, b, sb), (want, bound) = int8_case(M, N, K, out)
    tight = []
    for t in (a, b):
        rows, cols = t.shape
        ld = -(-cols // 16) * 16 + 16
        y = torch.empty((rows - 1) * ld + cols, dtype=torch.int8, device="cuda").as_strided((rows, cols), (ld, 1))
        y.copy_(t)
        tight.append(y)
    hold = torch.full((M + 2, -(-N // 8) * 8 + 24), 7.0, dtype=T[out], device="cuda")
    plan.gemm_int8(tight[0], sa, tight[1], sb, out=hold[1:M + 1, 8:8 + N])
    check(hold[1:M + 1, 8:8 + N], want, bound)
    hold[1:M + 1, 8:8 + N] = 7
    assert bool((hold == 7).all())


# -------------------------------------------------------------- special values
@pytest.mark.parametrize("M", [3, 40, 300])
def test_gated_nan_and_infinity_stay_in_their_rows_and_columns(plan, M):
    (x, wg, wu, act), want, bound = gated_case(M, 250, 200)
    base = plan.gated_linear(x, wg, wu, act)
    x[M - 1, 199] = float("nan")
    wg[249, 0] = float("inf")
    h = plan.gated_linear(x, wg, wu, act)
    assert bool(torch.isnan(h[M - 1]).all())
    assert torch.equal(h[:M - 1, :249], base[:M - 1, :249])
    g = x[:M - 1].double() @ wg.double()[249]  # infinite, of either sign, or NaN
    u = x[:M - 1].double() @ wu.double()[249]
    s = (g * torch.sigmoid(g) * u).to(torch.bfloat16)  # (-inf times 0: NaN)
    assert torch.equal(torch.isnan(h[:M - 1, 249]), torch.isnan(s))
    fine = ~torch.isnan(s)
    assert torch.equal(h[:M - 1, 249][fine], s[fine])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_gated_extreme_projections(plan, act, M):
    # projections from -1e30 to 1e30: activations saturate without a NaN
    e = torch.tensor([-1e30, -1e10, -300.0, -90.0, -87.0, -30.0, -10.0, -1.0, 0.0, 1e-20, 1.0, 10.0, 30.0, 90.0, 1e10, 1e30]).double()
    x = torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    wg = torch.zeros(16, 16, dtype=torch.bfloat16, device="cuda")
    wg[:, 0] = e.to(torch.bfloat16).cuda()
    wu = torch.zeros_like(wg)
    wu[:, 0] = 1
    want, bound = ref.gated(x, wg, wu, act)
    a, _ = ref.act(act, want[1])
    assert bool(torch.isfinite(a).all())
    # below exp's range fp32's logistic function is 0, in 64 bits up to 1e-36 times g
    check(plan.gated_linear(x, wg, wu, act), want[0], bound[0] + 1e-35)
    dh = torch.ones(M, 16, dtype=torch.bfloat16, device="cuda")
    g = wg[:, 0].expand(M, 16).contiguous()
    u = torch.ones_like(g)
    got = plan.gated_linear_backward(dh, g, u, x, wg / 1e30, wu, act)
    want, bound = ref.backward(dh, g, u, x, wg / 1e30, wu, act)
    for t, w, b in zip(got, want, bound):
        assert bool(torch.isfinite(t).all())
        check(t, w, b + 1e-30 * M)


def test_backward_nan_stays_in_its_token_and_weight_row(plan):
    (dh, g, u, x, wg, wu, act), _, _ = backward_case(140, 200, 136)
    base = plan.gated_linear_backward(dh, g, u, x, wg, wu, act)
    g[7, 31] = float("nan")
    dx, dwg, dwu = plan.gated_linear_backward(dh, g, u, x, wg, wu, act)
    rows = torch.arange(140, device="cuda") != 7
    assert bool(torch.isnan(dx[7]).all()) and torch.equal(dx[rows], base[0][rows])
    rows = torch.arange(200, device="cuda") != 31
    for t, b in ((dwg, base[1]), (dwu, base[2])):
        assert bool(torch.isnan(t[31]).all()) and torch.equal(t[rows], b[rows])


@pytest.mark.parametrize("M", [3, 40, 300])
def test_int8_scales_of_any_size(plan, M):
    (a, sa, b, sb), _ = int8_case(M, 70, 200, "fp32")
    sa[0], sa[M - 1], sb[3], sb[5] = 0.0, float("nan"), 1e30, 1e-30
    c = plan.gemm_int8(a, sa, b, sb, out_dtype=torch.float32)
    assert bool(torch.isnan(c[M - 1]).all()) and bool((c[0] == 0).all())
    want, bound = ref.product_int8(a[:M - 1], sa[:M - 1], b, sb, torch.float32)
    check(c[:M - 1], want, bound)


def test_quantised_rows_without_a_finite_largest_value_give_nan(plan):
    x = torch.randn(20, 304, device="cuda").bfloat16()
    w, sw = plan.quantize_int8(torch.randn(40, 304, device="cuda"))
    x[4, 303] = float("inf")
    x[19, 0] = float("nan")
    c = plan.gemm_int8(*plan.quantize_int8(x), w, sw)
    bad = torch.isnan(c).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [4, 19] and not torch.isnan(c[~bad]).any()


# ------------------------------------------------------------------ empty sizes
def test_empty_sizes(plan):
    for M, N, K in ((0, 16, 16), (16, 0, 16), (0, 0, 0)):
        x, wg, wu = (torch.zeros(r, K, dtype=torch.bfloat16, device="cuda") for r in (M, N, N))
        assert plan.gated_linear(x, wg, wu).shape == (M, N)
        a, b = (torch.zeros(r, K, dtype=torch.int8, device="cuda") for r in (M, N))
        assert plan.gemm_int8(a, torch.zeros(M, device="cuda"), b, torch.zeros(N, device="cuda")).shape == (M, N)
    for M in (5, 300):  # empty sums
        x, w = (torch.zeros(r, 0, dtype=torch.bfloat16, device="cuda") for r in (M, 20))
        for t in plan.gated_linear(x, w, w, keep=True):
            assert t.shape == (M, 20) and bool((t == 0).all())
        a, b = (torch.zeros(r, 0, dtype=torch.int8, device="cuda") for r in (M, 20))
        c = plan.gemm_int8(a, torch.full((M,), float("nan"), device="cuda"), b, torch.ones(20, device="cuda"))
        assert c.shape == (M, 20) and bool((c == 0).all())
    z = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dx, dwg, dwu = plan.gated_linear_backward(z(0, 20), z(0, 20), z(0, 20), z(0, 30), z(20, 30), z(20, 30))
    assert dx.shape == (0, 30) and dwg.shape == (20, 30) and bool((dwg == 0).all()) and bool((dwu == 0).all())
    dx, dwg, dwu = plan.gated_linear_backward(z(5, 0), z(5, 0), z(5, 0), z(5, 30), z(0, 30), z(0, 30))
    assert bool((dx == 0).all()) and dx.shape == (5, 30) and dwg.shape == (0, 30)
    dx, dwg, dwu = plan.gated_linear_backward(z(5, 20), z(5, 20), z(5, 20), z(5, 0), z(20, 0), z(20, 0))
    assert dx.shape == (5, 0) and dwg.shape == dwu.shape == (20, 0)
    q, s = plan.quantize_int8(z(0, 20))
    assert q.shape == (0, 20) and s.shape == (0,)


# -------------------------------------------------------- offsets past 32 bits
def test_offsets_past_32_bits(plan):
    # results and operands of more than 2^31 elements; rows from all over are checked
    M, N, K = 270_001, 8200, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, wg, wu = (torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16) for s in ((M, K), (N, K), (N, K)))
    rows = torch.cat([torch.arange(3), torch.randint(0, M, (40,), generator=torch.Generator().manual_seed(2)), torch.arange(M - 3, M)]).cuda()
    h, g, u = plan.gated_linear(x, wg, wu, keep=True)
    want, bound = ref.gated(x[rows], wg, wu, "silu")
    for t, w, e in zip((h, g, u), want, bound):
        check(t[rows], w, e)
    # ... as what is quantised, and as the long side of its product
    q, s = plan.quantize_int8(h)
    want, scale = ref.rows_int8(h[rows])
    assert torch.equal(q[rows], want) and torch.equal(s[rows], scale.float())
    # ... and the gradients of both: dX of these rows, the weights' of the tokens that have any
    dh = torch.zeros_like(h)
    dh[rows] = 0.3
    dx, dwg, dwu = plan.gated_linear_backward(dh, g, u, x, wg, wu)
    want, bound = ref.backward(dh[rows], g[rows], u[rows], x[rows], wg, wu, "silu")
    # (a row that was drawn twice counts once)
    only = torch.unique(rows)
    one, e1 = ref.backward(dh[only], g[only], u[only], x[only], wg, wu, "silu")
    check(dx[rows], want[0], bound[0])
    check(dwg, one[1], e1[1] + M * 2.0 ** -23 * one[1].abs())
    check(dwu, one[2], e1[2] + M * 2.0 ** -23 * one[2].abs())
    del dh, g, u, h, dx
    b, sb = ref.integers(200, N, 5)
    c = plan.gemm_int8(q, s, b, sb)
    check(c[rows], *ref.product_int8(q[rows], s[rows], b, sb, torch.bfloat16))
    few = plan.gemm_int8(b[:4], sb[:4], q, s)  # M = 4 rows against 270001 "weights"
    check(few[:, rows], *ref.product_int8(b[:4], sb[:4], q[rows], s[rows], torch.bfloat16))


# ---------------------------------------------------------------- refusals
def test_gated_refusals(plan):
    t = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    at, host = t.data_ptr(), np.zeros(64).ctypes.data // 16 * 16

    def raw(X=(at, 256), Wg=(at, 256), Wu=(at, 256), H=(at, 64), G=None, U=None, M=8, N=64, K=256, dtype=0, act=0):
        rec = [None if m is None else binding._MATRIX.pack(m[0] or 0, m[1]) for m in (X, Wg, Wu, H, G, U)]
        return plan.lib.bwgemm_gated(plan.handle, *rec, M, N, K, dtype, act, None)
    assert raw(M=0) == raw(N=0) == 0
    for bad in (dict(X=None), dict(Wg=None), dict(Wu=(0, 256)), dict(H=None), dict(G=(at, 64)), dict(U=(at, 64)), dict(M=-1), dict(N=-1),
                dict(K=-1), dict(dtype=2), dict(act=3), dict(act=-1), dict(X=(at, 248)), dict(Wg=(at, 255)), dict(H=(at, 63)),
                dict(G=(at, 64), U=(at, 56)), dict(X=(host, 256)), dict(H=(host, 64)), dict(Wu=(host, 256))):
        assert raw(**bad) == INVALID, bad
    for bad in (dict(X=(at + 2, 256)), dict(Wg=(at + 8, 256)), dict(Wu=(at, 257)), dict(H=(at, 65)), dict(G=(at + 4, 64), U=(at, 64))):
        assert raw(**bad) == ALIGN, bad
    for bad in (dict(M=1 << 31), dict(N=1 << 31, H=(at, 1 << 31)), dict(X=(at, 1 << 41))):
        assert raw(**bad) == UNSUP, bad


def test_backward_refusals(plan):
    t = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    at, host = t.data_ptr(), np.zeros(64).ctypes.data // 16 * 16
    need = binding._workspace_bytes("bwgemm_gated_backward_workspace", 8, 64)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda").data_ptr()
    names = ("dH", "G", "U", "X", "Wg", "Wu", "dX", "dWg", "dWu")

    def raw(M=8, N=64, K=256, dtype=0, act=0, workspace=ws, size=need, **m):
        rec = [m.get(n, (at, 64 if n in ("dH", "G", "U") else 256)) for n in names]
        rec = [None if r is None else binding._MATRIX.pack(r[0] or 0, r[1]) for r in rec]
        return plan.lib.bwgemm_gated_backward(plan.handle, *rec, M, N, K, dtype, act, workspace, size, None)
    assert raw(dX=None, dWg=None, dWu=None) == raw(K=0) == 0  # nothing is wanted
    for bad in (dict(dH=None), dict(G=None), dict(U=(0, 64)), dict(X=None), dict(Wg=None), dict(Wu=None), dict(dWg=None), dict(dWu=None),
                dict(M=-1), dict(N=-1), dict(K=-1), dict(dtype=2), dict(act=3), dict(dH=(at, 63)), dict(dX=(at, 255)), dict(X=(host, 256)),
                dict(dWu=(host, 256)), dict(workspace=host // 256 * 256)):
        assert raw(**bad) == INVALID, bad
    for bad in (dict(dH=(at + 2, 64)), dict(G=(at, 65)), dict(dX=(at + 8, 256)), dict(dWg=(at, 260)), dict(workspace=ws + 128)):
        assert raw(**bad) == ALIGN, bad
    assert raw(size=need - 1) == raw(workspace=None) == WORKSPACE
    assert raw(M=1 << 31) == UNSUP


def test_int8_refusals(plan):
    q = torch.zeros(64, 256, dtype=torch.int8, device="cuda")
    f = torch.zeros(64 * 64, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda").data_ptr()
    at, s, host = q.data_ptr(), f.data_ptr(), np.zeros(64).ctypes.data // 16 * 16
    need = binding._workspace_bytes("bwgemm_run_integer_workspace", 40, 64, 256)

    def raw(A=at, sa=s, B=at, sb=s, C=s, M=40, N=64, K=256, lda=256, ldb=256, ldc=64, out=0, workspace=ws, size=need):
        return plan.lib.bwgemm_run_integer(plan.handle, A, sa, B, sb, C, M, N, K, lda, ldb, ldc, out, workspace, size, None)
    assert raw(M=0) == raw(N=0) == raw(K=0, A=None, B=None, sa=None, sb=None, workspace=None, size=0) == 0
    for bad in (dict(A=None), dict(sa=None), dict(B=None), dict(sb=None), dict(C=None), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=255),
                dict(ldb=255), dict(ldc=63), dict(out=3), dict(A=host), dict(sb=host), dict(C=host), dict(workspace=host // 256 * 256)):
        assert raw(**bad) == INVALID, bad
    for bad in (dict(A=at + 8), dict(B=at + 1), dict(lda=264), dict(ldb=257), dict(C=s + 8), dict(ldc=65), dict(sa=s + 2), dict(sb=s + 1),
                dict(workspace=ws + 128)):
        assert raw(**bad) == ALIGN, bad
    assert raw(size=need - 1) == raw(workspace=None) == WORKSPACE
    assert raw(M=1 << 31) == raw(ldc=1 << 41) == UNSUP
    x = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")

    def rows(X=x.data_ptr(), dtype=0, r=64, c=256, ldx=256, Q=at, ldq=256, S=s):
        return plan.lib.bwgemm_quantize_integer(plan.handle, X, dtype, r, c, ldx, Q, ldq, S, None)
    assert rows() == rows(r=0) == rows(c=0) == 0
    for bad in (dict(X=None), dict(dtype=3), dict(r=-1), dict(c=-1), dict(ldx=255), dict(Q=None), dict(ldq=240), dict(S=None),
                dict(X=host), dict(Q=host), dict(S=host)):
        assert rows(**bad) == INVALID, bad
    for bad in (dict(X=x.data_ptr() + 2), dict(ldx=257), dict(Q=at + 8, r=1), dict(ldq=257, r=1), dict(S=s + 2)):
        assert rows(**bad) == ALIGN, bad
    with pytest.raises(binding.BwgemmError) as e:
        plan.quantize_int8(x[:, 1:])
    assert e.value.status == ALIGN


@pytest.mark.parametrize("make", [lambda: torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda").expand(20, 16),
                                  lambda: torch.zeros(400, dtype=torch.bfloat16, device="cuda").as_strided((20, 16), (8, 1))])
def test_rows_closer_than_their_length_are_refused(plan, make):
    bad, w = make(), torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.BwgemmError) as e:
        plan.gated_linear(bad, w, w)
    assert e.value.status == INVALID
    a, s = torch.zeros(20, 16, dtype=torch.int8, device="cuda"), torch.zeros(20, device="cuda")
    for kw in (dict(A=a[:1].expand(20, 16)), dict(B=a[:1].expand(20, 16)), dict(out=torch.zeros(1, 20, device="cuda").expand(20, 20))):
        with pytest.raises(binding.BwgemmError) as e:
            plan.gemm_int8(kw.get("A", a), s, kw.get("B", a), s, out=kw.get("out"))
        assert e.value.status == INVALID


# ------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("M,N,K", [(100, 520, 1024), (20, 3000, 1024), (700, 2000, 1024)])
def test_timeouts_are_reported(M, N, K):
    g, want, bound = gated_case(M, N, K)
    i, (c, e) = int8_case(M, N, K)
    b, wantb, boundb = backward_case(M, N, K)
    with binding.Plan(0, stall_kblock=1, timeout_ns=20_000_000) as p:
        for call in (lambda: p.gated_linear(*g), lambda: p.gemm_int8(*i), lambda: p.gated_linear_backward(*b)):
            call()
            assert p.status() == TIMEOUT and p.last_device_status() != 0
            assert p.status() == 0
    with binding.Plan(0) as p:
        check(p.gated_linear(*g), want[0], bound[0])
        check(p.gemm_int8(*i), c, e)
        for t, w, x in zip(p.gated_linear_backward(*b), wantb, boundb):
            check(t, w, x)
        assert p.status() == 0


# ------------------------------------------------------- streams, threads, graphs
SIZES = [(3, 700, 1000), (40, 300, 9000), (300, 1000, 700)]


def all_calls(p, M, N, K):
    """A call of everything on operands of its own, and what it gave at first."""
    g, b = gated_case(M, N, K)[0], backward_case(M, N, K)[0]
    i = int8_case(M, N, K)[0]
    x = g[0]

    def run(q=p, **kw):
        return [*q.gated_linear(*g, keep=True, **kw), q.gemm_int8(*i, **kw), *q.gated_linear_backward(*b, **kw), *q.quantize_int8(x, **kw)]
    return run


def test_another_stream_and_a_graph(plan):
    for size in SIZES:
        run = all_calls(plan, *size)
        want = run()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = run(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = run()
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert plan.status() == 0


def test_module_calls_on_two_streams_at_a_time(plan):
    work = [all_calls(plan, *s) for s in SIZES[1:]]
    want = [run() for run in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(15):
        for run, st, w in zip(work, streams, want):
            got.append((run(binding, stream=st), w))
    torch.cuda.synchronize()
    for outputs, w in got:
        assert all(torch.equal(a, b) for a, b in zip(outputs, w))


def test_module_calls_of_two_threads(plan):
    work = [all_calls(plan, *s) for s in SIZES[1:]]
    want = [run() for run in work]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream(), torch.cuda.Stream()]

    def run(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(15):
                got[i].append(work[i](binding))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 15
        for outputs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outputs, want[i]))


def test_the_first_module_call_of_a_stream_inside_a_capture(plan):
    run = all_calls(plan, *SIZES[1])
    want = run()
    torch.cuda.synchronize()
    fresh = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh):
        got = run(binding)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_of_one_plan_in_turns(plan):
    # one after the other on a stream, as launches of their plan: tiles in pieces use its workspace
    work = [all_calls(plan, *s) for s in SIZES[1:]]
    want = [run() for run in work]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, got = [], []
    for run in work:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            got.append(run())
    for outputs in got:
        for t in outputs:
            t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    for outputs, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs, w))
    assert plan.status() == 0


@pytest.mark.parametrize("M", [5, 40, 200])
def test_one_tensor_in_two_places(plan, M):
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear
    x, w, other = ref.layer(M, 136, 200, torch.bfloat16, M)
    apart = [t.clone().requires_grad_() for t in (x, w, w)]
    dh = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(M, 136)  # a sum's gradient: one element
    want = torch.autograd.grad(gated_linear(*apart), apart, dh)
    x.requires_grad_()
    w.requires_grad_()
    dx, dw = torch.autograd.grad(gated_linear(x, w, w), (x, w), dh)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1] + want[2])
    q, s = plan.quantize_int8(x.detach())
    check(plan.gemm_int8(q, s, q, s), *ref.product_int8(q, s, q, s, torch.bfloat16))


@pytest.mark.parametrize("op", ["gated", "int8", "backward", "rows"])
def test_weights_written_just_before_on_the_stream(plan, op):
    # kernels that start early read nothing that the kernel before them still writes
    M, N, K = 40, 6000, 2048
    (x, wg, wu, act), _, _ = gated_case(M, 2000, K)
    a, sa = plan.quantize_int8(x)
    rest = torch.randn(N, K, device="cuda")
    for i in range(5):
        w = (rest * (i + 1)).bfloat16()
        if op == "rows":
            q, s = plan.quantize_int8(w)
            want, scale = ref.rows_int8(w)
            assert torch.equal(q, want) and torch.equal(s, scale.float())
        elif op == "int8":
            q, s = plan.quantize_int8(w)
            c = plan.gemm_int8(a, sa, q, s)
            check(c, *ref.product_int8(a, sa, q, s, torch.bfloat16))
        elif op == "gated":
            want, bound = ref.gated(x, w[:2000], w[2000:4000], act)
            for t, v, e in zip(plan.gated_linear(x, w[:2000], w[2000:4000], act, keep=True), want, bound):
                check(t, v, e)
        else:
            h, g, u = plan.gated_linear(x, w[:2000], w[2000:4000], act, keep=True)
            want, bound = ref.backward(h, g, u, x, w[:2000], w[2000:4000], act)
            for t, v, e in zip(plan.gated_linear_backward(h, g, u, x, w[:2000], w[2000:4000], act), want, bound):
                check(t, v, e)


@pytest.mark.parametrize("M,N,K", [(6000, 40, 2048), (4000, 600, 1024)])
def test_tokens_written_just_before_in_the_lanes(plan, M, N, K):
    # A's bytes are copied before the kernel that widens B has ended
    assert binding.select_int8(sms(), M, N, K)["lanes"] == 3
    b, sb = plan.quantize_int8(torch.randn(N, K, device="cuda"))
    rest = torch.randn(M, K, device="cuda")
    held = [plan.quantize_int8(rest * (i + 1)) for i in range(2)]
    want = [plan.gemm_int8(q, s, b, sb) for q, s in held]
    torch.cuda.synchronize()
    got, flush = [], torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    a, sa = (torch.empty_like(t) for t in held[0])
    for i in range(8):
        x = rest * (i % 2 + 1)
        flush.add_(1)
        q, s = plan.quantize_int8(x)
        got.append(plan.gemm_int8(q, s, b, sb))
        a.copy_(held[i % 2][0])  # by a kernel that knows nothing of an early start
        sa.copy_(held[i % 2][1])
        got.append(plan.gemm_int8(a, sa, b, sb))
    torch.cuda.synchronize()
    for i, c in enumerate(got):
        assert torch.equal(c, want[i // 2 % 2])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("tokens", [1, 5, 70, 600])
def test_a_feed_forward_block_served(plan, tokens):
    # the gated layer in 16 bits, its result's rows to integers, the down projection on them
    inner, hidden = 264, 1000
    x, wg, wu = ref.layer(tokens, hidden, inner, torch.bfloat16, tokens)
    down, sd = plan.quantize_int8(torch.randn(inner, hidden, generator=torch.Generator().manual_seed(9)).cuda())
    h = plan.gated_linear(x, wg, wu)
    want, bound = ref.gated(x, wg, wu, "silu")
    check(h, want[0], bound[0])
    q, s = plan.quantize_int8(h)
    rows, scale = ref.rows_int8(h)
    assert torch.equal(q, rows)
    check(plan.gemm_int8(q, s, down, sd), *ref.product_int8(q, s, down, sd, torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,inner,hidden", [(70, 136, 200), (300, 61, 77)])
def test_gated_gradients_by_autograd(plan, dtype, act, tokens, inner, hidden):
    # against the formula's: the forward pass rounds G and U for the backward pass, which moves
    # dG and dU by the slopes' change, |act''| <= 1.2, over half a step of G
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear
    x, wg, wu = (t.clone().requires_grad_() for t in ref.layer(tokens, hidden, inner, T[dtype], tokens))
    v = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).to(T[dtype]).cuda()
    gated_linear(x, wg, wu, act).backward(v)
    r = ref.R[T[dtype]]
    with torch.no_grad():
        (h, g, u), (eh, eg, eu) = ref.gated(x, wg, wu, act)
        gr, ur = g.to(T[dtype]), u.to(T[dtype])
        want, bound = ref.backward(v, gr, ur, x, wg, wu, act)
        # what the rounded G and U that the kernels kept may differ by from these: their bounds
        a, slope = ref.act(act, g)
        dg = v.double().abs() * (eu * 1.13 + 1.2 * eg * (u.abs() + eu))
        du = v.double().abs() * 1.13 * eg
        dg, du = 2 * dg, 2 * du
        more = [dg @ wg.double().abs() + du @ wu.double().abs(), dg.t() @ x.double().abs(), du.t() @ x.double().abs()]
    for t, w, e, m in zip((x, wg, wu), want, bound, more):
        check(t.grad, w, e + (1 + r) * m)


def test_gated_gradients_against_differences(plan):
    # fp16 steps that are exact in x; the loss's difference against the gradient times the step
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear
    M, N, K = 24, 40, 48
    x, wg, wu = (t.double() for t in ref.layer(M, N, K, torch.float16, 3))
    v = torch.randn(M, N, generator=torch.Generator().manual_seed(4), dtype=torch.float64).cuda()
    leaves = [t.half().requires_grad_() for t in (x, wg, wu)]
    (gated_linear(*leaves).double() * v).sum().backward()

    def loss(x, wg, wu):
        a, _ = ref.act("silu", x @ wg.t())
        return float((a * (x @ wu.t()) * v).sum())
    for i in range(3):
        step = torch.randn(leaves[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64).cuda()
        eps = 1e-6
        ends = [[t + (s * eps * step if j == i else 0) for j, t in enumerate((x, wg, wu))] for s in (1, -1)]
        difference = (loss(*ends[0]) - loss(*ends[1])) / (2 * eps)
        got = float((leaves[i].grad.double() * step).sum())
        # dH, G, U, dG (dU) and the gradient are rounded to fp16, 2^-11 each, slopes 1.13: 8 such
        # roundings of every element's share, and differences good to 1e-6
        assert abs(got - difference) <= 8 * 2.0 ** -11 * float((leaves[i].grad.double().abs() * step.abs()).sum()) + 1e-5 * abs(difference)


@pytest.mark.parametrize("warm", [False, True])
def test_a_gated_training_step_inside_a_capture(plan, warm):
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear, scaled_linear
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, wg, wu, wd = (torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
                     for s in ((48, 264), (3000, 264), (3000, 264), (264, 3000)))

    def step():  # (detached: a graph that lives on keeps its leaves on the stream of its forward pass)
        y = scaled_linear(gated_linear(x, wg, wu), wd)
        return [t.detach() for t in (y, *torch.autograd.grad(y.float().square().sum(), (x, wg, wu, wd)))]

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


def test_training_with_a_gated_layer_runs(plan):
    from dense_gemm_blackwell_03_gb300 import linear_training
    losses = linear_training.train(tokens=64, inner=40, hidden=72, outer=24, steps=3, gated=True)
    assert len(losses) == 3 and all(np.isfinite(v) for v in losses)
