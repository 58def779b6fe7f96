"""GPU tests of the gated feed-forward layer, its gradients, and the 8-bit integers, against the
formulas in 64 bits (bounds: feed_forward_ref.py)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import feed_forward_ref as ref
from dense_gemm_blackwell_03_gb300 import binding
from feed_forward_ref import T, check

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
INVALID, ALIGN, UNSUP, WORKSPACE = 1, 2, 3, 7


@pytest.fixture(scope="module")
def plan():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library(build_if_missing=True)
    p = binding.Plan(0)
    yield p
    assert p.status() == 0
    p.close()


def check_gated(plan, M, N, K, dtype="bf16", act="silu", seed=0, keep=True):
    x, wg, wu = ref.layer(M, N, K, T[dtype], seed)
    got = plan.gated_linear(x, wg, wu, act, keep=keep)
    got = got if keep else (got,)
    assert plan.status() == 0
    want, bound = ref.gated(x, wg, wu, act)
    for t, w, e in zip(got, want, bound):
        assert t.dtype == T[dtype]
        check(t, w, e)
    if keep:
        assert torch.equal(plan.gated_linear(x, wg, wu, act), got[0])
    return x, wg, wu, got


# ------------------------------------------------------------------ 8-bit rows
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (3, 7), (5, 129), (130, 520), (4, 1024), (2, 1025), (9, 4100),
                                       (3, 16385), (2, 40000), (1030, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_to_int8(plan, rows, cols, dtype):
    gen = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=gen) * torch.exp2(torch.randint(-9, 5, (1, cols), generator=gen).float())
    x = ref.padded(x.to(T[dtype]).cuda(), 8)
    q, s = plan.quantize_int8(x)
    want, scale = ref.rows_int8(x)
    assert q.dtype == torch.int8 and torch.equal(q, want)
    assert torch.equal(s, scale.float())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_to_int8_between_two_integers(plan, dtype):
    # values on, next to and around every middle, for largest values that make the quotient a
    # tie exactly, nearly, and not at all
    rows = []
    for top in (127.0, 254.0, 1.0, 100.0, 3.140625, 65504.0, 0.0078125):
        top = float(torch.tensor(top).to(T[dtype]))
        mid = (torch.arange(-127, 127) + 0.5).double() * top / 127
        near = mid.to(T[dtype])
        up = torch.nextafter(near, torch.full_like(near, float("inf")))
        down = torch.nextafter(near, torch.full_like(near, -float("inf")))
        rows.append(torch.cat([near, up, down, torch.tensor([top, -top]).to(T[dtype])]).clamp(-top, top))
    x = ref.padded(torch.stack(rows).cuda(), 8)
    q, s = plan.quantize_int8(x)
    want, scale = ref.rows_int8(x)
    assert torch.equal(q, want) and torch.equal(s, scale.float())


@pytest.mark.parametrize("dtype,bits", [("bf16", 8), ("fp16", 11)])
def test_rows_to_int8_every_quotient(plan, dtype, bits):
    # every significand against every other as the row's largest, down to quotients below 1/2
    # (fp16: each 7th row, which meets all remainders)
    sig = torch.arange(2 ** (bits - 1), 2 ** bits, device="cuda").double()
    tops = sig if bits == 8 else sig[::7]
    x = torch.cat([sig * 2.0 ** -j for j in range(1, 10)] + [-sig * 2.0 ** -1])
    rows = torch.cat([tops[:, None], x.expand(len(tops), -1)], 1).to(T[dtype])
    wide = ref.padded(rows, 8)
    q, s = plan.quantize_int8(wide)
    want, scale = ref.rows_int8(wide)
    assert torch.equal(q, want) and torch.equal(s, scale.float())


def test_rows_to_int8_special_rows(plan):
    x = torch.randn(8, 3000, device="cuda")
    x[1] = 0
    x[2] *= 2.0 ** -120       # below the smallest scale
    x[3, 2999] = float("nan")
    x[4, 0] = float("inf")
    x[5] = 1e-45              # subnormal
    x[6, 5] = torch.finfo(torch.float32).max
    q, s = plan.quantize_int8(x)
    fine = [0, 1, 2, 5, 6, 7]
    want, scale = ref.rows_int8(x[fine])
    assert torch.equal(q[fine], want) and torch.equal(s[fine], scale.float())
    assert bool(torch.isnan(s[3:5]).all()) and not q[3:5].any()


def test_rows_to_int8_write_nothing_else(plan):
    x = ref.padded(torch.randn(67, 333, device="cuda").bfloat16(), 8, extra=2)
    q = torch.full((69, 352), 77, dtype=torch.int8, device="cuda")
    s = torch.full((70,), -1.0, device="cuda")
    rc = plan.lib.bwgemm_quantize_integer(plan.handle, x.data_ptr(), 0, 67, 333, x.stride(0), q.data_ptr(), 352, s.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want, scale = ref.rows_int8(x)
    assert torch.equal(q[:67, :333], want) and torch.equal(s[:67], scale.float())
    assert bool((q[67:] == 77).all()) and bool((q[:, 333:] == 77).all()) and bool((s[67:] == -1).all())


# -------------------------------------------------------------- 8-bit product
def check_int8(plan, M, N, K, out="bf16", seed=0):
    a, sa = ref.integers(M, K, seed)
    b, sb = ref.integers(N, K, seed + 1)
    c = plan.gemm_int8(a, sa, b, sb, out_dtype=T[out])
    assert plan.status() == 0 and c.dtype == T[out]
    check(c, *ref.product_int8(a, sa, b, sb, T[out]))
    return a, sa, b, sb, c


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 640])
@pytest.mark.parametrize("N,K", [(520, 640), (1000, 264)])
def test_int8_rows(plan, M, N, K):
    check_int8(plan, M, N, K, seed=M)


@pytest.mark.parametrize("K", [1, 15, 16, 127, 128, 129, 255, 384, 1024, 5005])
@pytest.mark.parametrize("M", [3, 48, 300])
def test_int8_depths(plan, M, K):
    check_int8(plan, M, 264, K, "fp32", seed=K)


@pytest.mark.parametrize("N", [1, 7, 8, 63, 129, 250, 1000, 3001])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M", [5, 260])
def test_int8_columns_and_outputs(plan, N, out, M):
    check_int8(plan, M, N, 512, out, seed=N)


@pytest.mark.parametrize("M,N,K", [(2000, 3000, 768), (4096, 300, 2048), (130, 9000, 1024), (64, 20000, 384), (1, 512, 30000),
                                   (300, 128, 20000), (700, 5000, 640)])
def test_int8_many_tiles(plan, M, N, K):
    a, sa, b, sb, c = check_int8(plan, M, N, K, seed=M + N)
    assert torch.equal(plan.gemm_int8(a, sa, b, sb), c)  # the same bits again


@pytest.mark.parametrize("M", [1, 40, 500])
def test_int8_sums_are_exact(plan, M):
    # the largest values: 1024 products of 2^14 are 2^24
    K = 1024
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((160, K), -128, dtype=torch.int8, device="cuda")
    b[1::2] = 127
    b[2, 7] = -127
    ones = [torch.ones(n, device="cuda") for n in (M, 160)]
    c = plan.gemm_int8(a, ones[0], b, ones[1], out_dtype=torch.float32)
    assert torch.equal(c.double(), a.double() @ b.double().t())


# ------------------------------------------------------------- gated, forward
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 257, 640])
@pytest.mark.parametrize("N,K", [(520, 640), (1000, 264)])
def test_gated_rows(plan, M, N, K):
    check_gated(plan, M, N, K, seed=M)


@pytest.mark.parametrize("K", [1, 7, 8, 63, 64, 65, 127, 128, 129, 200, 1152])
@pytest.mark.parametrize("M", [3, 48, 1500])
def test_gated_depths(plan, M, K):
    check_gated(plan, M, 264, K, seed=K)


@pytest.mark.parametrize("N", [1, 7, 8, 63, 65, 129, 250, 1001, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [5, 70, 1300])
def test_gated_columns_and_types(plan, N, dtype, M):
    check_gated(plan, M, N, 192, dtype, ACTS[N % 3], seed=N)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [4, 1024])
def test_gated_activations(plan, act, M):
    check_gated(plan, M, 520, 320, "fp16", act)
    check_gated(plan, M, 520, 320, "bf16", act, keep=False)


# ------------------------------------------------------------ gated, backward
def check_backward(plan, M, N, K, dtype="bf16", act="silu", seed=0):
    x, wg, wu = ref.layer(M, N, K, T[dtype], seed)
    gen = torch.Generator().manual_seed(seed + 5)
    dh, g, u = (ref.padded((f * torch.randn(M, N, generator=gen)).to(T[dtype]).cuda(), 8) for f in (0.3, 1.5, 1.5))
    got = plan.gated_linear_backward(dh, g, u, x, wg, wu, act)
    assert plan.status() == 0
    want, bound = ref.backward(dh, g, u, x, wg, wu, act)
    for t, w, e in zip(got, want, bound):
        assert t.dtype == T[dtype]
        check(t, w, e)
    return (dh, g, u, x, wg, wu), got


@pytest.mark.parametrize("M", [1, 3, 16, 65, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("N,K", [(520, 640), (1000, 264)])
def test_backward_rows(plan, M, N, K):
    check_backward(plan, M, N, K, seed=M)


@pytest.mark.parametrize("N,K", [(1, 8), (7, 1), (8, 9), (63, 65), (129, 127), (250, 1001), (1001, 250)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [5, 140])
def test_backward_odd_sizes(plan, N, K, dtype, M):
    check_backward(plan, M, N, K, dtype, ACTS[N % 3], seed=N)


@pytest.mark.parametrize("M,N,K", [(40, 6000, 200), (6000, 64, 128), (2048, 1024, 1024), (20, 3000, 4096)])
def test_backward_slices_and_many_tiles(plan, M, N, K):
    args, got = check_backward(plan, M, N, K, seed=M)
    for a, b in zip(plan.gated_linear_backward(*args), got):  # the same bits again
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(1856, 2752, 384), (1500, 2944, 1152), (1500, 2944, 512), (700, 2944, 4096)])
def test_backward_pairs_whose_rows_end_in_half_a_tile(plan, M, N, K):
    # N, K or both 128 past a multiple of 256: the pair's second CTA reads past whole rows
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert {p["tile"] for p in binding.select_gated_backward(152, M, N, K, 76)} == {256}
    check_backward(plan, M, N, K, seed=K)


def test_backward_of_one_side_alone(plan):
    (dh, g, u, x, wg, wu), (dx, dwg, dwu) = check_backward(plan, 130, 200, 264)
    only_x = plan.gated_linear_backward(dh, g, u, None, wg, wu, weight_grads=False)
    only_w = plan.gated_linear_backward(dh, g, u, x, None, None, input_grad=False)
    assert torch.equal(only_x[0], dx) and only_x[1] is only_x[2] is None
    assert only_w[0] is None and torch.equal(only_w[1], dwg) and torch.equal(only_w[2], dwu)
