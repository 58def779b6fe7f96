"""GPU parity of the 8-bit quantiser, the block-scaled product and the
orthogonalisation against plain numpy forms in 64 bits.

Tolerances, all fixed from the arithmetic:

* quantise: every step is one correctly rounded fp32 operation, so values and
  scales equal the same operations in numpy bit for bit.
* product: the 128 products of a block are exact in fp32 and summed in fp32 (in
  any order and rounding mode: 128 steps of at most 2^-23 of the sum of
  magnitudes), then weighted and added over the K blocks (3 roundings of 2^-24
  each): |error| <= (128 + 2 blocks + 4) 2^-23 sum |a| |b| sa sb, plus the
  result's own rounding (2^-8, 2^-11 or 2^-24 of it).
* orthogonalise: relative 2-norm 4.1e-3: rounding the result to bf16 gives at
  most 2^-9 / sqrt(3) * 1.5 = 1.7e-3, five products of operands rounded to fp16
  about 5 * 2^-11 = 2.4e-3.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding

pytestmark = pytest.mark.gpu

F8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 57344.0, 2, -14)}
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INVALID, ALIGN, WORKSPACE, TIMEOUT = 1, 2, 7, 6


@pytest.fixture(scope="module")
def plan():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library(build_if_missing=True)
    p = binding.Plan(0)
    yield p
    assert p.status() == 0
    p.close()


def host(t):
    """A tensor's values as float64."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def bits8(t):
    return t.detach().view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------- quantise
def round8(v, kind):
    """float32 values to the nearest 8-bit value, ties to even, from the format's definition."""
    _, _, mantissa, least = F8[kind]
    v = v.astype(np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(v)
        step = np.exp2(np.maximum(e - 1, least) - mantissa)
        return np.round(v / step) * step


def quantize_ref(x, square, pow2, kind):
    """(values, scales) of float32 x: the header's operations one by one in float32."""
    limit = np.float32(F8[kind][1])
    rows, cols = x.shape
    q = np.empty((rows, cols))
    rb = 128 if square else 1
    scales = np.empty((-(-cols // 128), -(-rows // rb)), np.float32)
    with np.errstate(all="ignore"):
        for kb in range(scales.shape[0]):
            for r in range(scales.shape[1]):
                blk = x[r * rb:(r + 1) * rb, kb * 128:(kb + 1) * 128]
                a = np.abs(blk).max()
                a = a if np.isnan(a) else np.maximum(a, np.float32(2.0 ** -100))
                s, f = np.float32(a / limit), np.float32(limit / a)
                if pow2 and not np.isnan(a):
                    s = ((s.view(np.uint32) + np.uint32(0x7FFFFF)) & np.uint32(0x7F800000)).view(np.float32)
                    f = np.float32(np.float32(1.0) / s)
                q[r * rb:(r + 1) * rb, kb * 128:(kb + 1) * 128] = round8(blk * f, kind)
                scales[kb, r] = s
    return q, scales


def padded_matrix(values, dtype, extra=0, fill=7.0):
    """values in CUDA rows on 16-byte boundaries, `extra` more elements apart, the rest filled."""
    rows, cols = values.shape
    per = 16 // torch.tensor([], dtype=dtype).element_size()
    wide = torch.full((rows, -(-cols // per) * per + extra * per), fill, dtype=torch.float32)
    wide[:, :cols] = torch.from_numpy(np.ascontiguousarray(values, np.float32))
    return wide.to(dtype).cuda()[:, :cols]


def check_quantize(plan, x, kind, square, pow2, transposed):
    out = plan.quantize(x, blocks="square" if square else "row", transposed=transposed, pow2=pow2, dtype=F8[kind][0])
    xf = x.detach().float().cpu().numpy()
    q, s = quantize_ref(xf, square, pow2, kind)
    want = [q, s]
    if transposed:
        want += [q.T, s.T] if square else list(quantize_ref(np.ascontiguousarray(xf.T), False, pow2, kind))
    assert len(out) == len(want)
    for got, ref in zip(out, want):
        assert tuple(got.shape) == ref.shape
        np.testing.assert_array_equal(host(got), ref.astype(np.float64))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (1, 129), (127, 128), (128, 127), (129, 257), (300, 1000),
                                       (5, 4100), (257, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_sizes(plan, rows, cols, dtype):
    rng = np.random.default_rng(rows * 7919 + cols)
    x = padded_matrix(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 6, (1, cols))), T[dtype], extra=1)
    for square in (False, True):
        check_quantize(plan, x, "e4m3", square, pow2=False, transposed=True)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("square", [False, True])
def test_quantize_forms(plan, kind, pow2, transposed, square):
    rng = np.random.default_rng(11)
    x = padded_matrix(rng.standard_normal((200, 333)), torch.bfloat16)
    check_quantize(plan, x, kind, square, pow2, transposed)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_quantize_every_16_bit_value(plan, kind):
    # all finite bf16 values, a block per 128 consecutive bit patterns (ties, subnormals, the largest)
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float().numpy()
    v = v[np.isfinite(v)]
    x = padded_matrix(v[:len(v) // 128 * 128].reshape(-1, 128), torch.bfloat16)
    for pow2 in (False, True):
        check_quantize(plan, x, kind, False, pow2, False)


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_special_blocks(plan, square, pow2):
    # a block of zeros, one below the smallest scale, one with a NaN, with an infinity, the largest fp32
    x = np.random.default_rng(3).standard_normal((256, 640)).astype(np.float32)
    x[:, :128] = 0
    x[:, 128:256] *= np.float32(2.0 ** -120)
    x[5, 260] = np.nan
    x[130, 390] = np.inf
    x[7, 515] = np.finfo(np.float32).max
    check_quantize(plan, padded_matrix(x, torch.float32), "e4m3", square, pow2, True)


def test_quantize_writes_nothing_else(plan):
    # raw call with rows further apart than needed: the bytes between stay
    rows, cols = 131, 200
    x = padded_matrix(np.random.default_rng(4).standard_normal((rows, cols)), torch.bfloat16)
    q = torch.full((rows + 1, 256), 0xA5, dtype=torch.uint8, device="cuda")
    qt = torch.full((cols + 1, 192), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((3, rows + 3), -1.0, device="cuda")
    st = torch.full((3, cols + 5), -1.0, device="cuda")
    rc = plan.lib.bwgemm_quantize(plan.handle, x.data_ptr(), 0, rows, cols, x.stride(0), 0, 0, 0, q.data_ptr(), 256,
                                  s.data_ptr(), s.stride(0), qt.data_ptr(), 192, st.data_ptr(), st.stride(0),
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want = plan.quantize(x, transposed=True)
    assert (q[rows:] == 0xA5).all() and (q[:, cols:] == 0xA5).all()
    assert (qt[cols:] == 0xA5).all() and (qt[:, rows:] == 0xA5).all()
    assert (s[2:] == -1).all() and (s[:, rows:] == -1).all() and (st[2:] == -1).all() and (st[:, cols:] == -1).all()
    np.testing.assert_array_equal(q[:rows, :cols].cpu().numpy(), bits8(want[0]))
    np.testing.assert_array_equal(qt[:cols, :rows].cpu().numpy(), bits8(want[2]))


def test_quantize_refusals(plan):
    x = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        plan.quantize(x.double())
    with pytest.raises(TypeError):
        plan.quantize(x, dtype=torch.int8)
    with pytest.raises(ValueError):
        plan.quantize(x, blocks="column")
    with pytest.raises(ValueError):
        plan.quantize(x.t())
    with pytest.raises(ValueError):
        plan.quantize(x.cpu())
    with pytest.raises(binding.BwgemmError) as e:
        plan.quantize(x[:, 1:])  # rows off 16-byte boundaries
    assert e.value.status == ALIGN
    q = torch.zeros(64, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 64, device="cuda")

    def raw(X=x.data_ptr(), dtype=0, rows=64, cols=256, ldx=256, block=0, kind=0, Q=q.data_ptr(), ldq=256,
            S=s.data_ptr(), lds=64, QT=None, ldqt=0, ST=None, ldst=0):
        return plan.lib.bwgemm_quantize(plan.handle, X, dtype, rows, cols, ldx, block, kind, 0, Q, ldq, S, lds, QT,
                                        ldqt, ST, ldst, None)
    assert raw() == 0 and raw(rows=0) == 0 and raw(cols=0) == 0
    for bad in (dict(dtype=3), dict(rows=-1), dict(ldx=255), dict(block=2), dict(kind=2), dict(Q=None), dict(ldq=240),
                dict(S=None), dict(lds=63), dict(QT=q.data_ptr()), dict(QT=q.data_ptr(), ST=s.data_ptr(), ldqt=48, ldst=256),
                dict(X=np.zeros(4).ctypes.data // 16 * 16)):
        assert raw(**bad) == INVALID, bad
    for bad in (dict(X=x.data_ptr() + 2), dict(ldx=257), dict(Q=q.data_ptr() + 8, rows=1), dict(ldq=257, rows=1),
                dict(S=s.data_ptr() + 2)):
        assert raw(**bad) == ALIGN, bad


# ------------------------------------------------------------- scaled product
def random_scaled(rows, K, kind, square, seed, scale_pow2=False):
    """Random 8-bit values (device, padded rows), fp32 scales (device) and both as float64."""
    rng = np.random.default_rng(seed)
    v = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32) * 20).to(F8[kind][0])
    wide = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.uint8)
    wide[:, :K] = v.view(torch.uint8)
    per = -(-rows // 128) if square else rows
    s = np.exp2(rng.uniform(-9, 1, (-(-K // 128), per))).astype(np.float32)
    if scale_pow2:
        s = np.exp2(np.round(np.log2(s))).astype(np.float32)
    full = np.repeat(s, 128, axis=1)[:, :rows] if square and rows > 1 else s
    values = v.double().numpy() * np.repeat(full.T.astype(np.float64), 128, axis=1)[:, :K]
    return wide.cuda().view(F8[kind][0])[:, :K], torch.from_numpy(s).cuda(), values


def product_bound(a, b, out):
    """Elementwise bound of the module's docstring, and the exact product."""
    exact = a @ b.T
    blocks = -(-a.shape[1] // 128)
    own = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}[out]
    return exact, (128 + 2 * blocks + 4) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + own * np.abs(exact) + 2.0 ** -24


def check_product(plan, M, N, K, out="fp32", a_square=False, b_square=True, a_kind="e4m3", b_kind="e4m3", seed=0):
    A, sa, a = random_scaled(M, K, a_kind, a_square, seed)
    B, sb, b = random_scaled(N, K, b_kind, b_square, seed + 1)
    C = plan.gemm_scaled(A, sa, B, sb, out_dtype=T[out])
    assert plan.status() == 0
    exact, bound = product_bound(a, b, out)
    assert C.shape == (M, N) and C.dtype == T[out]
    assert (np.abs(host(C) - exact) <= bound).all()
    return C


# every tile form: 16 to 128 rows swapped, 128 and 256 columns in order, and their edges
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 257, 640])
@pytest.mark.parametrize("b_square", [True, False])
def test_scaled_rows(plan, M, b_square):
    check_product(plan, M, 520, 640, b_square=b_square, seed=M)


@pytest.mark.parametrize("K", [1, 15, 16, 127, 128, 129, 255, 256, 384, 513, 1152, 5005])
@pytest.mark.parametrize("M", [3, 48, 300])
def test_scaled_depths(plan, M, K):
    # partial last blocks, odd numbers of blocks (stages of two and four), splits over K
    check_product(plan, M, 264, K, seed=K)


@pytest.mark.parametrize("N", [1, 7, 8, 63, 129, 250, 1000, 3001])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M", [5, 260])
def test_scaled_columns_and_outputs(plan, N, out, M):
    check_product(plan, M, N, 512, out=out, seed=N)


@pytest.mark.parametrize("a_square", [False, True])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("kinds", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M", [20, 140, 600])
def test_scaled_forms(plan, M, a_square, b_square, kinds):
    check_product(plan, M, 700, 900, a_square=a_square, b_square=b_square, a_kind=kinds[0], b_kind=kinds[1], seed=M)


# the kernel for few rows: both groups of eight, every pair of types and kind of block,
# one to many K blocks per warp
@pytest.mark.parametrize("a_square", [False, True])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("kinds", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M,N,K", [(1, 259, 2056), (7, 131, 4200), (8, 1001, 128), (9, 130, 3900), (16, 77, 1030)])
def test_scaled_few_rows_forms(plan, M, N, K, a_square, b_square, kinds):
    check_product(plan, M, N, K, a_square=a_square, b_square=b_square, a_kind=kinds[0], b_kind=kinds[1], seed=M)


# so many weights that tiles take even a few rows
@pytest.mark.parametrize("M", [1, 5, 13])
@pytest.mark.parametrize("b_square", [False, True])
def test_scaled_few_rows_many_weights(plan, M, b_square):
    check_product(plan, M, 20008, 6100, b_square=b_square, seed=M)


@pytest.mark.parametrize("M", [2, 12])
def test_scaled_few_rows_in_the_last_bytes(plan, M):
    # operands that end with the last value of their last row, a sum onto C in place
    N, K, ld = 40, 1030, 1040
    A, sa, a = random_scaled(M, K, "e4m3", False, 5)
    B, sb, b = random_scaled(N, K, "e4m3", True, 6)
    tight = []
    for x, rows in ((A, M), (B, N)):
        y = torch.zeros((rows - 1) * ld + K, dtype=torch.uint8, device="cuda").as_strided((rows, K), (ld, 1))
        y.copy_(x.view(torch.uint8))
        tight.append(y.view(torch.float8_e4m3fn))
    C = torch.ones(M, N, device="cuda")
    plan.gemm_scaled(tight[0], sa, tight[1], sb, out=C, accumulate=True)
    exact, bound = product_bound(a, b, "fp32")
    assert (np.abs(host(C) - (exact + 1)) <= bound + 2.0 ** -24 * (np.abs(exact) + 1)).all()


@pytest.mark.parametrize("M", [3, 11])
def test_scaled_few_rows_nan_stays_in_its_row(plan, M):
    A, sa, _ = random_scaled(M, 1100, "e4m3", False, 1)
    B, sb, _ = random_scaled(90, 1100, "e4m3", True, 2)
    want = plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32)
    A.view(torch.uint8)[M - 1, 1099] = 0x7F
    got = plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32)
    assert torch.isnan(got[M - 1]).all() and torch.equal(got[: M - 1], want[: M - 1])


@pytest.mark.parametrize("M,N,K", [(2000, 3000, 768), (4096, 300, 2048), (130, 9000, 1024), (64, 20000, 384),
                                   (1, 512, 30000), (300, 128, 20000)])
def test_scaled_many_tiles(plan, M, N, K):
    # several tiles per CTA, the last wave split over K, tiles split many ways
    check_product(plan, M, N, K, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(300, 520, 5005), (1, 512, 30000), (48, 300, 9000), (700, 400, 1000)])
def test_scaled_integers_bit_exact_and_repeatable(plan, M, N, K):
    # values -2..2 and power-of-two scales of one size: every sum is exact in fp32
    rng = np.random.default_rng(5)
    out = []
    for rows in (M, N):
        v = torch.from_numpy(rng.integers(-2, 3, (rows, K)).astype(np.float32)).to(torch.float8_e4m3fn)
        wide = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.uint8)
        wide[:, :K] = v.view(torch.uint8)
        out += [wide.cuda().view(torch.float8_e4m3fn)[:, :K], torch.full((-(-K // 128), rows), 0.25, device="cuda"),
                v.double().numpy() * 0.25]
    A, sa, a, B, sb, b = out
    C = plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32)
    np.testing.assert_array_equal(host(C), a @ b.T)
    for _ in range(3):
        assert torch.equal(plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32), C)


def test_scaled_same_bits_again(plan):
    A, sa, _ = random_scaled(300, 7000, "e4m3", False, 1)
    B, sb, _ = random_scaled(500, 7000, "e4m3", True, 2)
    first = plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32), first)


def test_scaled_small_workspace():
    # no room for partial tiles: whole tiles only, the same product
    with binding.Plan(0, workspace_bytes=(1 << 20) + 4096) as p:
        check_product(p, 300, 520, 5005, seed=8)
        check_product(p, 4, 520, 20000, seed=9)


@pytest.mark.parametrize("M", [40, 300])
def test_scaled_accumulate_and_padding(plan, M):
    A, sa, a = random_scaled(M, 400, "e4m3", False, 3)
    B, sb, b = random_scaled(333, 400, "e4m3", True, 4)
    exact, bound = product_bound(a, b, "fp32")
    wide = torch.full((M + 2, 340), 3.0, device="cuda")
    out = wide[1:M + 1, :333]
    for i in range(1, 4):
        plan.gemm_scaled(A, sa, B, sb, out=out, accumulate=True)
        # i products and i additions to a sum of known magnitude
        assert (np.abs(host(out) - 3.0 - i * exact) <= i * bound + 2 * i * 2.0 ** -24 * (3 + i * np.abs(exact))).all()
    assert (wide[0] == 3).all() and (wide[M + 1] == 3).all() and (wide[:, 333:] == 3).all()
    half = torch.full((M + 2, 344), 3.0, dtype=torch.bfloat16, device="cuda")
    plan.gemm_scaled(A, sa, B, sb, out=half[1:M + 1, :333])
    assert (half[0] == 3).all() and (half[M + 1] == 3).all() and (half[:, 333:] == 3).all()
    exact, bound = product_bound(a, b, "bf16")
    assert (np.abs(host(half[1:M + 1, :333]) - exact) <= bound).all()


@pytest.mark.parametrize("M", [30, 200])
def test_scaled_special_values(plan, M):
    # zero scales, a NaN value, an infinite scale: each stays in its own row or column
    A, sa, a = random_scaled(M, 384, "e4m3", False, 6)
    B, sb, b = random_scaled(260, 384, "e4m3", False, 7)
    sa[:, 3] = 0
    A.view(torch.uint8)[9, 200] = 0x7F  # NaN
    sb[1, 17] = float("inf")
    C = host(plan.gemm_scaled(A, sa, B, sb, out_dtype=torch.float32))
    assert np.isnan(C[9]).all() and np.isnan(C[3, 17]) and not np.isfinite(C[:, 17]).any()
    rows = [i for i in range(M) if i not in (3, 9)]
    cols = [j for j in range(260) if j != 17]
    exact, bound = product_bound(a[rows], b[cols], "fp32")
    assert (np.abs(C[np.ix_(rows, cols)] - exact) <= bound).all() and (C[3][cols] == 0).all()


def test_scaled_empty_sizes(plan):
    A, sa, _ = random_scaled(6, 256, "e4m3", False, 1)
    B, sb, _ = random_scaled(8, 256, "e4m3", True, 2)
    assert plan.gemm_scaled(A[:0], sa[:, :0], B, sb).shape == (0, 8)
    z = plan.gemm_scaled(A[:, :0], sa[:0], B[:, :0], sb[:0])
    assert z.shape == (6, 8) and (z == 0).all()
    out = torch.full((6, 8), 2.0, device="cuda")
    plan.gemm_scaled(A[:, :0], sa[:0], B[:, :0], sb[:0], out=out, accumulate=True)
    assert (out == 2).all()


def test_scaled_offsets_past_32_bits(plan):
    # rows of A more than 2^31 bytes apart, rows of C more than 2^31 elements
    M, N, K = 3, 200, 256
    ld, ldc = (1 << 31) + 16, (1 << 31) + 8
    A0, sa, a = random_scaled(M, K, "e4m3", False, 1)
    B, sb, b = random_scaled(N, K, "e4m3", True, 2)
    big = torch.empty((M - 1) * ld + K, dtype=torch.uint8, device="cuda")
    A = big.as_strided((M, K), (ld, 1))
    A.copy_(A0.view(torch.uint8))
    flat = torch.empty((M - 1) * ldc + N, dtype=torch.bfloat16, device="cuda")
    C = flat.as_strided((M, N), (ldc, 1))
    plan.gemm_scaled(A.view(torch.float8_e4m3fn), sa, B, sb, out=C)
    exact, bound = product_bound(a, b, "bf16")
    assert (np.abs(host(C) - exact) <= bound).all()


def test_scaled_other_stream_and_graph(plan):
    A, sa, a = random_scaled(70, 640, "e4m3", False, 1)
    B, sb, b = random_scaled(300, 640, "e4m3", True, 2)
    want = plan.gemm_scaled(A, sa, B, sb)
    side = torch.cuda.Stream()
    out = torch.zeros(70, 304, dtype=want.dtype, device="cuda")[:, :300]  # rows on 16-byte boundaries
    side.wait_stream(torch.cuda.current_stream())
    plan.gemm_scaled(A, sa, B, sb, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        q = plan.quantize(want)
        plan.gemm_scaled(A, sa, B, sb, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    np.testing.assert_array_equal(bits8(q[0]), bits8(plan.quantize(want)[0]))


def test_scaled_refusals(plan):
    A, sa, _ = random_scaled(16, 256, "e4m3", False, 1)
    B, sb, _ = random_scaled(32, 256, "e4m3", True, 2)
    ok = dict(A=A, scale_a=sa, B=B, scale_b=sb)
    for error, change in ((TypeError, dict(A=A.view(torch.uint8))), (TypeError, dict(scale_a=sa.double())),
                          (ValueError, dict(scale_a=sa[:, :7])), (ValueError, dict(scale_b=sb[:1])),
                          (ValueError, dict(B=B[:, :128], scale_b=sb[:1])), (ValueError, dict(A=A.cpu())),
                          (ValueError, dict(accumulate=True)), (TypeError, dict(out_dtype=torch.float64)),
                          (ValueError, dict(out=torch.zeros(16, 31, device="cuda")))):
        with pytest.raises(error):
            plan.gemm_scaled(**{**ok, **change})
    with pytest.raises(binding.BwgemmError) as e:
        plan.gemm_scaled(**ok, out=torch.zeros(16, 32, dtype=torch.bfloat16, device="cuda"), accumulate=True)
    assert e.value.status == INVALID
    with pytest.raises(binding.BwgemmError) as e:
        plan.gemm_scaled(**ok, out=torch.zeros(16, 33, dtype=torch.bfloat16, device="cuda")[:, :32])
    assert e.value.status == ALIGN

    def raw(c=torch.zeros(16, 32, device="cuda"), M=16, N=32, K=256, ldc=32, out=2, **change):
        a = binding.Scaled(A.data_ptr(), 256, sa.data_ptr(), 16, 0, 0)
        b = binding.Scaled(B.data_ptr(), 256, sb.data_ptr(), 1, 0, 1)
        for k, v in change.items():
            setattr(a, k, v)
        return plan.lib.bwgemm_run_scaled(plan.handle, ctypes.addressof(a), ctypes.addressof(b), c.data_ptr(), M, N, K,
                                          ldc, out, 0, None)
    assert raw() == 0
    for bad in (dict(M=-1), dict(out=3), dict(ldc=31), dict(values=None), dict(scales=None), dict(ld=240),
                dict(ld_scales=15), dict(type=2), dict(block=2), dict(values=np.zeros(64).ctypes.data // 16 * 16)):
        assert raw(**bad) == INVALID, bad
    for bad in (dict(values=A.data_ptr() + 8), dict(ld=264), dict(scales=sa.data_ptr() + 2), dict(ldc=33)):
        assert raw(**bad) == ALIGN, bad
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [24, 300])
def test_scaled_timeout_is_reported(M):
    # the producer of CTA 0 never fills a stage: the bounded waits run out and
    # the plan works again afterwards
    A, sa, a = random_scaled(M, 1024, "e4m3", False, 1)
    B, sb, b = random_scaled(300, 1024, "e4m3", True, 2)
    with binding.Plan(0, stall_kblock=1, timeout_ns=20_000_000) as p:
        p.gemm_scaled(A, sa, B, sb)
        assert p.status() == TIMEOUT and p.last_device_status() != 0
        assert p.status() == 0
    with binding.Plan(0) as p:
        check_product(p, M, 300, 1024, seed=1)


# ------------------------------------------------------------ orthogonalise
COEF = (3.4445, -4.7750, 2.0315)


def orthogonalize_ref(g, steps=5, coefficients=COEF, eps=1e-7, scale=1.0):
    g = g.astype(np.float64)
    x = g if g.shape[0] <= g.shape[1] else g.T
    x = x / (np.linalg.norm(x) + eps)
    for i in range(steps):
        a, b, c = coefficients if np.ndim(coefficients) == 1 else coefficients[i]
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return scale * (x if g.shape[0] <= g.shape[1] else x.T)


def rel(got, want):
    return np.linalg.norm(host(got) - want) / np.linalg.norm(want)


def gradient(rows, cols, seed, loud=0.25):
    rng = np.random.default_rng(seed)
    return 1e-3 * (rng.standard_normal((rows, cols)) + loud * rng.standard_normal((rows, 4)) @ rng.standard_normal((4, cols)))


@pytest.mark.parametrize("rows,cols", [(64, 64), (128, 128), (129, 129), (100, 700), (700, 100), (300, 1000), (1000, 301),
                                       (17, 3000), (3000, 17), (384, 385), (600, 520)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_orthogonalize_sizes(plan, rows, cols, dtype):
    g = torch.from_numpy(gradient(rows, cols, rows + cols)).to(T[dtype]).cuda()
    x = plan.orthogonalize(g)
    assert plan.status() == 0 and x.shape == g.shape and x.dtype == torch.bfloat16
    assert rel(x, orthogonalize_ref(host(g))) <= 4.1e-3


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 500), (500, 1), (2, 3), (5, 5)])
def test_orthogonalize_tiny(plan, rows, cols):
    g = torch.from_numpy(gradient(rows, cols, 3) * 1e3).float().cuda()
    assert rel(plan.orthogonalize(g), orthogonalize_ref(host(g))) <= 4.1e-3


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_orthogonalize_steps_and_coefficients(plan, steps, dtype):
    g = torch.from_numpy(gradient(200, 330, steps)).to(T[dtype]).cuda()
    assert rel(plan.orthogonalize(g, steps=steps, scale=0.5), orthogonalize_ref(host(g), steps, scale=0.5)) <= 4.1e-3
    table = [(2.0 - 0.1 * i, -1.5 + 0.05 * i, 0.5) for i in range(steps)]
    assert rel(plan.orthogonalize(g, steps=steps, coefficients=table), orthogonalize_ref(host(g), steps, table)) <= 4.1e-3


def test_orthogonalize_dominant_directions(plan):
    # eight directions 30 times the rest: what one fp16 term of X cannot carry
    rng = np.random.default_rng(9)
    g = rng.standard_normal((512, 640)) / 30 + rng.standard_normal((512, 8)) @ rng.standard_normal((8, 640))
    g = torch.from_numpy(g).to(torch.bfloat16).cuda()
    assert rel(plan.orthogonalize(g), orthogonalize_ref(host(g))) <= 4.1e-3


def test_orthogonalize_singular_values(plan):
    g = torch.from_numpy(gradient(256, 512, 1, loud=0)).to(torch.bfloat16).cuda()
    s = np.linalg.svd(host(plan.orthogonalize(g)), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.25


@pytest.mark.parametrize("power", [-30, -10, 0, 12, 40])
def test_orthogonalize_ignores_size(plan, power):
    # a power of two times G gives the same bits (until eps counts)
    g = torch.from_numpy(gradient(130, 260, 5) * 1e3).float().cuda()
    assert torch.equal(plan.orthogonalize(g * 2.0 ** power, eps=0.0), plan.orthogonalize(g, eps=0.0))


def test_orthogonalize_stack_is_each_alone(plan):
    g = torch.stack([torch.from_numpy(gradient(150, 272, s)) for s in range(7)]).to(torch.bfloat16).cuda()
    x = plan.orthogonalize(g)
    for i in range(7):
        assert rel(x[i], orthogonalize_ref(host(g[i]))) <= 4.1e-3
    assert torch.equal(plan.orthogonalize(g), x)
    h = g.transpose(1, 2).contiguous()
    for i in range(7):
        assert rel(plan.orthogonalize(h)[i], orthogonalize_ref(host(h[i]))) <= 4.1e-3


@pytest.mark.parametrize("out_dtype", ["bf16", "fp16"])
def test_orthogonalize_strides_and_padding(plan, out_dtype):
    # rows off 16-byte boundaries, matrices apart, and nothing written between them
    for rows, cols in ((90, 200), (200, 91)):
        wide = torch.zeros(3, rows + 1, cols + 9, dtype=torch.float32, device="cuda")
        for i in range(3):
            wide[i, 1:, 5:5 + cols] = torch.from_numpy(gradient(rows, cols, i)).float()
        g = wide[:, 1:, 5:5 + cols]
        hold = torch.full((3, rows + 2, cols + 7), 9.0, dtype=T[out_dtype], device="cuda")
        out = hold[:, 1:rows + 1, 3:3 + cols]
        plan.orthogonalize(g, out=out)
        for i in range(3):
            assert rel(out[i], orthogonalize_ref(host(g[i]))) <= 4.1e-3
        keep = torch.ones_like(hold, dtype=torch.bool)
        keep[:, 1:rows + 1, 3:3 + cols] = False
        assert (hold[keep] == 9).all()
        aligned = torch.full((3, rows + 2, 256), 9.0, dtype=T[out_dtype], device="cuda")
        plan.orthogonalize(g, out=aligned[:, 1:rows + 1, :cols])
        assert torch.equal(aligned[:, 1:rows + 1, :cols], out)
        assert (aligned[:, :, cols:] == 9).all() and (aligned[:, 0] == 9).all() and (aligned[:, rows + 1] == 9).all()


def test_orthogonalize_in_place(plan):
    g = torch.from_numpy(gradient(256, 384, 2)).to(torch.bfloat16).cuda()
    want = plan.orthogonalize(g)
    assert plan.orthogonalize(g, out=g) is g and torch.equal(g, want)


def test_orthogonalize_zeros_and_nans(plan):
    g = torch.zeros(3, 140, 200, device="cuda")
    g[1] = torch.from_numpy(gradient(140, 200, 1)).float()
    g[2] = g[1]
    g[2, 5, 7] = float("nan")
    x = plan.orthogonalize(g)
    assert (x[0] == 0).all() and torch.isnan(x[2]).all()
    assert rel(x[1], orthogonalize_ref(host(g[1]))) <= 4.1e-3  # its neighbours leave it alone
    assert plan.orthogonalize(g[:0]).shape == (0, 140, 200)
    assert plan.orthogonalize(g[0, :0]).shape == (0, 200)
    # a workspace that held NaNs leaves no trace
    assert rel(plan.orthogonalize(g[1]), orthogonalize_ref(host(g[1]))) <= 4.1e-3


def test_orthogonalize_stream_and_graph(plan):
    g = torch.from_numpy(gradient(300, 500, 4)).to(torch.bfloat16).cuda()
    want = plan.orthogonalize(g)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.orthogonalize(g, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.orthogonalize(g, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_orthogonalize_refusals(plan):
    g = torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda")
    for error, call in ((TypeError, lambda: plan.orthogonalize(g.double())), (ValueError, lambda: plan.orthogonalize(g[0])),
                        (ValueError, lambda: plan.orthogonalize(g.cpu())), (ValueError, lambda: plan.orthogonalize(g.t())),
                        (TypeError, lambda: plan.orthogonalize(g, out=torch.zeros(64, 128, device="cuda"))),
                        (ValueError, lambda: plan.orthogonalize(g, out=torch.zeros_like(g[:3]))),
                        (ValueError, lambda: plan.orthogonalize(g, coefficients=[COEF] * 4))):
        with pytest.raises(error):
            call()
    for kw in (dict(steps=0, coefficients=[COEF]), dict(eps=-1.0), dict(eps=float("nan")), dict(steps=65)):
        with pytest.raises((binding.BwgemmError, ValueError)):
            plan.orthogonalize(g, **kw)
    x = torch.zeros_like(g)
    n = ctypes.c_uint64()
    assert plan.lib.bwgemm_orthogonalize_workspace(1, 64, 128, ctypes.byref(n)) == 0
    ws = torch.zeros(n.value + 256, dtype=torch.uint8, device="cuda")

    def raw(G=g.data_ptr(), dtype=0, X=x.data_ptr(), out=0, batch=1, rows=64, cols=128, ldg=128, sg=0, ldx=128, sx=0,
            steps=5, w=ws.data_ptr(), wb=n.value):
        return plan.lib.bwgemm_orthogonalize(plan.handle, G, dtype, X, out, batch, rows, cols, ldg, sg, ldx, sx, steps,
                                             None, 1e-7, 1.0, w, wb, None)
    assert raw() == 0
    for bad in (dict(G=None), dict(X=None), dict(w=None), dict(dtype=3), dict(out=2), dict(rows=-1), dict(ldg=127),
                dict(ldx=127), dict(steps=0), dict(steps=65), dict(batch=2, sg=100, sx=8192),
                dict(G=np.zeros(4).ctypes.data // 16 * 16)):
        assert raw(**bad) == INVALID, bad
    assert raw(wb=n.value - 1) == WORKSPACE
    for bad in (dict(w=ws.data_ptr() + 16), dict(G=g.data_ptr() + 1), dict(X=x.data_ptr() + 1)):
        assert raw(**bad) == ALIGN, bad
    torch.cuda.synchronize()


# deep K in slices, tiles of 128 and of 256, above and below the diagonal
@pytest.mark.parametrize("rows,cols", [(1024, 9000), (9000, 700), (520, 6001), (129, 30000)])
def test_orthogonalize_slices(plan, rows, cols):
    g = torch.from_numpy(gradient(rows, cols, rows)).to(torch.bfloat16).cuda()
    x = plan.orthogonalize(g)
    assert torch.equal(plan.orthogonalize(g), x)
    assert rel(x, orthogonalize_ref(host(g))) <= 4.1e-3


def test_orthogonalize_small_workspace():
    # no room for slices: whole tiles
    g = torch.from_numpy(gradient(200, 9000, 1)).to(torch.bfloat16).cuda()
    with binding.Plan(0, workspace_bytes=(1 << 20) + 4096) as p:
        assert rel(p.orthogonalize(g), orthogonalize_ref(host(g))) <= 4.1e-3


# Singular values close together: B is close to a multiple of I, whose rounding
# would show in the whole result.  Tolerance: 1.45 times the rounding of the result
# to bf16 (1.7e-3) in a simulation of every other rounding, and a quarter more.
@pytest.mark.parametrize("rows,cols", [(20, 2816), (41, 1860), (3500, 27), (64, 5000), (384, 9000), (6000, 200)])
@pytest.mark.parametrize("seed", range(4))
def test_orthogonalize_even_singular_values(plan, rows, cols, seed):
    g = np.random.default_rng(seed).standard_normal((rows, cols)).astype(np.float32)
    g = torch.from_numpy(g).to(torch.bfloat16)
    assert rel(plan.orthogonalize(g.cuda()), orthogonalize_ref(host(g))) <= 3.1e-3


def test_orthogonalize_timeout_is_reported():
    g = torch.from_numpy(gradient(256, 512, 4)).to(torch.bfloat16).cuda()
    with binding.Plan(0, stall_kblock=1, timeout_ns=20_000_000) as p:
        p.orthogonalize(g)
        assert p.status() == TIMEOUT
        assert p.status() == 0
    with binding.Plan(0) as p:
        assert rel(p.orthogonalize(g), orthogonalize_ref(host(g))) <= 4.1e-3


@pytest.mark.parametrize("op", ["quantize", "gemm_scaled", "orthogonalize"])
def test_other_streams_results_are_not_this_streams_memory(plan, op):
    # memory freed here may still be read by work pending here, which the other
    # stream does not wait for
    x = torch.randn(512, 1024, device="cuda").to(torch.bfloat16)
    q, s = plan.quantize(x)
    call = {"quantize": lambda st: plan.quantize(x, stream=st)[0], "orthogonalize": lambda st: plan.orthogonalize(x, stream=st),
            "gemm_scaled": lambda st: plan.gemm_scaled(q, s, q, s, stream=st)}[op]
    torch.cuda.synchronize()
    want = call(None)
    freed = want.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = freed.data_ptr()
    del freed
    got = call(side)
    side.synchronize()
    assert got.data_ptr() != at
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


# ----------------------------------------------------------------- together
def dequantized(q, s):
    rows, cols = q.shape
    full = s if s.shape[1] == rows else s.repeat_interleave(128, dim=1)[:, :rows]
    return host(q) * np.repeat(host(full).T, 128, axis=1)[:, :cols]


@pytest.mark.parametrize("tokens,inner,outer", [(96, 200, 136), (300, 128, 520)])
def test_linear_gradients(plan, tokens, inner, outer):
    from dense_gemm_blackwell_03_gb300.linear_training import scaled_linear
    rng = np.random.default_rng(tokens)
    x = torch.from_numpy(rng.standard_normal((tokens, inner))).float().cuda().requires_grad_()
    w = torch.from_numpy(rng.standard_normal((outer, inner)) / inner ** 0.5).float().cuda().requires_grad_()
    dy = torch.from_numpy(rng.standard_normal((tokens, outer))).float().cuda()
    y = scaled_linear(x, w)
    y.backward(dy)
    # against the formulas on the quantised operands
    xq, xs, xtq, xts = plan.quantize(x.detach(), transposed=True)
    wq, ws, wtq, wts = plan.quantize(w.detach(), blocks="square", transposed=True)
    gq, gs, gtq, gts = plan.quantize(dy, transposed=True)
    for got, a, b in ((y, (xq, xs), (wq, ws)), (x.grad, (gq, gs), (wtq, wts)), (w.grad, (gtq, gts), (xtq, xts))):
        exact, bound = product_bound(dequantized(*a), dequantized(*b), "fp32")
        assert (np.abs(host(got) - exact) <= bound).all()
    # against differences of the unquantised loss <y, dy>: e4m3 is within 2^-4 of a
    # value, two operands a product, errors of random sign
    for t, other in ((x, w), (w, x)):
        d = torch.from_numpy(rng.standard_normal(tuple(t.shape))).double().cuda()
        pair = (lambda v: (v @ other.detach().double().t())) if t is x else (lambda v: (x.detach().double() @ v.t()))
        h = 1e-3
        diff = ((pair(t.detach().double() + h * d) - pair(t.detach().double() - h * d)) * dy.double()).sum() / (2 * h)
        got = (t.grad.double() * d).sum()
        spread = t.grad.double().norm() * d.norm() / d.numel() ** 0.5  # size of such a product of random directions
        assert abs(float(got - diff)) <= 2 * 2.0 ** -4 * float(spread) * 3


def test_linear_training_converges():
    from dense_gemm_blackwell_03_gb300.linear_training import train
    losses = train(steps=60)
    assert all(np.isfinite(losses)) and np.mean(losses[-5:]) < 0.5 * np.mean(losses[:5])
