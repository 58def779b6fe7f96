"""What the Python calls of the operators hand to the library (no GPU): a plan
over a library that only records, host tensors in place of CUDA ones."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding


class Recorder:
    """The library's operator calls: their arguments are kept, nothing runs."""

    def __init__(self, real):
        self.calls = []
        self.before = lambda: None
        self.bwgemm_orthogonalize_workspace = real.bwgemm_orthogonalize_workspace

    def bwgemm_orthogonalize(self, *args):
        names = ("plan", "G", "dtype", "X", "out", "batch", "rows", "cols", "ldg", "stride_g", "ldx", "stride_x", "steps",
                 "coefficients", "eps", "scale", "workspace", "workspace_bytes", "stream")
        self.calls.append(dict(zip(names, args, strict=True)))
        return 0

    def bwgemm_run_scaled(self, *args):
        self.before()
        names = ("plan", "A", "B", "C", "M", "N", "K", "ldc", "out", "accumulate", "stream")
        self.calls.append(dict(zip(names, args, strict=True)))
        return 0


@pytest.fixture
def plan(monkeypatch):
    real = binding.load_library(build_if_missing=True)
    binding._torch()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    p = binding.Plan.__new__(binding.Plan)
    p.lib, p.handle, p.device = Recorder(real), ctypes.c_void_p(), -1  # -1: get_device() of a host tensor
    yield p
    p.handle = None


# ------------------------------------------------------------ orthogonalise
def test_orthogonalize_passes_the_strides_there_are(plan):
    dense = torch.zeros(3, 8, 40, dtype=torch.bfloat16)
    out = torch.zeros(3, 10, 64, dtype=torch.bfloat16)[:, 1:9, :40]
    plan.orthogonalize(dense, out=out)
    plan.orthogonalize(dense[0, :1], out=out[0, :1])  # a single row has no next one
    plan.orthogonalize(dense[0, :, :1], out=out[0, :, :1])
    stack, row, column = plan.lib.calls
    assert [stack[k] for k in ("ldg", "stride_g", "ldx", "stride_x")] == [40, 320, 64, 640]
    assert row["ldg"] == row["ldx"] == 40
    assert (column["ldg"], column["ldx"]) == (40, 64)


@pytest.mark.parametrize("make", [lambda: torch.zeros(1, 40, dtype=torch.bfloat16).expand(8, 40),
                                  lambda: torch.zeros(200, dtype=torch.bfloat16).as_strided((8, 40), (16, 1)),
                                  lambda: torch.zeros(8, 1, dtype=torch.bfloat16)[:1].expand(8, 1),
                                  lambda: torch.zeros(3, 1, 40, dtype=torch.bfloat16).expand(3, 8, 40)])
def test_orthogonalize_rows_closer_than_their_length_reach_the_library_as_they_are(plan, make):
    # which refuses them: it reads (writes) ldg (ldx) elements a row
    t = make()
    dense = torch.zeros(t.shape, dtype=torch.bfloat16)
    plan.orthogonalize(t, out=dense)
    plan.orthogonalize(dense, out=t)
    as_g, as_x = plan.lib.calls
    assert as_g["ldg"] == t.stride(-2) < t.shape[-1] and as_g["ldx"] == dense.stride(-2)
    assert as_x["ldx"] == t.stride(-2) < t.shape[-1] and as_x["ldg"] == dense.stride(-2)


# ------------------------------------------------------------ scaled product
def scaled(rows, K):
    return (torch.zeros(rows, K, dtype=torch.uint8).view(torch.float8_e4m3fn),
            torch.ones(-(-K // 128), rows))


@pytest.mark.parametrize("make", [lambda: torch.zeros(64, 2)[:, :1].t(),             # a column seen as a row
                                  lambda: torch.zeros(1, 128)[:, ::2],
                                  lambda: torch.zeros(1, 1).expand(1, 64),
                                  lambda: torch.zeros(1, 64, 2)[:, :, 0]])
@pytest.mark.parametrize("K", [256, 0])
def test_scaled_product_refuses_a_strided_row_as_result(plan, make, K):
    out = make()
    assert out.shape == (1, 64) and out.stride(1) != 1
    with pytest.raises(ValueError, match="unit stride"):
        plan.gemm_scaled(*scaled(1, K), *scaled(64, K), out=out)
    assert plan.lib.calls == []


def test_scaled_product_row_and_column_results(plan):
    plan.gemm_scaled(*scaled(1, 256), *scaled(61, 256), out=torch.zeros(1, 61))
    plan.gemm_scaled(*scaled(1, 256), *scaled(61, 256), out=torch.zeros(5, 80)[2:3, 16:77])
    plan.gemm_scaled(*scaled(5, 256), *scaled(1, 256), out=torch.zeros(5, 80)[:, 16:17])
    plan.gemm_scaled(*scaled(1, 256), *scaled(1, 256), out=torch.zeros(5, 80)[:1, 16:17])
    assert [(c["M"], c["N"], c["ldc"]) for c in plan.lib.calls] == [(1, 61, 64), (1, 61, 64), (5, 1, 80), (1, 1, 8)]


def record(argument):
    """The bwgemm_scaled_t that the library would read: the argument is its address, or its bytes."""
    if isinstance(argument, bytes):
        return binding.Scaled.from_buffer_copy(argument)
    return binding.Scaled.from_address(argument)


def test_scaled_product_describes_its_own_operands(plan):
    a, b = scaled(3, 300), (torch.zeros(40, 304, dtype=torch.uint8).view(torch.float8_e5m2)[:, :300], torch.ones(3, 1))
    plan.gemm_scaled(*a, *b, out_dtype=torch.float32)
    call, = plan.lib.calls
    A, B = record(call["A"]), record(call["B"])
    assert (A.values, A.ld, A.scales, A.ld_scales, A.type, A.block) == (a[0].data_ptr(), 300, a[1].data_ptr(), 3, 0, 0)
    assert (B.values, B.ld, B.scales, B.ld_scales, B.type, B.block) == (b[0].data_ptr(), 304, b[1].data_ptr(), 1, 1, 1)


def test_scaled_products_of_two_threads_keep_their_operands_apart(plan):
    # ctypes lets other threads run during a call: while the first thread's product is in
    # the library, a second thread starts and ends one of its own
    first, second = (scaled(3, 256), scaled(40, 256)), (scaled(9, 512), scaled(70, 512))
    inside, go = threading.Event(), threading.Event()
    main = threading.get_ident()
    seen = []

    def before():
        if threading.get_ident() != main:
            inside.set()
            assert go.wait(30)

    def run():
        plan.gemm_scaled(*first[0], *first[1])
        call = plan.lib.calls[-1]
        seen.append((call["M"], record(call["A"]).values, record(call["B"]).values))

    plan.lib.before = before
    t = threading.Thread(target=run)
    t.start()
    assert inside.wait(30)
    plan.gemm_scaled(*second[0], *second[1])
    go.set()
    t.join(30)
    assert seen == [(3, first[0][0].data_ptr(), first[1][0].data_ptr())]


# -------------------------------------------------------------- default plans
class Handle:
    """A CUDA tensor as far as the choice of a plan goes."""
    device = torch.device("cuda:0")

    def get_device(self):
        return 0


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def plans(monkeypatch):
    made = []

    class Made:
        def __init__(self, device):
            self.device = device
            made.append(self)

        def gemm(self, *args, **kw):
            return self

        quantize = gemm_scaled = orthogonalize = gemm

    monkeypatch.setattr(binding, "Plan", Made)
    monkeypatch.setattr(binding, "_plans", {})
    binding._torch()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 7, raising=False)
    return made


CALLS = [lambda stream: binding.gemm(Handle(), None, stream=stream), lambda stream: binding.quantize(Handle(), stream=stream),
         lambda stream: binding.gemm_scaled(Handle(), None, None, None, stream=stream),
         lambda stream: binding.orthogonalize(Handle(), stream=stream)]


@pytest.mark.parametrize("call", CALLS)
def test_default_plans_are_of_one_stream_and_one_thread(plans, call):
    # a plan's workspace and status serve one thread and one stream at a time
    here = call(None)
    assert call(None) is here and call(Stream(7)) is here
    side = call(Stream(8))
    assert side is not here and call(Stream(8)) is side
    other = []
    t = threading.Thread(target=lambda: other.extend((call(None), call(None))))
    t.start()
    t.join(30)
    assert other[0] is other[1] and other[0] not in (here, side)
    assert [p.device for p in plans] == [0, 0, 0]


def test_the_calls_share_a_default_plan(plans):
    assert len({id(call(None)) for call in CALLS}) == 1
