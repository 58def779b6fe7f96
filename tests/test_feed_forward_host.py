"""The gated layer's and the 8-bit integers' host side (no GPU): struct layouts, refusals that need
no device, workspace sizes, the division of the work, and what the Python calls hand on."""
from __future__ import annotations

import ctypes
import os
import random
import shutil
import subprocess
import threading

import pytest
import torch

from dense_gemm_blackwell_03_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, ALIGN, UNSUP, WORKSPACE = 1, 2, 3, 7
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def lib():
    return binding.load_library(build_if_missing=True)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_layouts_and_codes(tmp_path):
    structs = (("bwgemm_matrix_t", binding.Matrix), ("bwgemm_lanes_config_t", binding.LanesConfig))
    fields = [(name, s, f) for name, s in structs for f, _ in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bwgemm.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", offsetof({n}, {f}));\n' for n, _, f in fields)
                   + "".join(f'  printf("%zu\\n", sizeof({n}));\n' for n, _ in structs)
                   + '  printf("%d %d %d\\n", BWGEMM_SILU, BWGEMM_GELU, BWGEMM_GELU_TANH);\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == ([getattr(s, f).offset for _, s, f in fields] + [ctypes.sizeof(s) for _, s in structs]
                   + [binding.SILU, binding.GELU, binding.GELU_TANH])


def test_package_exports_the_operators():
    import dense_gemm_blackwell_03_gb300 as pkg
    for name in ("gated_linear", "gated_linear_backward", "quantize_int8", "gemm_int8"):
        assert name in pkg.__all__ and getattr(pkg, name) is getattr(binding, name)


def test_null_plans_are_refused(lib):
    m = ctypes.addressof(binding.Matrix(0x1000, 64))
    assert lib.bwgemm_gated(None, m, m, m, m, None, None, 1, 8, 8, 0, 0, None) == INVALID
    assert lib.bwgemm_gated_backward(None, *[m] * 9, 1, 8, 8, 0, 0, 0x1000, 1 << 20, None) == INVALID
    assert lib.bwgemm_quantize_integer(None, 0x1000, 0, 1, 16, 16, 0x2000, 16, 0x3000, None) == INVALID
    assert lib.bwgemm_run_integer(None, 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 1, 8, 16, 16, 16, 8, 0, None, 0,
                                  None) == INVALID


def test_host_tensors_are_refused():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: binding.gated_linear(x, x, x), lambda: binding.gated_linear_backward(x, x, x, x, x, x),
                 lambda: binding.quantize_int8(x), lambda: binding.gemm_int8(q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# --------------------------------------------------------------- workspaces
def workspace(lib, name, *sizes):
    n = ctypes.c_uint64(123)
    rc = getattr(lib, name)(*sizes, ctypes.byref(n))
    return rc, n.value


def test_backward_workspace(lib):
    name = "bwgemm_gated_backward_workspace"
    assert lib.bwgemm_gated_backward_workspace(1, 1, None) == INVALID
    assert workspace(lib, name, 0, 5) == workspace(lib, name, 5, 0) == (0, 0)
    assert workspace(lib, name, -1, 5)[0] == workspace(lib, name, 5, -1)[0] == INVALID
    assert workspace(lib, name, 1 << 31, 5)[0] == workspace(lib, name, (1 << 31) - 256, (1 << 31) - 256)[0] == UNSUP
    for M, N in ((1, 1), (3, 1001), (4096, 28672)):  # dG and dU, rows padded to 8
        rc, n = workspace(lib, name, M, N)
        need = 2 * M * (-(-N // 8) * 8) * 2
        assert rc == 0 and need <= n < need + 512 and n % 512 == 0


def test_integer_workspace(lib):
    name = "bwgemm_run_integer_workspace"
    assert lib.bwgemm_run_integer_workspace(1, 1, 1, None) == INVALID
    for sizes in ((0, 5, 5), (50, 0, 5), (50, 5, 0), (1, 8192, 8192), (16, 28672, 8192), (32, 8000, 8000), (8, 16, 1 << 20)):
        assert workspace(lib, name, *sizes) == (0, 0)
    assert workspace(lib, name, 5, 5, -1)[0] == INVALID
    assert workspace(lib, name, 1 << 31, 5, 5)[0] == workspace(lib, name, (1 << 31) - 256, 1, (1 << 31) - 256)[0] == UNSUP
    # A as fp16, or B where it has far fewer rows, but more than 32; rows padded to 128
    for M, N, K in ((33, 5, 5), (17, 28672, 8192), (4096, 1, 129), (4096, 33, 129), (300, 300, 300), (300, 299, 300)):
        rc, n = workspace(lib, name, M, N, K)
        need = (33 if N == 33 else M) * (-(-K // 128) * 128) * 2
        assert rc == 0 and need <= n < need + 256


def test_few_rows_of_integers_whose_sums_fit():
    # 32-bit sums of products of up to 2^14
    assert binding.select_int8(SMS, 8, 16, 131071)["lanes"] == 2 and binding.select_int8(SMS, 8, 16, 131072)["lanes"] == 1


# ------------------------------------------------------------ division of the work
def cdiv(a, b):
    return -(-a // b)


def sizes(rng, low, high):
    return max(low, min(high, round(2 ** rng.uniform(0, 15))))


@pytest.mark.parametrize("opts", [{}, {"max_ctas": 1}, {"max_ctas": 7}, {"workspace_bytes": 1 << 21}])
def test_every_plan_covers_its_product_in_bounds(opts):
    rng = random.Random(str(opts))
    room = (opts.get("workspace_bytes", 64 << 20) - (1 << 20)) // 4
    cap = opts.get("max_ctas", SMS)
    for _ in range(1500):
        M, N, K = sizes(rng, 1, 8192), sizes(rng, 1, 28672), sizes(rng, 1, 28672)
        for select, most, widths in ((binding.select_gated, 64, (16, 32, 64, 128)), (binding.select_int8, 128, (16, 32, 64, 128, 256))):
            s = select(SMS, M, N, K, max_pairs=76, **opts)
            if s["lanes"] == 2:
                assert M <= s["tile_x"] in (8, 16) and s["dp_tiles"] == s["workers"] == 0
                continue
            if s["lanes"] == 0:
                assert select is binding.select_gated and s["tile_x"] == 256 and s["tile_w"] == 128
                assert s["dp_tiles"] == cdiv(M, 256) * cdiv(N, 128) and s["sk_tiles"] == 0
                assert 1 <= s["workers"] <= min(s["dp_tiles"], cap // 2)
                continue
            ctas = 2 if s["tile_x"] == 256 else 1
            assert s["tile_x"] in widths and s["tile_w"] % 8 == 0 and 8 <= s["tile_w"] <= most * ctas
            rows, cols = (M, N) if s["lanes"] == 3 else (N, M)
            assert s["lanes"] == 1 or (s["lanes"] == 3 and select is binding.select_int8 and M > N > 32)
            tiles = cdiv(rows, s["tile_w"]) * cdiv(cols, s["tile_x"])
            assert s["dp_tiles"] + s["sk_tiles"] == tiles
            assert 1 <= s["workers"] <= (min(76, cap // 2) if ctas == 2 else cap)
            if s["sk_tiles"]:
                steps = s["sk_tiles"] * cdiv(K, 128)
                assert s["sk_tiles"] < s["workers"] or s["dp_tiles"] == 0
                assert s["workers"] <= steps  # every worker has a step
                # a worker's two partial tiles, and its counters
                assert s["workers"] * 2 * ctas * s["tile_x"] * 128 * (2 if select is binding.select_gated else 1) <= room
                assert s["sk_tiles"] * ctas * 8 * 4 <= 1 << 20
            else:
                assert s["workers"] <= tiles


@pytest.mark.parametrize("opts", [{}, {"max_ctas": 1}, {"max_ctas": 7}, {"workspace_bytes": 1 << 21}])
def test_every_backward_plan_covers_its_products(opts):
    rng = random.Random(str(opts) + "b")
    room = opts.get("workspace_bytes", 64 << 20) - (1 << 20)
    cap = opts.get("max_ctas", SMS)
    for _ in range(1500):
        M, N, K = sizes(rng, 1, 8192), sizes(rng, 1, 28672), sizes(rng, 1, 8192)
        x, w = binding.select_gated_backward(SMS, M, N, K, max_pairs=76, **opts)
        t = x["tile"]
        assert t in (128, 256) and w["tile"] == t and x["workers"] == w["workers"]
        assert x["tiles"] == cdiv(M, t) * cdiv(K, t) and w["tiles"] == 2 * cdiv(N, t) * cdiv(K, t)
        assert 1 <= x["workers"] <= (cap if t == 128 else min(76, cap // 2))
        # every slice has a step of K, and the slices' sums their room
        assert x["splits"] <= 2 * cdiv(N, 128) and w["splits"] <= cdiv(M, 128)
        units = (x["tiles"] * x["splits"] if x["splits"] > 1 or w["splits"] > 1 else 0) + (w["tiles"] * w["splits"] if w["splits"] > 1 else 0)
        assert units * t * t * 4 <= room


def test_select_refusals(lib):
    s, o = binding.LanesConfig(), (binding.OrthoConfig * 2)()
    for name, out in (("gated", ctypes.byref(s)), ("integer", ctypes.byref(s)), ("gated_backward", o)):
        f = getattr(lib, f"bwgemm_select_{name}")
        ok = [SMS, 0, 64, 128, 256, None]
        assert f(*ok, out) == 0 and f(*ok, None) == INVALID
        for i, v in ((0, 0), (1, -1), (2, 0), (3, 0), (4, -1)):
            assert f(*ok[:i], v, *ok[i + 1:], out) == INVALID
        assert f(SMS, 0, 64, 1 << 31, 256, None, out) == UNSUP


def test_all_forms_are_taken_by_some_size():
    seen = set()
    for M in (1, 9, 20, 40, 100, 300, 1000, 8192):
        for N in (64, 1000, 8192, 28672):
            for K in (64, 1000, 8192, 28672):
                for name, select in (("gated", binding.select_gated), ("int8", binding.select_int8)):
                    s = select(SMS, M, N, K, max_pairs=76)
                    seen.add((name, s["lanes"], s["tile_x"], s["sk_tiles"] > 0))
    for x in (16, 32, 64, 128):
        assert ("int8", 1, x, False) in seen or x == 128
        assert ("int8", 1, x, True) in seen
        assert ("gated", 1, x, False) in seen or ("gated", 1, x, True) in seen
    assert {("int8", 1, 256, False), ("int8", 1, 256, True), ("gated", 0, 256, False), ("int8", 2, 8, False),
            ("int8", 2, 16, False), ("gated", 2, 8, False), ("gated", 2, 16, False)} <= seen


# ----------------------------------------------------- what the calls hand on
class Recorder:
    """The library's calls: their arguments are kept, nothing runs."""

    def __init__(self):
        self.calls = []

    def _keep(self, names, args):
        self.calls.append(dict(zip(names.split(), args, strict=True)))
        return 0

    def bwgemm_gated(self, *args):
        return self._keep("plan X Wg Wu H G U M N K dtype activation stream", args)

    def bwgemm_gated_backward(self, *args):
        return self._keep("plan dH G U X Wg Wu dX dWg dWu M N K dtype activation workspace workspace_bytes stream", args)

    def bwgemm_quantize_integer(self, *args):
        return self._keep("plan X dtype rows cols ldx q ldq scales stream", args)

    def bwgemm_run_integer(self, *args):
        return self._keep("plan A sa B sb C M N K lda ldb ldc out workspace workspace_bytes stream", args)


@pytest.fixture
def plan(monkeypatch):
    binding._torch()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    p = binding.Plan.__new__(binding.Plan)
    p.lib, p.handle, p.device = Recorder(), ctypes.c_void_p(), -1  # -1: get_device() of a host tensor
    yield p
    p.handle = None


def matrix(record):
    m = binding.Matrix.from_buffer_copy(record)
    return m.data, m.ld


def z(*shape, dtype=torch.bfloat16, wide=None):
    t = torch.zeros(shape[0], wide or shape[1], dtype=dtype)
    return t[:, :shape[1]]


def test_gated_describes_its_matrices(plan):
    x, wg, wu = z(5, 20, wide=24), z(9, 20, wide=32), z(18, 24)[9:, 4:]  # (the last off 16 bytes: the library's to refuse)
    h, g, u = plan.gated_linear(x, wg, wu, "gelu", keep=True)
    call, = plan.lib.calls
    assert [matrix(call[k]) for k in ("X", "Wg", "Wu")] == [(x.data_ptr(), 24), (wg.data_ptr(), 32), (wu.data_ptr(), 24)]
    assert [matrix(call[k]) for k in "HGU"] == [(t.data_ptr(), 16) for t in (h, g, u)]
    assert all(t.shape == (5, 9) and t.stride() == (16, 1) for t in (h, g, u))
    assert [call[k] for k in ("M", "N", "K", "dtype", "activation")] == [5, 9, 20, binding.BF16, binding.GELU]
    plan.gated_linear(x.half(), wg.half(), wu.half())
    call = plan.lib.calls[-1]
    assert call["G"] is call["U"] is None and call["dtype"] == binding.FP16 and call["activation"] == binding.SILU


def test_single_rows_have_no_next_one(plan):
    row = z(1, 20, wide=4).as_strided((1, 4), (1, 1))
    plan.gated_linear(row, z(1, 4, wide=9), z(3, 8, wide=24)[1:2, :4])
    call, = plan.lib.calls
    assert [matrix(call[k])[1] for k in ("X", "Wg", "Wu", "H")] == [8, 8, 8, 8]


@pytest.mark.parametrize("make", [lambda: torch.zeros(1, 16, dtype=torch.bfloat16).expand(8, 16),
                                  lambda: torch.zeros(200, dtype=torch.bfloat16).as_strided((8, 16), (8, 1))])
def test_rows_closer_than_their_length_reach_the_library_as_they_are(plan, make):
    # which refuses them
    t, d = make(), z(8, 16)
    plan.gated_linear(t, d, d)
    plan.gated_linear(d, d, t)
    a, b = plan.lib.calls
    assert matrix(a["X"])[1] == t.stride(0) < 16 and matrix(b["Wu"])[1] == t.stride(0)


def test_gated_refusals_before_the_library(plan):
    x, w = z(4, 16), z(8, 16)
    for bad in ((x, w, z(8, 24)), (x, w, z(7, 16)), (x, z(8, 24), w), (x[0], w, w), (x, w[0], w), (x, w, z(16, 8).t()),
                (z(16, 4).t(), w, w)):
        with pytest.raises(ValueError):
            plan.gated_linear(*bad)
    for bad in ((x, w.half(), w), (x, w, w.float()), (x.float(), w.float(), w.float())):
        with pytest.raises(TypeError):
            plan.gated_linear(*bad)
    with pytest.raises(ValueError, match="activation"):
        plan.gated_linear(x, w, w, "relu")
    h = z(4, 8)
    for bad in ((z(4, 9), h, h, x, w, w), (h, z(3, 8), h, x, w, w), (h, h, z(4, 9), x, w, w), (h, h, h, z(5, 16), w, w),
                (h, h, h, x, z(9, 16), w), (h, h, h, x, w, z(8, 17))):
        with pytest.raises(ValueError):
            plan.gated_linear_backward(*bad)
    with pytest.raises(TypeError):
        plan.gated_linear_backward(h, h, h.half(), x, w, w)
    with pytest.raises(ValueError, match="activation"):
        plan.gated_linear_backward(h, h, h, x, w, w, "tanh")
    assert plan.lib.calls == []


def test_backward_describes_what_is_wanted(plan):
    h, x, w = z(4, 9, wide=16), z(4, 20, wide=24), z(9, 20, wide=24)
    dx, dwg, dwu = plan.gated_linear_backward(h, h, h, x, w, w, "gelu_tanh")
    assert plan.gated_linear_backward(h, h, h, None, w, w, weight_grads=False)[1:] == (None, None)
    assert plan.gated_linear_backward(h, h, h, x, None, None, input_grad=False)[0] is None
    assert plan.gated_linear_backward(h, h, h, None, None, None, input_grad=False, weight_grads=False) == (None, None, None)
    both, only_x, only_w = plan.lib.calls
    assert [matrix(both[k]) for k in ("dX", "dWg", "dWu")] == [(t.data_ptr(), 24) for t in (dx, dwg, dwu)]
    assert dx.shape == (4, 20) and dwg.shape == dwu.shape == (9, 20) and both["activation"] == binding.GELU_TANH
    assert [both[k] for k in "MNK"] == [4, 9, 20] and both["workspace_bytes"] == 512
    assert only_x["X"] is only_x["dWg"] is only_x["dWu"] is None and only_x["Wg"] is not None
    assert only_w["Wg"] is only_w["Wu"] is only_w["dX"] is None and only_w["X"] is not None and only_w["K"] == 20


def test_integers_describe_their_operands(plan):
    x = z(3, 20, dtype=torch.float32, wide=32)
    q, s = plan.quantize_int8(x)
    call, = plan.lib.calls
    assert [call[k] for k in ("X", "dtype", "rows", "cols", "ldx", "q", "ldq", "scales")] == [
        x.data_ptr(), binding.FP32, 3, 20, 32, q.data_ptr(), 32, s.data_ptr()]
    assert q.shape == (3, 20) and q.stride() == (32, 1) and q.dtype == torch.int8 and s.shape == (3,)
    b, sb = z(40, 20, dtype=torch.int8, wide=48), torch.zeros(40)
    c = plan.gemm_int8(q, s, b, sb, out_dtype=torch.float16)
    call = plan.lib.calls[-1]
    assert [call[k] for k in ("A", "sa", "B", "sb", "C", "M", "N", "K", "lda", "ldb", "ldc", "out", "workspace", "workspace_bytes")] == [
        q.data_ptr(), s.data_ptr(), b.data_ptr(), sb.data_ptr(), c.data_ptr(), 3, 40, 20, 32, 48, 40, binding.FP16, None, 0]
    out = z(37, 61, dtype=torch.float32, wide=80)
    assert plan.gemm_int8(z(37, 20, dtype=torch.int8, wide=32), torch.zeros(37), z(61, 20, dtype=torch.int8, wide=32),
                          torch.zeros(61), out=out) is out
    call = plan.lib.calls[-1]
    assert call["ldc"] == 80 and call["out"] == binding.FP32 and call["workspace_bytes"] == 37 * 128 * 2
    assert call["workspace"] is not None
    q0, s0 = plan.quantize_int8(z(3, 0))  # rows without a value: as rows of zeros
    assert q0.shape == (3, 0) and (s0 == torch.tensor(2.0 ** -100 / 127)).all()


def test_integer_refusals_before_the_library(plan):
    a, s = z(4, 16, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(TypeError):
        plan.quantize_int8(a)
    for bad in (z(4, 16)[0], z(16, 4).t(), z(4, 32)[:, ::2]):
        with pytest.raises(ValueError):
            plan.quantize_int8(bad)
    for bad in ((z(4, 16, dtype=torch.uint8), s, a, s), (a, s.double(), a, s), (a, s, a, s.half())):
        with pytest.raises(TypeError):
            plan.gemm_int8(*bad)
    for bad in ((a, torch.zeros(5), a, s), (a, s[:, None], a, s), (a, s, z(4, 17, dtype=torch.int8), s), (a[0], s, a, s),
                (a, torch.zeros(8)[::2], a, s), (z(16, 4, dtype=torch.int8).t(), s, a, s)):
        with pytest.raises(ValueError):
            plan.gemm_int8(*bad)
    with pytest.raises(TypeError):
        plan.gemm_int8(a, s, a, s, out_dtype=torch.int32)
    for out in (z(4, 5), z(4, 4, dtype=torch.float32).double().float().t().expand(4, 4)[:, :3], torch.zeros(4, 8)[:, ::2]):
        with pytest.raises(ValueError):
            plan.gemm_int8(a, s, a, s, out=out)
    with pytest.raises(ValueError):
        plan.gemm_int8(a, s, a, s, out=z(4, 4), out_dtype=torch.float32)
    assert plan.lib.calls == []


# -------------------------------------------------------------- default plans
class Handle:
    """A CUDA tensor as far as the choice of a plan goes."""

    def get_device(self):
        return 0


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


CALLS = [lambda stream: binding.gated_linear(Handle(), None, None, stream=stream),
         lambda stream: binding.gated_linear_backward(Handle(), None, None, None, None, None, stream=stream),
         lambda stream: binding.quantize_int8(Handle(), stream=stream),
         lambda stream: binding.gemm_int8(Handle(), None, None, None, stream=stream)]


@pytest.fixture
def plans(monkeypatch):
    made = []

    class Made:
        def __init__(self, device):
            made.append(self)

        def gated_linear(self, *args, **kw):
            return self

        gated_linear_backward = quantize_int8 = gemm_int8 = gated_linear

    monkeypatch.setattr(binding, "Plan", Made)
    monkeypatch.setattr(binding, "_plans", {})
    binding._torch()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 7, raising=False)
    return made


@pytest.mark.parametrize("call", CALLS)
def test_default_plans_are_of_one_stream_and_one_thread(plans, call):
    here = call(None)
    assert call(None) is here and call(Stream(7)) is here and call(Stream(8)) is not here
    other = []
    t = threading.Thread(target=lambda: other.append(call(None)))
    t.start()
    t.join(30)
    assert other[0] is not here and len(plans) == 3


def test_the_calls_share_a_default_plan(plans):
    assert len({id(call(None)) for call in CALLS}) == 1


# ------------------------------------------------------------------- autograd
class Plain:
    """The two operators of the gated layer in 64 bits; what they are asked for is kept."""

    def __init__(self):
        self.asked = []

    @staticmethod
    def _rows(*ts):
        for t in ts:
            if t is not None:
                assert t.shape[1] <= 1 or t.stride(1) == 1
                assert t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) * t.element_size() % 16 == 0), "refused"
                assert t.data_ptr() % 16 == 0

    def gated_linear(self, x, wg, wu, activation, keep=False):
        self._rows(x, wg, wu)
        self.asked.append(keep)
        g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
        h = (torch.nn.functional.silu(g) * u).to(x.dtype)
        wide = [torch.zeros(len(g), -(-g.shape[1] // 8) * 8, dtype=torch.float64) for _ in range(2)]
        for w, v in zip(wide, (g, u)):
            w[:, :g.shape[1]] = v
        return (h, *(w[:, :g.shape[1]] for w in wide)) if keep else h

    def gated_linear_backward(self, dh, g, u, x, wg, wu, activation, input_grad, weight_grads):
        self._rows(dh, g, u, x, wg, wu)
        self.asked.append((input_grad, weight_grads))
        s = torch.sigmoid(g)
        dg, du = dh.double() * u * (s + g * s * (1 - s)), dh.double() * g * s
        dx = (dg @ wg.double() + du @ wu.double()).to(x.dtype) if input_grad else None
        return (dx, *((d.t() @ x.double()).to(x.dtype) if weight_grads else None for d in (dg, du)))


@pytest.fixture
def plain(monkeypatch):
    from dense_gemm_blackwell_03_gb300 import linear_training
    p = Plain()
    monkeypatch.setattr(linear_training, "binding", p)
    return p


def leaves(tokens, inner, hidden):
    gen = torch.Generator().manual_seed(tokens)
    return [torch.randn(*s, generator=gen).requires_grad_() for s in ((tokens, inner), (hidden, inner), (hidden, inner))]


@pytest.mark.parametrize("loss", [lambda y: (y.sum(0) * torch.arange(y.shape[1])).sum(), lambda y: y.sum(1).square().sum(),
                                  lambda y: y.sum(), lambda y: (y.t() @ torch.ones(y.shape[0], 3, dtype=y.dtype)).square().sum(),
                                  lambda y: torch.cat([y, y], 1)[:, 1:].square().sum()])
@pytest.mark.parametrize("sizes", [(12, 16, 24), (7, 9, 13), (1, 16, 5), (6, 8, 1)])
def test_gradients_of_any_layout(plain, loss, sizes):
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear
    ts = leaves(*sizes)
    loss(gated_linear(*ts)).backward()
    ref = [t.detach().double().requires_grad_() for t in ts]
    loss(torch.nn.functional.silu(ref[0] @ ref[1].t()) * (ref[0] @ ref[2].t())).backward()
    for got, want in zip(ts, ref):
        assert (got.grad - want.grad).abs().max() <= 1e-4 * want.grad.abs().max() + 1e-30


@pytest.mark.parametrize("wanted", [(1, 1, 1), (1, 0, 0), (0, 1, 1), (0, 1, 0), (0, 0, 1), (0, 0, 0)])
def test_only_what_gradients_read(plain, wanted):
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear
    ts = leaves(12, 16, 24)
    for t, of in zip(ts, wanted):
        t.requires_grad_(bool(of))
    y = gated_linear(*ts)
    assert plain.asked == [any(wanted)]
    if any(wanted):
        y.sum().backward()
        assert plain.asked[1:] == [(bool(wanted[0]), bool(wanted[1] or wanted[2]))]
    assert [t.grad is not None for t in ts] == [bool(of) for of in wanted]
    with torch.no_grad():
        assert not gated_linear(*leaves(12, 16, 24)).requires_grad and plain.asked[-1] is False


def test_a_second_derivative_raises(plain):
    from dense_gemm_blackwell_03_gb300.linear_training import gated_linear
    ts = leaves(12, 16, 24)
    gx, = torch.autograd.grad((gated_linear(*ts) ** 3).sum(), ts[0], create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        gx.square().sum().backward()
