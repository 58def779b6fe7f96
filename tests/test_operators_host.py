"""Host-only checks of the 8-bit and orthogonalisation entry points (no GPU):
struct layout, workspace sizes, argument checks that need no device."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from dense_gemm_blackwell_03_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUP = 1, 3


@pytest.fixture(scope="module")
def lib():
    return binding.load_library(build_if_missing=True)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_scaled_operand_layout_and_codes(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "bwgemm.h"\n'
        "int main(void) {\n"
        '  printf("%zu %zu %zu %zu %zu %zu %d %d %d %d %d\\n", sizeof(bwgemm_scaled_t), '
        "offsetof(bwgemm_scaled_t, ld), offsetof(bwgemm_scaled_t, scales), "
        "offsetof(bwgemm_scaled_t, ld_scales), offsetof(bwgemm_scaled_t, type), "
        "offsetof(bwgemm_scaled_t, block), BWGEMM_FP32, BWGEMM_E4M3, BWGEMM_E5M2, BWGEMM_BLOCK_ROW, "
        "BWGEMM_BLOCK_SQUARE);\n  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    s = binding.Scaled
    assert got == [ctypes.sizeof(s), s.ld.offset, s.scales.offset, s.ld_scales.offset, s.type.offset, s.block.offset,
                   binding.FP32, binding.E4M3, binding.E5M2, binding.BLOCK_ROW, binding.BLOCK_SQUARE]


def test_null_plans_are_refused(lib):
    assert lib.bwgemm_quantize(None, 0x1000, 0, 1, 128, 128, 0, 0, 0, 0x2000, 128, 0x3000, 1, None, 0, None, 0,
                               None) == INVALID
    s = binding.Scaled(0x1000, 128, 0x2000, 1, 0, 0)
    assert lib.bwgemm_run_scaled(None, ctypes.addressof(s), ctypes.addressof(s), 0x3000, 1, 1, 128, 8, 0, 0,
                                 None) == INVALID
    assert lib.bwgemm_orthogonalize(None, 0x1000, 0, 0x2000, 0, 1, 8, 8, 8, 64, 8, 64, 5, None, 1e-7, 1.0, 0x4000,
                                    1 << 20, None) == INVALID


def workspace(lib, batch, rows, cols):
    n = ctypes.c_uint64(123)
    rc = lib.bwgemm_orthogonalize_workspace(batch, rows, cols, ctypes.byref(n))
    return rc, n.value


def test_orthogonalize_workspace_sizes(lib):
    assert lib.bwgemm_orthogonalize_workspace(1, 8, 8, None) == INVALID
    for sizes in ((0, 8, 8), (1, 0, 8), (1, 8, 0)):
        assert workspace(lib, *sizes) == (0, 0)
    assert workspace(lib, -1, 8, 8)[0] == INVALID
    assert workspace(lib, 1 << 16, 8, 8)[0] == UNSUP
    assert workspace(lib, 1, 1 << 25, 8)[0] == UNSUP
    # four fp16 matrices of G's size (columns padded to 64), three of the short side's (S, B
    # and B's low part)
    for batch, rows, cols in ((1, 300, 1000), (3, 1000, 300), (2, 512, 512), (1, 1, 1)):
        pad = lambda v: -(-v // 64) * 64  # noqa: E731
        rc, n = workspace(lib, batch, rows, cols)
        m = min(rows, cols)
        need = batch * 2 * (4 * rows * pad(cols) + 3 * m * pad(m))
        assert rc == 0 and need <= n <= need + (1 << 20)
    # the two orientations hold the same matrices
    assert abs(workspace(lib, 1, 1024, 4096)[1] - workspace(lib, 1, 4096, 1024)[1]) < (1 << 20)


def test_package_exports_the_operators():
    import dense_gemm_blackwell_03_gb300 as pkg
    for name in ("quantize", "gemm_scaled", "orthogonalize"):
        assert name in pkg.__all__ and getattr(pkg, name) is getattr(binding, name)


def test_host_tensors_are_refused():
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q = torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(1, 4)
    for call in (lambda: binding.quantize(x), lambda: binding.gemm_scaled(q, s, q, s), lambda: binding.orthogonalize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
