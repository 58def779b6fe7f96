"""How the operators divide their work, asked on the host (no GPU): the
structs' layout, refusals, and that every plan covers its product in bounds."""
from __future__ import annotations

import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest

from dense_gemm_blackwell_03_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUP = 1, 3
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def lib():
    return binding.load_library(build_if_missing=True)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_config_layouts(tmp_path):
    fields = [(name, f) for name, s in (("bwgemm_scaled_config_t", binding.ScaledConfig),
                                        ("bwgemm_ortho_config_t", binding.OrthoConfig)) for f, _ in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bwgemm.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", offsetof({s}, {f}));\n' for s, f in fields)
                   + '  printf("%zu %zu\\n", sizeof(bwgemm_scaled_config_t), sizeof(bwgemm_ortho_config_t));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    mine = [getattr(s, f).offset for s in (binding.ScaledConfig, binding.OrthoConfig) for f, _ in s._fields_]
    assert got == mine + [ctypes.sizeof(binding.ScaledConfig), ctypes.sizeof(binding.OrthoConfig)]


def test_refusals(lib):
    s, o = binding.ScaledConfig(), (binding.OrthoConfig * 3)()
    ok = [SMS, 64, 128, 256, 0, None]
    assert lib.bwgemm_select_scaled(*ok, ctypes.byref(s)) == 0 and lib.bwgemm_select_scaled(*ok, None) == INVALID
    for i, v in ((0, 0), (1, 0), (2, -1), (3, 0), (4, 2)):
        assert lib.bwgemm_select_scaled(*ok[:i], v, *ok[i + 1:], ctypes.byref(s)) == INVALID
    assert lib.bwgemm_select_scaled(SMS, 64, 1 << 31, 256, 0, None, ctypes.byref(s)) == UNSUP
    ok = [SMS, 0, 1, 64, 128, 0, 0, None]
    assert lib.bwgemm_select_orthogonalize(*ok, o) == 0 and lib.bwgemm_select_orthogonalize(*ok, None) == INVALID
    for i, v in ((0, 0), (1, -1), (2, 0), (3, 0), (4, -1), (5, 3), (6, -1), (6, 64)):
        assert lib.bwgemm_select_orthogonalize(*ok[:i], v, *ok[i + 1:], o) == INVALID
    assert lib.bwgemm_select_orthogonalize(SMS, 0, 1 << 16, 64, 128, 0, 0, None, o) == UNSUP


def cdiv(a, b):
    return -(-a // b)


def sizes(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


@pytest.mark.parametrize("workspace", [0, (1 << 20) + 4096, 8 << 20])
def test_scaled_plans_cover_their_product(workspace):
    rng = random.Random(workspace)
    for _ in range(3000):
        M, N, K = sizes(rng, 1, 20000), sizes(rng, 1, 60000), sizes(rng, 1, 60000)
        blocks = rng.choice(["row", "square"])
        c = binding.select_scaled(SMS, M, N, K, blocks, workspace_bytes=workspace)
        if c["few_rows"]:
            assert M <= 16
            continue
        lane, other = (N, M) if c["swap_ab"] else (M, N)
        assert c["dp_tiles"] + c["sk_tiles"] == cdiv(lane, c["tile_l"]) * cdiv(other, c["tile_c"])
        assert 1 <= c["workers"] <= SMS and c["column_scales"] == (c["swap_ab"] or blocks == "row")
        assert c["tile_l"] == 128 if not c["swap_ab"] else (c["tile_l"] % 8 == 0 and 8 <= c["tile_l"] <= 128)
        if c["sk_tiles"]:
            room = (workspace or 64 << 20) - (1 << 20)
            assert c["workers"] * 2 * 128 * c["tile_c"] * 4 <= room and c["sk_tiles"] * 8 * 4 <= 1 << 20


@pytest.mark.parametrize("workspace", [0, (1 << 20) + 4096])
def test_ortho_plans_cover_their_products(workspace):
    rng = random.Random(workspace)
    for _ in range(1000):
        batch, rows, cols = rng.choice([1, 1, 2, 7, 32, 300]), sizes(rng, 1, 6000), sizes(rng, 1, 30000)
        step, dtype = rng.randrange(5), rng.choice([binding.BF16, binding.FP32])
        products = binding.select_orthogonalize(SMS, batch, rows, cols, dtype, step, workspace_bytes=workspace)
        m = min(rows, cols)
        for which, c in enumerate(products):
            t = c["tile"]
            assert t in (128, 256) and 1 <= c["workers"] <= SMS * 128 // t
            r = cdiv(m if which < 2 else rows, t), cdiv(m if which < 2 else cols, t)
            assert c["tiles"] == batch * (r[0] * (r[0] + 1) // 2 if which < 2 else r[0] * r[1])
            assert c["splits"] == 1 or which == 0
            if c["splits"] > 1:
                assert c["tiles"] * c["splits"] * t * t * 4 <= (workspace or 64 << 20) - (1 << 20)
                assert c["tiles"] <= 65535  # of the joining kernel's grid


# a size of every compiled form of the scaled product, small ones
FORMS = {(256, 0, 0): (7348, 389, 200, "square"), (256, 0, 1): (7431, 394, 200, "row"), (128, 0, 0): (4913, 179, 200, "square"),
         (128, 0, 1): (5024, 184, 200, "row"), (64, 1, 1): (4987, 16, 200, "square"), (32, 1, 1): (17, 48, 200, "row"),
         (16, 1, 1): (9, 18939, 553, "row")}


def test_every_compiled_form_of_the_scaled_product_is_taken():
    source = open(os.path.join(ROOT, "dense_gemm_blackwell_03_gb300", "csrc", "operators.h")).read()
    table = re.search(r"kScaledVariants\[\] = \{(.*?)\};", source, re.S).group(1)
    compiled = {(int(bn), int(swap == "true"), int(col == "true"))
                for bn, swap, col in re.findall(r"\{(\d+), (true|false), (true|false)\}", table)}
    taken = set()
    for M, N, K, blocks in FORMS.values():
        c = binding.select_scaled(SMS, M, N, K, blocks)
        taken.add((c["tile_c"], c["swap_ab"], c["column_scales"]))
    assert taken == compiled == set(FORMS)


def test_more_tiles_than_a_launch_counts_are_unsupported(lib):
    c = binding.ScaledConfig()
    assert lib.bwgemm_select_scaled(SMS, (1 << 31) - 1, (1 << 31) - 1, 128, 0, None, ctypes.byref(c)) == UNSUP


@pytest.mark.parametrize("cap", [1, 2, 3, 40, 151, 1000])
def test_the_cap_on_the_persistent_grid_holds(cap):
    rng = random.Random(cap)
    for _ in range(300):
        M, N, K = sizes(rng, 17, 20000), sizes(rng, 64, 60000), sizes(rng, 128, 30000)
        c = binding.select_scaled(SMS, M, N, K, rng.choice(["row", "square"]), max_ctas=cap)
        assert 1 <= c["workers"] <= min(cap, SMS)
        for p in binding.select_orthogonalize(SMS, rng.choice([1, 20]), *rng.sample([64, 500, 1024, 4096, 9000], 2),
                                              step=rng.randrange(5), max_ctas=cap):
            assert 1 <= p["workers"] * p["tile"] // 128 <= min(cap, SMS)


@pytest.mark.parametrize("size", [(1 << 31) - 1, (1 << 31) - 100, (1 << 31) - 255])
def test_sizes_whose_last_tile_would_pass_32_bits_are_unsupported(lib, size):
    # the kernels count rows and columns of a tile, up to 256 past its first, in 32 bits
    c = binding.ScaledConfig()
    for sizes_ in ((1, size, 16), (size, 64, 16), (64, 64, size)):
        assert lib.bwgemm_select_scaled(SMS, *sizes_, 0, None, ctypes.byref(c)) == UNSUP
    for sizes_ in ((1, (1 << 31) - 256, 16), ((1 << 31) - 256, 64, 16), (64, 64, (1 << 31) - 256)):
        assert lib.bwgemm_select_scaled(SMS, *sizes_, 0, None, ctypes.byref(c)) == 0
