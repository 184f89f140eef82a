"""Every kernel that the launcher of the MXFP4 products can pick is reached by a GPU test, and every choice is one that exists:
csrc/tiles.h built for the CPU, asked with the sizes of tests/test_gpu_mx_tiles.py."""
import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_mx_tiles as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FEW_ROWS = -1


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the HIP headers")
    so = str(tmp_path_factory.mktemp("tiles") / "mx_tile_choice.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "quantized_moe_expert_topk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host", "mx_tile_choice.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def choice(tiles, case, tile16):
    rows, N, K = case
    if isinstance(rows, int):
        return tiles.mx_choose(0, 1, rows, rows, N, K, tile16)
    return tiles.mx_choose(1, len(rows), sum(rows) + 3 * len(rows) + 5, sum(rows), N, K, tile16)


@pytest.mark.parametrize("tile16", [0, 1])
def test_every_tile_is_tested(tiles, tile16):
    want = set(range(tiles.mx_tile_count())) | {FEW_ROWS}
    by = {n: choice(tiles, c, tile16) for n, c in L.CASES.items()}
    assert set(by.values()) == want, by
    nt = tiles.mx_tile_count() - 1  # non-temporal weights: for experts only
    assert {choice(tiles, c, tile16) for c in L.CASES.values() if isinstance(c[0], int)} == want - {nt}, by


def test_every_tile_is_tested_with_odd_rows(tiles):
    got = {n: choice(tiles, c, 0) for n, c in L.ODD.items()}
    assert set(got.values()) - {FEW_ROWS} == set(range(tiles.mx_tile_count())), got


@pytest.mark.parametrize("name,want", [("few rows", -1), ("few rows, dense", -1), ("32 rows", 0), ("32 rows, dense", 0),
                                       ("100 rows", 1), ("100 rows, dense", 1), ("100 rows, dense, one stage", 1),
                                       ("128 rows", 1), ("128 rows, dense", 1), ("128 rows, dense, one stage", 1),
                                       ("large", 2), ("large, dense", 2), ("large, one stage", 2), ("large, two stages", 2),
                                       ("large, dense, one stage", 2), ("large, whole lines", 2), ("many experts", 3),
                                       ("many experts, one stage", 3), ("many experts, whole stages", 3)])
def test_cases_take_the_tiles_they_are_named_by(tiles, name, want):
    assert choice(tiles, L.CASES[name], 1) == want


def test_choices_exist_over_the_whole_range(tiles):
    """No size, however large, makes the choice overflow into a tile that is not there."""
    sizes = [32, 64, 288, 4096, 2097120]
    for E, M, N, K in itertools.product([1, 7, 60, 1024], [1, 16, 333, 70000, 0x7FFFFC00], [1, *sizes], sizes):
        for rows in {1, min(M, 100), M}:
            for grouped, tile16 in itertools.product((0, 1), (0, 1)):
                t = tiles.mx_choose(grouped, E if grouped else 1, M, rows, N, K, tile16)
                assert FEW_ROWS <= t < tiles.mx_tile_count()


def test_whole_lines(tiles):
    whole = lambda out, pitch: tiles.whole(ctypes.c_uint64(out), ctypes.c_longlong(pitch))
    assert whole(1 << 40, 4096) == 1 and whole((1 << 40) + 128, 128) == 1
    assert whole((1 << 40) + 64, 4096) == 0 and whole(1 << 40, 1040) == 0
