"""Every kernel that the launchers of the grouped products can pick is reached by a GPU test, and every choice is one
that exists: csrc/tiles.h built for the CPU, asked with the sizes of those tests."""
import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_block_sums as B
from tests import test_gpu_grouped as G
from tests import test_gpu_grouped_tiles as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORWARD, DGRAD, WGRAD, BLOCK = range(4)
FEW_ROWS = -1


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the HIP headers")
    so = str(tmp_path_factory.mktemp("tiles") / "tile_choice.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "quantized_moe_expert_topk_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host", "tile_choice.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def bf16_shapes():
    """(E, M, rows, N, K) of the parametrised product tests."""
    for (name, counts), (N, K) in itertools.product(G.COUNTS.items(), G.SIZES):
        if not (name.startswith("mean") and (N, K) not in ((264, 200), (520, 1032), (1024, 512))):  # (skipped there)
            yield len(counts), sum(counts), sum(counts), N, K
    for counts, N, K in L.CASES.values():
        yield len(counts), sum(counts) + 3 * len(counts) + 5, sum(counts), N, K


def fp8_shapes():
    """(grouped, E, M, rows, N, K)."""
    for M, N, K in B.DENSE:
        yield 0, 1, M, M, N, K
    for counts, (N, K) in itertools.product(B.GROUPS.values(), [(144, 272), (1040, 2048)]):
        yield 1, len(counts), sum(counts), sum(counts), N, K


@pytest.mark.parametrize("prod", [FORWARD, DGRAD, WGRAD])
def test_every_bf16_tile_is_tested(tiles, prod):
    reached = {tiles.choose(prod, 1, *s) for s in bf16_shapes()}
    want = set(range(tiles.tile_count(prod))) | ({FEW_ROWS} if prod == FORWARD else set())
    assert reached == want, f"not reached: {want - reached}"


def test_every_fp8_tile_is_tested_dense_and_grouped(tiles):
    want = set(range(tiles.tile_count(BLOCK))) | {FEW_ROWS}
    for grouped in (0, 1):
        reached = {tiles.choose(BLOCK, *s) for s in fp8_shapes() if s[0] == grouped}
        assert reached == want, f"grouped {grouped}, not reached: {want - reached}"


@pytest.mark.parametrize("case,prod,p", [("large", FORWARD, 2008), ("large", DGRAD, 2056), ("two stages", FORWARD, 4104),
                                         ("two stages, dgrad", DGRAD, 4104), ("one stage", FORWARD, 4104),
                                         ("one stage, dgrad", DGRAD, 4104), ("whole lines", FORWARD, 2048),
                                         ("whole lines", DGRAD, 4160), ("many stages", FORWARD, 2056),
                                         ("many stages", DGRAD, 4104)])
def test_the_large_cases_take_256_x_256(tiles, case, prod, p):
    counts, N, K = L.CASES[case]
    assert (N if prod == FORWARD else K) == p
    t = tiles.choose(prod, 1, len(counts), sum(counts) + 3 * len(counts) + 5, sum(counts), N, K)
    assert tiles.tile_outputs(prod, t) == 256256


def test_choices_exist_over_the_whole_range(tiles):
    """No size, however large, makes the choice overflow into a tile that is not there."""
    sizes = [8, 64, 264, 4096, 2097136]
    for E, M, N, K in itertools.product([1, 7, 60, 1024], [1, 16, 333, 70000, 0x7FFFFC00], sizes, sizes):
        for rows in {1, min(M, 100), M}:
            for prod in (FORWARD, DGRAD, WGRAD, BLOCK):
                for grouped in ((1,) if prod != BLOCK else (0, 1)):
                    t = tiles.choose(prod, grouped, E if grouped else 1, M, rows, N, K)
                    assert (-1 if prod in (FORWARD, BLOCK) else 0) <= t < tiles.tile_count(prod)


def test_only_whole_lines_are_written_through(tiles):
    """Large outputs whose rows begin and end with a 128-byte line; a view 16 bytes further does neither."""
    through = lambda out, nbytes, pitch: tiles.through(ctypes.c_uint64(out), ctypes.c_double(nbytes), ctypes.c_longlong(pitch))
    assert through(1 << 40, 1e8, 4096) == 1
    assert through((1 << 40) + 128, 1e8, 128) == 1
    for off in (16, 32, 64, 112):
        assert through((1 << 40) + off, 1e8, 4096) == 0
    assert through(1 << 40, 1e8, 4096 + 64) == 0
    assert through(1 << 40, 1e6, 4096) == 0
