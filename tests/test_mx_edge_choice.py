"""The sizes and hints of tests/test_gpu_mx_edges.py reach every kernel of the MXFP4 products (csrc/tiles.h on the CPU), so that a
change of the rule cannot take the edges away from one of them unseen."""
import pytest

from tests import test_gpu_mx_edges as L
from tests.test_mx_tile_choice import FEW_ROWS, tiles  # noqa: F401


def choice(tiles, name, tile16):  # noqa: F811
    rows, N, K = L.EDGES[name]
    if isinstance(rows, int):
        return tiles.mx_choose(0, 1, rows, rows, N, K, tile16)
    return tiles.mx_choose(1, len(rows), sum(rows) + 3 * len(rows) + 5, sum(rows), N, K, tile16)


@pytest.mark.parametrize("tile16", [0, 1])
def test_edges_reach_every_kernel(tiles, tile16):  # noqa: F811
    every = {FEW_ROWS, *range(tiles.mx_tile_count())}
    by = {n: choice(tiles, n, tile16) for n in L.EDGES}
    assert set(by.values()) == every, by
    # weights are non-temporal for experts only
    assert {t for n, t in by.items() if "dense" in n} == every - {tiles.mx_tile_count() - 1}, by


@pytest.mark.parametrize("tile16", [0, 1])
def test_hints_reach_every_kernel(tiles, tile16):  # noqa: F811
    by = {h: tiles.mx_choose(1, 6, L.RANGES_M, h, L.RANGES_N, L.RANGES_K, tile16) for h in L.HINTS}
    assert set(by.values()) == {FEW_ROWS, *range(tiles.mx_tile_count())}, by
