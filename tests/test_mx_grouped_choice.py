"""The grouped MXFP4 products' choice between the kernel for few rows and the tiles (csrc/tiles.h on the CPU), in both orders of
the weights, at sizes where the two were measured to be far apart."""
import pytest

from tests.test_mx_tile_choice import FEW_ROWS, tiles  # noqa: F401


def choice(tiles, E, rows, N, K, tile16):  # noqa: F811
    return tiles.mx_choose(1, E, rows, rows, N, K, tile16)


# experts, rows, N, K: 1.4 to 2.4 times the time on the kernel for few rows, in the orders of the weights given
@pytest.mark.parametrize("size,orders", [((5, 100, 2048, 7168), (0, 1)), ((8, 100, 2048, 14336), (0, 1)), ((8, 256, 1024, 14336), (0, 1)),
                                         ((8, 600, 512, 14336), (0, 1)), ((2, 40, 4096, 7168), (0,)), ((5, 40, 4096, 14336), (0,))],
                         ids=str)
def test_many_rows_of_few_experts_take_tiles(tiles, size, orders):  # noqa: F811
    for tile16 in orders:
        assert choice(tiles, *size, tile16) != FEW_ROWS


@pytest.mark.parametrize("size", [(8, 8, 1024, 2048), (8, 8, 512, 4096), (8, 16, 512, 7168), (1, 1, 4096, 4096)], ids=str)
def test_few_rows(tiles, size):  # noqa: F811
    for tile16 in (0, 1):
        assert choice(tiles, *size, tile16) == FEW_ROWS
