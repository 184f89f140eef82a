"""The dense MXFP4 products' choice between the kernel for few rows and the tiles (csrc/tiles.h on the CPU), at sizes where the
two were measured to be far apart."""
import itertools

import pytest

from tests.test_mx_tile_choice import FEW_ROWS, choice, tiles  # noqa: F401

# M, N, K; 2 to 6 times the time on the kernel for few rows (960 x 960 x 128: one of its 3600 tiles after the other, most of its
# waves without columns)
SHORT = [(960, 960, 128), (8192, 112, 128), (512, 1600, 128), (2000, 1800, 32), (500, 1024, 128), (64, 8192, 128), (40, 8192, 256),
         (64, 4096, 256), (2000, 112, 256), (64, 4096, 512), (350, 2500, 96), (3000, 200, 96)]
# a fifth to a half faster on the kernel for few rows: few rows by wide weights, and long contractions of little else
FEW = [(1, 8192, 4096), (1, 8192, 8192), (1, 8192, 14336), (16, 8192, 4096), (16, 4096, 14336), (64, 112, 14336), (256, 512, 2048)]


@pytest.mark.parametrize("tile16", [0, 1])
@pytest.mark.parametrize("size", SHORT, ids=str)
def test_short_contractions_take_tiles(tiles, size, tile16):  # noqa: F811
    assert choice(tiles, size, tile16) != FEW_ROWS


@pytest.mark.parametrize("tile16", [0, 1])
@pytest.mark.parametrize("size", FEW, ids=str)
def test_few_rows(tiles, size, tile16):  # noqa: F811
    assert choice(tiles, size, tile16) == FEW_ROWS


def test_many_tiles_of_a_short_contraction(tiles):  # noqa: F811
    """600 tiles of 16 x 16 take longer than a few stages of the larger ones, whatever their shape."""
    for M, N, K in itertools.product([1, 16, 90, 600, 5000, 100000], [16, 112, 1024, 8192, 65536], [32, 96, 256, 512]):
        if -(-M // 16) * -(-N // 16) >= 600:
            assert choice(tiles, (M, N, K), 0) != FEW_ROWS, (M, N, K)

@pytest.mark.parametrize("size,want", [((64, 4096, 4096), 0), ((64, 4096, 4352), 1), ((64, 4096, 14336), 1), ((256, 4096, 4096), 0),
                                       ((256, 4096, 7168), 1)], ids=str)
def test_long_contractions_take_the_larger_tile(tiles, size, want):  # noqa: F811
    assert choice(tiles, size, 0) == want
