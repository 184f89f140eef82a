"""The MXFP4 products at every tile that the launcher picks, in both orders of the weights (tests/test_mx_tile_choice.py checks
that these sizes reach them): ragged and empty experts, sizes off the tile, contractions of one, a few and many stages with
whole and partial last ones, more tiles than workgroups, rows of whole pieces and others, outputs past L2 of whole lines.

Tolerances as in tests/test_gpu_mx.py.
"""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import gen, ranges, rows_of
from tests.test_gpu_mx import ROWS, TILE16, check_product, decode, group, operand, weights

pytestmark = pytest.mark.gpu

DEV = "cuda"
BOTH = (torch.bfloat16, torch.float32)

# rows of each expert (an int: dense), N, K
CASES = {
    "few rows": ([3, 0, 1, 7], 1040, 2080),
    "few rows, one stage": ([9, 0, 20], 272, 96),
    "few rows, dense": (11, 1040, 4128),
    "32 rows": ([(5 * i) % 23 for i in range(64)], 1040, 2080),
    "32 rows, one stage": ([(5 * i) % 23 for i in range(64)], 1040, 160),
    "32 rows, dense": (200, 1040, 2080),
    "100 rows": ([70, 0, 61, 130, 1, 200], 2064, 2080),
    "100 rows, dense": (500, 2064, 2080),
    "100 rows, dense, one stage": (1000, 1040, 256),
    "128 rows": ([300, 0, 700, 1, 290], 2064, 544),
    "128 rows, dense": (1300, 2064, 1056),
    "128 rows, dense, one stage": (1300, 2064, 224),
    "large": ([1900, 0, 1100, 2300, 1700], 2064, 2080),
    "large, one stage": ([1900, 0, 1100, 2300, 1700], 4112, 96),
    "large, two stages": ([1900, 0, 1100, 2300, 1700], 4112, 288),
    "large, dense": (4000, 2064, 2080),
    "large, dense, one stage": (9000, 4112, 256),
    "large, whole lines": ([1900, 0, 1100, 2300, 1700], 2048, 512),
    "many stages": ([901, 600, 1, 700], 2064, 8224),
    "many experts": ([(29 * i) % 231 for i in range(64)], 1040, 2080),
    "many experts, one stage": ([(29 * i) % 231 for i in range(64)], 1040, 64),
    "many experts, whole stages": ([(29 * i) % 131 for i in range(64)], 1040, 1024),
}
# row-major weights of any N: rows that are not whole pieces of 16 bytes
ODD = {
    "odd, 32 rows": ([(5 * i) % 23 for i in range(64)], 1001, 544),
    "odd, dense": (1000, 1037, 544),
    "odd, 128 rows": ([300, 0, 700, 1, 290], 2055, 544),
    "odd, large": ([1900, 0, 1100, 2300, 1700], 2061, 288),
    "odd, many experts": ([(29 * i) % 231 for i in range(64)], 1026, 512),
    "narrow": (5000, 3, 288),
    "one column": (70, 1, 64),
}


def run(case, layout):
    rows, N, K = case
    dense = isinstance(rows, int)
    counts = [rows] if dense else rows
    off, cnt, M = ranges(counts, gap=0 if dense else 3, lead=0 if dense else 5)
    M = rows if dense else M
    E, g = len(counts), gen(N + K + M)
    idle = torch.ones(M, dtype=torch.bool, device=DEV)
    for r in rows_of(off, cnt):
        idle[r] = False
    for kind in ("ints", "binades"):
        xq, xb = operand(g, M, K, kind)
        xb[idle] = 255
        xs = group(xb)
        w, ws, values = weights(g, E, N, K, kind, layout)
        for dt in BOTH:
            print(f"[mx tiles] {case[1:]} rows {sum(counts)} {kind} {dt} layout {layout}", flush=True)
            buf = torch.full((M * N + 64,), 7.0, dtype=dt, device=DEV)
            y = buf[:M * N].view(M, N)
            if dense:
                qm.moe_mx_mm(xq, xs, w[0], ws if layout == ROWS else ws[0], layout=layout, out=y)
            else:
                qm.moe_grouped_mx_mm(xq, xs, w, ws, off, cnt, sum(counts), layout=layout, out=y)
            torch.cuda.synchronize()
            assert bool((buf[M * N:] == 7).all()) and bool((y[idle] == 7).all())
            for e, r in enumerate(rows_of(off, cnt)):
                if r.stop > r.start:
                    check_product(f"expert {e}", y[r], decode(xq[r], xb[r]), values[e], kind)


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_products(case, layout):
    run(CASES[case], layout)


@pytest.mark.parametrize("case", ODD, ids=str)
def test_odd_widths(case):
    run(ODD[case], ROWS)


@pytest.mark.parametrize("shift", [8, 24, 64])
def test_outputs_off_a_line(shift):
    """Views whose rows are whole pieces, but begin inside a 128-byte line."""
    M, N, K = 5000, 2048, 256
    g = gen(shift)
    xq, xb = operand(g, M, K, "ints")
    w, ws, values = weights(g, 1, N, K, "ints", ROWS)
    buf = torch.full((M * N + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = qm.moe_mx_mm(xq, group(xb), w[0], ws, out=buf[shift:shift + M * N].view(M, N))
    check_product("shifted", y, decode(xq, xb), values[0], "ints")
    assert bool((buf[:shift] == 7).all()) and bool((buf[shift + M * N:] == 7).all())
