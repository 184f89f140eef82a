"""The grouped products at the largest tiles and at every weight hint: sizes that the launcher sends to the forms which
smaller tests do not reach (tests/test_tile_choice.py checks that they do), with sizes off the tile, ragged and empty
experts and contractions of one, two and many stages.

Tolerances as in tests/test_gpu_grouped.py: integer inputs come out exactly in fp32, others within n * 2^-23 of the sum of
magnitudes, and rounded once to bf16.
"""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import bf16, check, fill_outside, gen, ints, ranges, rows_of

pytestmark = pytest.mark.gpu

DEV = "cuda"

# (rows of each expert, N, K): forward tiles are over N and rows, dgrad's over K and rows, wgrad's over N and K
CASES = {
    "large": ([1900, 0, 1100, 2300, 1700], 2008, 2056),
    "two stages": ([1900, 0, 1100, 2300, 1700], 4104, 72),  # forward K 72, dgrad far from few
    "two stages, dgrad": ([1900, 0, 1100, 2300, 1700], 72, 4104),
    "one stage": ([1900, 0, 1100, 2300, 1700], 4104, 8),
    "one stage, dgrad": ([1900, 0, 1100, 2300, 1700], 8, 4104),
    "whole lines": ([1900, 0, 1100, 2300, 1700], 2048, 4160),  # outputs past L2 whose rows are whole 128-byte lines
    "many stages": ([3001, 2600, 1, 3000], 2056, 4104),
    "many small experts": ([(11 * i) % 97 for i in range(64)], 1032, 2056),
    "many tiny experts": ([(5 * i) % 23 for i in range(64)], 1032, 2056),
    "ragged": ([(29 * i) % 331 for i in range(64)], 1032, 2056),
}


@pytest.mark.parametrize("kind", ["ints", "normal"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_products(case, kind):
    counts, N, K = CASES[case]
    off, cnt, M = ranges(counts, gap=3, lead=5)
    E, g, make = len(counts), gen(N + K + M), ints if kind == "ints" else bf16
    x, w, dy = make(g, M, K), make(g, E, N, K), make(g, M, N)
    fill_outside(dy, off, cnt, float("nan"))
    idle = fill_outside(x, off, cnt, float("nan"))
    for dt in (torch.float32, torch.bfloat16):
        y, dx = torch.full((M, N), 7.0, dtype=dt, device=DEV), torch.full((M, K), 7.0, dtype=dt, device=DEV)
        dw = torch.full((E + 1, N, K), 7.0, dtype=dt, device=DEV)
        print(f"[tiles] {case} {kind} {dt}", flush=True)
        qm.moe_grouped_mm(x, w, off, cnt, sum(counts), out=y)
        qm.moe_grouped_mm_dgrad(dy, w, off, cnt, sum(counts), out=dx)
        qm.moe_grouped_mm_wgrad(dy, x, off, cnt, sum(counts), out=dw[:E])
        torch.cuda.synchronize()
        assert bool((y[idle] == 7).all()) and bool((dx[idle] == 7).all()) and bool((dw[E] == 7).all())
        for e, r in enumerate(rows_of(off, cnt)):
            X, W, D = x[r].double(), w[e].double(), dy[r].double()
            for name, got, a, b in (("y", y[r], X, W.t()), ("dx", dx[r], D, W), ("dw", dw[e], D.t(), X)):
                ref = a @ b
                if kind == "ints":
                    assert torch.equal(got, ref.to(dt)), (name, e)
                else:
                    check(f"{name} {e}", got, ref, a.abs() @ b.abs(), max(1, a.shape[1]))
