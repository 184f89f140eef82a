"""Sums of the fp8 block products on the GPU: fp32 throughout, whatever the output's type, the number of rows and
``expected_rows``.

Exact cases: every 8 consecutive k hold 448 * 448, 448 * -448 and one product a_r * b_n of small integers, in an order
that changes from group to group.  A block of 128 sums 16 such groups: integers whose partial sums stay below
16 * 448^2 < 2^22 in any order, so fp32 holds every one of them and the result is a_r * b_n * K / 8, rounded once to the
output's type.  An adder that aligns products to the largest of a group and keeps fewer than 18 bits below it loses
a_r * b_n.

Other inputs: the bound of tests/test_gpu_grouped.py's check(), sums of n products off by at most n * 2^-23 of the sum of
magnitudes, for outputs of either type.
"""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import check, dequant_rows, dequant_weights, fp8_rows, fp8_weights, gen, ranges, rows_of, tile16

pytestmark = pytest.mark.gpu

DEV, FP8 = "cuda", torch.float8_e4m3fn
BOTH = (torch.float32, torch.bfloat16)

# (M, N, K): one row, few rows, and each tile that the launcher picks by rows and outputs
DENSE = [(1, 1024, 2048), (5, 4096, 128), (16, 8192, 128), (40, 4096, 128), (64, 130, 2048), (100, 384, 1040), (256, 4096, 512), (500, 4096, 272),
         (600, 1320, 1040), (1000, 2050, 272), (2100, 4096, 272), (4100, 4100, 400)]
GROUPS = {
    "tiny": [3, 0, 1, 2],
    "mean 2": [i % 5 for i in range(130)],
    "mean 24": [(7 * i) % 49 for i in range(130)],
    "mean 48": [(11 * i) % 97 for i in range(130)],
    "mean 80": [(13 * i) % 161 for i in range(130)],
    "wide": [300, 257, 255, 0, 256],
    "huge": [1300, 0, 900],
}


def cancelling(g, M, N, K):
    """Codes of rows and weights whose products cancel but for a_r * b_n in every 8 consecutive k, and the exact result."""
    a = torch.randint(1, 4, (M, 1), device=DEV, generator=g).double()
    b = torch.randint(1, 4, (N, 1), device=DEV, generator=g).double()
    order = torch.rand(K // 8, 8, device=DEV, generator=g).argsort(1).view(-1)  # of each group's eight places
    big = (order == 0) | (order == 1)
    sign = torch.where(order == 1, -1.0, 1.0).double()
    x = torch.where(big, 448.0, 0.0) + torch.where(order == 2, a, 0.0)
    w = torch.where(big, 448.0 * sign, 0.0) + torch.where(order == 2, b, 0.0)
    assert torch.equal(x.float().to(FP8).double(), x) and torch.equal(w.float().to(FP8).double(), w)
    return x.float().to(FP8), w.float().to(FP8), (a @ b.t()) * (K // 8)


def ones(*shape):
    return torch.ones(*shape, device=DEV)


@pytest.mark.parametrize("M,N,K", DENSE)
def test_small_terms_survive_cancelling_ones(M, N, K):
    xq, wq, ref = cancelling(gen(M + N + K), M, N, K)
    NB, KB = -(-N // 128), -(-K // 128)
    for dt in BOTH:
        for layout in (qm.MOE_LAYOUT_ROWS, qm.MOE_LAYOUT_TILE16):
            if layout == qm.MOE_LAYOUT_TILE16 and N % 16:
                continue
            w = tile16(wq[None])[0] if layout == qm.MOE_LAYOUT_TILE16 else wq
            y = qm.moe_block_mm(xq, ones(KB, M), w, ones(NB, KB), layout, out_dtype=dt)
            torch.cuda.synchronize()
            assert torch.equal(y, ref.to(dt)), (dt, layout, float(y.double().min()), float(ref.min()))


@pytest.mark.parametrize("N,K", [(144, 272), (1024, 272), (1040, 2048)])
@pytest.mark.parametrize("counts", GROUPS, ids=str)
def test_small_terms_survive_by_expert(counts, N, K):
    off, cnt, M = ranges(GROUPS[counts])
    E, g = len(GROUPS[counts]), gen(N + K + M)
    xq, w1, ref = cancelling(g, M, N, K)
    wq, ws = w1.expand(E, N, K).contiguous(), ones(E, -(-N // 128), -(-K // 128))
    for dt in BOTH:
        for hint in (None, 1):
            y = qm.moe_grouped_block_mm(xq, ones(-(-K // 128), M), wq, ws, off, cnt, hint, out_dtype=dt)
            torch.cuda.synchronize()
            assert torch.equal(y, ref.to(dt)), (dt, hint)


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense_sums_within_the_fp32_bound(M, N, K):
    g = gen(M + N + K)
    xq, xs = fp8_rows(g, M, K)
    wq, ws = fp8_weights(g, 1, N, K)
    X, W = dequant_rows(xq, xs), dequant_weights(wq[0], ws[0])
    for dt in BOTH:
        y = qm.moe_block_mm(xq, xs, wq[0], ws[0], out_dtype=dt)
        torch.cuda.synchronize()
        check(f"block mm {M} {N} {K} {dt}", y, X @ W.t(), X.abs() @ W.abs().t(), K + K // 128 + 3)


@pytest.mark.parametrize("N,K", [(144, 272), (1040, 2048)])
@pytest.mark.parametrize("counts", GROUPS, ids=str)
def test_sums_by_expert_within_the_fp32_bound(counts, N, K):
    off, cnt, M = ranges(GROUPS[counts])
    E, g = len(GROUPS[counts]), gen(N + K + M)
    xq, xs = fp8_rows(g, M, K)
    wq, ws = fp8_weights(g, E, N, K)
    for dt in BOTH:
        y = qm.moe_grouped_block_mm(xq, xs, wq, ws, off, cnt, out_dtype=dt)
        again = qm.moe_grouped_block_mm(xq, xs, wq, ws, off, cnt, out_dtype=dt)
        torch.cuda.synchronize()
        assert torch.equal(y, again)
        for e, r in enumerate(rows_of(off, cnt)):
            X, W = dequant_rows(xq[r], xs[:, r]), dequant_weights(wq[e], ws[e])
            check(f"by expert {counts} {e} {dt}", y[r], X @ W.t(), X.abs() @ W.abs().t(), K + K // 128 + 3)
