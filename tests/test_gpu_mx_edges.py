"""The MXFP4 products' edges at every kernel that the launcher picks, in both orders of the weights: scales that are NaN, of the
smallest and largest value, sums that cancel, ranges out of order and ranges that are none (tests/test_mx_edge_choice.py checks
that these sizes and hints reach every kernel).

Bounds as in tests/test_gpu_mx.py.  Where every sum of any of a result's terms is a whole multiple of one power of two, less than
2^24 of them, fp32 sums have no rounding in whatever order: those results have to be exact.
"""
import itertools

import numpy as np
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import check, gen, ranges, rows_of
from tests.test_gpu_mx import ROWS, TILE16, decode, group, operand, tile16
from tests.test_gpu_rows import some_slots

pytestmark = pytest.mark.gpu

DEV = "cuda"
BOTH = (torch.bfloat16, torch.float32)

# rows of each expert (an int: dense), N, K: 17 blocks of 32 columns are two stages of 256 and a part, 32 are four whole ones
EDGES = {
    "few rows": ([9, 0, 21, 1], 96, 544),
    "few rows, dense": (336, 64, 544),
    "32 rows": ([(5 * i) % 23 for i in range(64)], 1040, 544),
    "32 rows, dense": (336, 1040, 544),
    "128 rows": ([300, 0, 700, 1, 290], 2064, 544),
    "128 rows, dense": (1300, 2064, 544),
    "large": ([1900, 0, 1100, 2300, 1700], 2064, 544),
    "large, dense": (4000, 2064, 544),
    "many experts": ([(29 * i) % 231 for i in range(64)], 1040, 544),
    "many experts, whole stages": ([(29 * i) % 131 for i in range(64)], 1040, 1024),
}


class Case:
    """A product's sizes, and the call with codes and scale bytes [rows, K / 32] of both sides."""
    def __init__(self, name, layout):
        rows, self.N, self.K = EDGES[name]
        self.dense, self.layout, self.name = isinstance(rows, int), layout, name
        self.off, self.cnt, self.M = ranges([rows] if self.dense else rows, *(() if self.dense else (3, 1, 5)))
        self.E, self.total = len(self.cnt), int(self.cnt.sum())
        self.idle = torch.ones(self.M, dtype=torch.bool, device=DEV)
        for r in rows_of(self.off, self.cnt):
            self.idle[r] = False

    def product(self, xq, xb, wq, wb, dt):
        print(f"[mx edges] {self.name} layout {self.layout} {dt}", flush=True)
        w, ws = wq.view(self.E, self.N, -1), group(wb)
        if self.layout == TILE16:
            w, ws = tile16(w, 16), tile16(wb.view(self.E, self.N, -1), 1)
        y = torch.full((self.M, self.N), 7.0, dtype=dt, device=DEV)
        if self.dense:
            qm.moe_mx_mm(xq, group(xb), w[0], ws if self.layout == ROWS else ws[0], layout=self.layout, out=y)
        else:
            qm.moe_grouped_mx_mm(xq, group(xb), w, ws, self.off, self.cnt, self.total, layout=self.layout, out=y)
        assert bool((y[self.idle] == 7).all())
        return y

    def experts(self, xq, xb, wq, wb):
        """(rows, values of x, values of w) of each expert that has rows, in 64 bits."""
        for e, r in enumerate(rows_of(self.off, self.cnt)):
            if r.stop > r.start:
                n = slice(e * self.N, e * self.N + self.N)
                yield r, decode(xq[r], xb[r]), decode(wq[n], wb[n])


every_kernel = pytest.mark.parametrize("name,layout", list(itertools.product(EDGES, (ROWS, TILE16))), ids=str)


@every_kernel
def test_scales_of_255(name, layout):
    """Blocks that are NaN, in rows of x and in weight rows, at every place of a stage: NaN in the outputs of those rows and
    columns, and nowhere else."""
    c = Case(name, layout)
    g = gen(c.M + c.N)
    xq, xb = operand(g, c.M, c.K, "binades")
    wq, wb = operand(g, c.E * c.N, c.K, "binades")
    for b in (xb, wb):
        rows = torch.randperm(len(b), device=DEV, generator=g)[:len(b) // 6 + 1]
        b[rows, torch.randint(0, c.K // 32, (len(rows),), device=DEV, generator=g)] = 255
    xb[c.idle] = 255
    for dt in BOTH:
        y = c.product(xq, xb, wq, wb, dt)
        for r, X, W in c.experts(xq, xb, wq, wb):
            ref, bad = X @ W.t(), X.isnan().any(1)[:, None] | W.isnan().any(1)[None, :]
            assert torch.equal(y[r].isnan(), bad)
            check(name, torch.where(bad, 0, y[r]), torch.where(bad, 0.0, ref),
                  torch.where(bad, 0.0, X.abs().nan_to_num() @ W.abs().nan_to_num().t()), c.K)


@every_kernel
def test_scales_at_the_ends(name, layout):
    """Scale bytes of both sides from 0 to 254, another pair for each block, whose products are near 1: exact."""
    c = Case(name, layout)
    g = gen(c.M + c.K)
    xq, _ = operand(g, c.M, c.K, "ints")
    wq, _ = operand(g, c.E * c.N, c.K, "ints")
    rows, some = [torch.randint(-3, 4, (n, 1), device=DEV, generator=g) for n in (c.M, c.E * c.N)]
    block = torch.randint(3, 252, (1, c.K // 32), device=DEV, generator=g)
    block[0, :4] = torch.tensor([3, 251, 3, 251], device=DEV)
    xb, wb = (block + rows).to(torch.uint8), (254 - block + some).to(torch.uint8)
    assert int(xb.min()) == 0 and int(xb.max()) == 254 and int(wb.min()) == 0 and int(wb.max()) == 254
    y = c.product(xq, xb, wq, wb, torch.float32)
    for r, X, W in c.experts(xq, xb, wq, wb):
        assert torch.equal(y[r].double(), X @ W.t())


@every_kernel
def test_products_past_the_range(name, layout):
    """2^127 * 2^127 is infinite, 2^-127 * 2^-127 is 0, whatever the codes are beside them."""
    c = Case(name, layout)
    ones = torch.full((c.M, c.K // 2), 0x22, dtype=torch.uint8, device=DEV)
    w = torch.full((c.E * c.N, c.K // 2), 0x22, dtype=torch.uint8, device=DEV)
    xb, wb = [torch.zeros(len(t), c.K // 32, dtype=torch.uint8, device=DEV) for t in (ones, w)]
    for dt in BOTH:
        assert bool((c.product(ones, xb, w, wb, dt)[~c.idle] == 0).all())
        assert bool((c.product(ones, xb + 254, w, wb + 254, dt)[~c.idle] == float("inf")).all())


@every_kernel
@pytest.mark.parametrize("s", [10, 18, 23])
def test_sums_that_cancel(name, layout, s):
    """Every row of x has 2^s in one block, -2^s in a second and a small number in a third, the blocks in every order within
    an instruction, a stage, and across them: what is left is the small number's product, exactly.  (Whole numbers of at most
    2^23 + 12, times the row's and the column's own powers of two.)"""
    c = Case(name, layout)
    g, blocks = gen(c.M + s), c.K // 32
    near = list(itertools.permutations((0, 1, 4, 5, 8, 16), 3))
    rng = np.random.default_rng(s)
    places = np.array((near + [tuple(rng.permutation(blocks)[:3]) for _ in range(c.M)])[:c.M])
    rng.shuffle(places)
    at, i = torch.from_numpy(places).to(DEV), torch.arange(c.M, device=DEV)
    # columns 0 and 1 of a block are the two halves of its first byte: 1 and -1 in column 0, the small number in column 1
    xq = torch.zeros(c.M, blocks, 16, dtype=torch.uint8, device=DEV)
    small = torch.tensor([0x2, 0x4, 0x5, 0x6, 0x7, 0xA, 0xC, 0xD], dtype=torch.uint8, device=DEV)  # 1 2 3 4 6 -1 -2 -3
    xq[i, at[:, 0], 0] = 0x2
    xq[i, at[:, 1], 0] = 0xA
    xq[i, at[:, 2], 0] = small[torch.randint(0, 8, (c.M,), device=DEV, generator=g)] << 4
    xb = torch.randint(0, 255, (c.M, blocks), device=DEV, generator=g)
    own = torch.randint(110, 140, (c.M,), device=DEV, generator=g)
    xb[i, at[:, 0]] = xb[i, at[:, 1]] = own + s
    xb[i, at[:, 2]] = own
    wq, _ = operand(g, c.E * c.N, c.K, "ints")
    pair = torch.tensor([0x22, 0x42, 0xA2, 0xC2], dtype=torch.uint8, device=DEV)  # 1 in column 0; 1 2 -1 -2 in column 1
    wq = wq.view(-1, blocks, 16)
    wq[:, :, 0] = pair[torch.randint(0, 4, wq.shape[:2], device=DEV, generator=g)]
    wb = torch.randint(110, 140, (c.E * c.N, 1), device=DEV, generator=g).repeat(1, blocks)
    xq, wq, xb, wb = xq.view(c.M, -1), wq.view(c.E * c.N, -1), xb.to(torch.uint8), wb.to(torch.uint8)
    for dt in BOTH:
        y = c.product(xq, xb, wq, wb, dt)
        for r, X, W in c.experts(xq, xb, wq, wb):
            ref = X @ W.t()  # exact in 64 bits as well
            assert bool((ref != 0).all())
            assert torch.equal(y[r], ref.to(dt)), name


# ------------------------------------------------------------------------------------------- ranges

HINTS = [1, 60, 300, 1500, 2100]  # how many rows the call is told to expect, of what it is then given
RANGES_N, RANGES_K, RANGES_M = 4112, 2048, 2100


def ranged(layout, off, cnt, hint, seed=0):
    """The product of M rows with 6 experts, in the middle of a buffer of sevens."""
    g = gen(seed)
    xq, xb = operand(g, RANGES_M, RANGES_K, "binades")
    wq, wb = operand(g, 6 * RANGES_N, RANGES_K, "binades")
    w, ws = wq.view(6, RANGES_N, -1), group(wb)
    if layout == TILE16:
        w, ws = tile16(w, 16), tile16(wb.view(6, RANGES_N, -1), 1)
    buf = torch.full((RANGES_M + 16, RANGES_N), 7.0, device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    c = None if cnt is None else torch.tensor(cnt, dtype=torch.int32, device=DEV)
    print("[mx edges]", off, cnt, "hint", hint, "layout", layout, flush=True)
    y = qm.moe_grouped_mx_mm(xq, group(xb), w, ws, o, c, hint, layout=layout, out=buf[8:-8])
    torch.cuda.synchronize()
    assert bool((buf[:8] == 7).all()) and bool((buf[-8:] == 7).all())
    return y, xq, xb, wq, wb


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("off,cnt", [([2000, 5, 1100, 900, 300, 299], [100, 294, 800, 130, 597, 1]),
                                     ([40, 0, 0, 60, 20, 10], [16, 0, 3, 33, 1, 7]),
                                     ([0, 0, 2100, 0, 2100, 2100], [0, 0, 0, 2100, 0, 0])], ids=str)
def test_ranges_in_any_order(layout, hint, off, cnt):
    """Experts whose rows lie in another order than the experts, many rows or few, whatever number the call was told."""
    y, xq, xb, wq, wb = ranged(layout, off, cnt, hint)
    idle = torch.ones(RANGES_M, dtype=torch.bool, device=DEV)
    for e in range(6):
        r, n = slice(off[e], off[e] + cnt[e]), slice(e * RANGES_N, (e + 1) * RANGES_N)
        if cnt[e]:
            idle[r] = False
            X, W = decode(xq[r], xb[r]), decode(wq[n], wb[n])
            check(f"expert {e}", y[r], X @ W.t(), X.abs() @ W.abs().t(), RANGES_K)
    assert bool((y[idle] == 7).all())


BIG, SMALL = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("layout", [ROWS, TILE16])
@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("off,cnt", [([0, 1500, 20, 2100, 10, 600, 2100], None), ([BIG] * 7, None),
                                     ([SMALL, 0, BIG, 5, SMALL, 2100, BIG], None), ([0] * 7, [BIG] * 6),
                                     ([-5, 1900, 4000, 0, 10, 10, 0], [30, 300, 5, SMALL, 2100, 0])], ids=str)
def test_ranges_that_are_not_ranges(layout, hint, off, cnt):
    """Whatever the device arrays hold, nothing outside y is written, and the call ends."""
    ranged(layout, off, cnt, hint)


# ------------------------------------------------------------------------------------------- another stream

def test_rows_quantised_into_slots_on_a_stream_of_their_own():
    """Every row has its pair, so all of both outputs is compared."""
    T, k, K = 100, 3, 512
    x = torch.randn(T, K, device=DEV, generator=gen(2)).to(torch.bfloat16)
    slots = some_slots(T, k, T * k, 2, lost=0.0)
    want = [t.clone() for t in qm.moe_quantize_mx(x, slots)]
    torch.cuda.synchronize()
    S = torch.cuda.Stream()
    with torch.cuda.stream(S):
        got = qm.moe_quantize_mx(x, slots, stream=S)
    S.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q, s = qm.moe_quantize_mx(x)
    at = slots.view(-1).long()
    assert torch.equal(want[0][at], q.repeat_interleave(k, 0)) and torch.equal(want[1][:, at], s.repeat_interleave(k, 1))
