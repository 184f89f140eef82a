"""Rows to the experts and back, and the quantiser, at sizes that the smaller tests do not reach: more than 100 MB of pair rows,
which are read past the caches by kernels of their own (csrc/rows.hip), and more tokens or pairs than a launch has workgroups
(2^20, or 2^22 waves), which take several turns each.

Bounds as in tests/test_gpu_rows.py.
"""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import check, gen
from tests.test_gpu_mx import decode, ungroup
from tests.test_gpu_rows import there

pytestmark = pytest.mark.gpu

DEV = "cuda"
BOTH = (torch.bfloat16, torch.float32)
PAST_CACHES, GROUPS, WAVES = 100_000_000, 1 << 20, 1 << 22

# tokens, choices, columns
LARGE = [(8192, 8, 1024), (7001, 8, 1000), (GROUPS + 333, 1, 64), (GROUPS + 77, 2, 8), (WAVES // 2 + 5, 2, 8)]


def inputs(T, k, H, dtype, g, lost=0.05):
    """Rows, and different ones of them for the pairs; a share of the pairs has none."""
    M = T * k + 3
    rows = torch.empty(M, H, dtype=dtype, device=DEV).normal_(generator=g)
    slots = torch.randperm(M, device=DEV, generator=g)[:T * k].to(torch.int32)
    slots[torch.rand(T * k, device=DEV, generator=g) < lost] = -1
    return rows, slots.view(T, k)


def parts(T):
    """The tokens in parts that a reference in 64 bits has room for."""
    return [slice(t, min(t + 65536, T)) for t in range(0, T, 65536)]


def pair_rows(rows, slots, part):
    s = slots[part]
    return torch.where((s >= 0)[:, :, None], rows[s.clamp_min(0).long()].double(), 0.0)


def test_sizes_are_past_the_limits():
    sizes = [T * k * H * 2 > PAST_CACHES for T, k, H in LARGE]
    assert sizes == [True, True, True, False, False]
    assert [T > GROUPS for T, _, _ in LARGE] == [False, False, True, True, True]
    assert LARGE[-1][0] * LARGE[-1][1] > WAVES


@pytest.mark.parametrize("out", BOTH, ids=str)
@pytest.mark.parametrize("dtype", BOTH, ids=str)
@pytest.mark.parametrize("T,k,H", LARGE)
def test_combine_rows(T, k, H, dtype, out):
    g = gen(T + H)
    rows, slots = inputs(T, k, H, dtype, g)
    w = torch.randn(T, k, device=DEV, generator=g)
    add = torch.empty(T, H, dtype=out, device=DEV).normal_(generator=g)
    print(f"[rows] combine {T} {k} {H} {dtype} {out}", flush=True)
    got = qm.moe_combine_rows(rows, slots, w, add=add, out_dtype=out)
    plain = qm.moe_combine_rows(rows, slots, out_dtype=out)
    for p in parts(T):
        y = pair_rows(rows, slots, p)
        wy = torch.where((slots[p] >= 0)[:, :, None], y * w[p].double()[:, :, None], 0.0)
        a = add[p].double()
        check("weighted", got[p], wy.sum(1) + a, wy.abs().sum(1) + a.abs(), k + 2)
        check("plain", plain[p], y.sum(1), y.abs().sum(1), k + 2)


@pytest.mark.parametrize("dout_type", BOTH, ids=str)
@pytest.mark.parametrize("dtype", BOTH, ids=str)
@pytest.mark.parametrize("T,k,H", LARGE)
def test_combine_rows_grad(T, k, H, dtype, dout_type):
    g = gen(T + H)
    rows, slots = inputs(T, k, H, dtype, g)
    w = torch.randn(T, k, device=DEV, generator=g)
    dout = torch.empty(T, H, dtype=dout_type, device=DEV).normal_(generator=g)
    drows = torch.full_like(rows, 7.0)
    print(f"[rows] gradients {T} {k} {H} {dtype} {dout_type}", flush=True)
    _, dw = qm.moe_combine_rows_grad(dout, rows, slots, w, drows=drows)
    ok = there(slots, len(rows))
    for p in parts(T):
        d = dout[p].double()[:, None, :]
        y = pair_rows(rows, slots, p) * d
        check("dweights", dw[p], y.sum(2), y.abs().sum(2), H)
        ref = (w[p].double()[:, :, None] * d)[ok[p]]
        check("drows", drows[slots[p][ok[p]].long()], ref, ref.abs(), 1)
    idle = torch.ones(len(rows), dtype=torch.bool, device=DEV)
    idle[slots[ok].long()] = False
    assert bool((drows[idle] == 7).all()) and bool((dw[~ok] == 0).all())


@pytest.mark.parametrize("T,k,H", LARGE)
def test_gather_rows(T, k, H):
    g = gen(T)
    rows, slots = inputs(T, k, H, torch.bfloat16, g)
    x = rows[:T].clone()
    out = torch.full_like(rows, 7.0)
    qm.moe_gather_rows(x, slots, out=out)
    ok = there(slots, len(rows))
    want = torch.full_like(rows, 7.0)
    want[slots[ok].long()] = x[torch.nonzero(ok)[:, 0]]
    assert torch.equal(out, want)


def test_pair_slots():
    """More pairs than fit 2^22, of few experts: each is found."""
    T, k, E = WAVES // 2 + 5, 2, 8
    first = torch.randint(0, E, (T,), device=DEV, generator=gen(1))
    ids = torch.stack([first, (first + 1 + torch.randint(0, E - 1, (T,), device=DEV, generator=gen(2))) % E], 1).to(torch.int32)
    al = qm.moe_align(ids, E, 16)
    got = qm.moe_pair_slots(ids, al.sorted_ids, al.offsets, al.counts)
    assert torch.equal(al.sorted_ids[got.view(-1).long()], torch.arange(T * k, dtype=torch.int32, device=DEV))


def test_quantiser():
    """More rows than a launch has waves, there and back: every value within the block's half step, codes of the grid as they
    were."""
    T, K = WAVES + 9, 32
    x = torch.empty(T, K, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(3))
    q, s = qm.moe_quantize_mx(x)
    y = qm.moe_dequantize_mx(q, s)
    for p in parts(T):
        assert torch.equal(y[p].double(), decode(q[p], ungroup(s[:, p], K)))
    unit = torch.exp2(s.view(T, 4)[:, :1].float() - 127)  # powers of two near 1
    # steps of 1/2, 1 and 2 units below 2, 4 and 6 units
    a = x.float().abs() / unit
    half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0))
    assert bool(((y.float() - x.float()).abs() <= half * unit).all()) and bool((a.amax(1) <= 6).all())
    assert bool((a.amax(1) > 3).all())  # a smaller unit would not do
    again, s2 = qm.moe_quantize_mx(y)
    grid = (y.float() / unit).abs().amax(1) > 3  # whose largest value, rounded, still needs the unit
    assert torch.equal(again[grid], q[grid]) and torch.equal(s2.view(T, 4)[grid], s.view(T, 4)[grid])
    slots = torch.randperm(T, device=DEV, generator=gen(4)).to(torch.int32).view(T, 1)
    q2, s2 = qm.moe_quantize_mx(x, slots)
    at = slots.view(-1).long()
    assert torch.equal(q2[at], q) and torch.equal(s2[:, at], s)
