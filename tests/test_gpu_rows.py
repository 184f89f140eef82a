"""Rows to the experts and back on the GPU, against plain references in 64 bits.

Bounds: those of test_gpu_grouped's ``check``: a sum of n fp32 terms is off by at most n 2^-23 S, S the sum of the terms'
magnitudes, and storing it adds eps / 2 of its type.  Copied rows and places are exact.
"""
import numpy as np
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import check, gen

pytestmark = pytest.mark.gpu

DEV = "cuda"
BOTH = (torch.bfloat16, torch.float32)


def aligned(ids, E, block_m=16):
    """moe_align's outputs for a host array of ids [T, k]."""
    return qm.moe_align(torch.from_numpy(np.ascontiguousarray(ids, dtype=np.int32)).to(DEV), E, block_m)


def routing(T, k, E, seed=0, lost=0.0):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < lost] = -1
    return ids


def tight(ids, E):
    """The tight alignment of ids: sorted_ids [T k], offsets [E + 1], as torch tensors."""
    flat = ids.ravel()
    pairs = np.flatnonzero((flat >= 0) & (flat < E))
    pairs = pairs[np.argsort(flat[pairs], kind="stable")]
    out = np.full(flat.size, flat.size, dtype=np.int32)
    out[:len(pairs)] = pairs
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[pairs], minlength=E))]).astype(np.int32)
    return torch.from_numpy(out).to(DEV), torch.from_numpy(off).to(DEV)


def places(ids, sorted_ids):
    """The slots [T, k] that sorted_ids gives."""
    want = np.full(ids.size + 1, -1, dtype=np.int64)
    want[sorted_ids.cpu().numpy()] = np.arange(sorted_ids.numel())
    return want[:-1].reshape(ids.shape)


def some_slots(T, k, M, seed=0, lost=0.1):
    """Different rows of [0, M) for the pairs; some have none, told in every way there is."""
    rng = np.random.default_rng(seed)
    s = rng.permutation(M)[:T * k].astype(np.int64)
    s = np.concatenate([s, np.full(T * k - len(s), -1)])
    out = rng.random(T * k) < lost
    s[out] = rng.choice([-1, M, M + 7, -2 ** 31, 2 ** 31 - 1], size=int(out.sum()))
    return torch.from_numpy(s.astype(np.int32).reshape(T, k)).to(DEV)


def there(slots, M):
    return (slots >= 0) & (slots < M)


# ------------------------------------------------------------------------------------------- slots

@pytest.mark.parametrize("T,k,E,block_m,lost", [(1, 1, 1, 16, 0), (1, 8, 256, 16, 0), (3, 2, 8, 16, 0.3), (64, 8, 256, 16, 0),
                                                (333, 6, 60, 32, 0.1), (1500, 4, 5, 128, 0.02), (4096, 8, 256, 128, 0),
                                                (700, 1, 1024, 16, 0.5), (257, 3, 4, 64, 1.0)])
def test_pair_slots(T, k, E, block_m, lost):
    ids = routing(T, k, E, T, lost)
    ids[ids < 0] = np.random.default_rng(1).choice([-1, E, 2 ** 31 - 1, -2 ** 31], size=int((ids < 0).sum()))
    al = aligned(ids, E, block_m)
    tid = torch.from_numpy(ids).to(DEV)
    got = qm.moe_pair_slots(tid, al.sorted_ids, al.offsets, al.counts)
    assert got.dtype == torch.int32 and (got.cpu().numpy() == places(ids, al.sorted_ids)).all()
    srt, off = tight(ids, E)
    got = qm.moe_pair_slots(tid, srt, off)
    assert (got.cpu().numpy() == places(ids, srt)).all()


def test_pair_slots_of_arrays_that_are_no_alignment():
    """Whatever the device arrays hold, every slot is written, and is -1 or the place of its pair."""
    rng = np.random.default_rng(5)
    T, k, E, M = 200, 4, 16, 700
    ids = torch.from_numpy(rng.integers(-2, E + 2, (T, k)).astype(np.int32)).to(DEV)
    for off in (rng.integers(-900, 900, E + 1), np.full(E + 1, 2 ** 31 - 1), np.full(E + 1, -2 ** 31), np.arange(E + 1)[::-1] * 50):
        for cnt in (None, rng.integers(-900, 2000, E), np.full(E, 2 ** 31 - 1)):
            srt = torch.from_numpy(rng.integers(-3, T * k + 3, M).astype(np.int32)).to(DEV)
            c = None if cnt is None else torch.from_numpy(cnt.astype(np.int32)).to(DEV)
            got = qm.moe_pair_slots(ids, srt, torch.from_numpy(off.astype(np.int32)).to(DEV), c,
                                    slots=torch.full((T, k), -77, dtype=torch.int32, device=DEV)).cpu().numpy().ravel()
            s = srt.cpu().numpy()
            assert ((got >= -1) & (got < M)).all()
            found = got >= 0
            assert (s[got[found]] == np.flatnonzero(found)).all()


# ------------------------------------------------------------------------------------------- gather

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8], ids=str)
@pytest.mark.parametrize("T,k,H", [(1, 8, 2048), (1, 1, 16), (7, 3, 48), (130, 2, 1040), (64, 70, 64), (2100, 4, 2064),
                                   (513, 1, 8192)])
def test_gather_rows(T, k, H, dtype):
    M = T * k + 11
    x = torch.randint(0, 256, (T, H * torch.empty(0, dtype=dtype).element_size()), dtype=torch.uint8, device=DEV,
                      generator=gen(T)).view(dtype)
    slots = some_slots(T, k, M, T + k)
    buf = torch.full((M + 8, x.view(torch.uint8).shape[1]), 99, dtype=torch.uint8, device=DEV)
    got = qm.moe_gather_rows(x, slots, out=buf[4:M + 4].view(dtype)).view(torch.uint8)
    want = torch.full_like(got, 99)
    ok = there(slots, M)
    want[slots[ok].long()] = x.view(torch.uint8)[torch.nonzero(ok)[:, 0]]
    assert torch.equal(got, want)
    assert bool((buf[:4] == 99).all()) and bool((buf[M + 4:] == 99).all())


# ------------------------------------------------------------------------------------------- combine

def combine_ref(rows, slots, weights, add, H):
    M, ok = rows.shape[0], there(slots, rows.shape[0])
    T, k = slots.shape
    w = torch.ones(T, k, device=DEV, dtype=torch.float64) if weights is None else weights.double()
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    for j in range(k):
        if M:
            term = torch.where(ok[:, j, None], w[:, j, None] * rows[torch.where(ok[:, j], slots[:, j], 0).long()].double(), 0.0)
            ref += term
            mag += term.abs()
    if add is not None:
        ref += add.double()
        mag += add.double().abs()
    return ref, mag


@pytest.mark.parametrize("out", BOTH, ids=str)
@pytest.mark.parametrize("dtype", BOTH, ids=str)
@pytest.mark.parametrize("T,k,H", [(1, 8, 2048), (1, 1, 8), (5, 3, 200), (64, 8, 2048), (33, 9, 520), (40, 70, 136),
                                   (300, 2, 4104), (129, 64, 64)])
def test_combine_rows(T, k, H, dtype, out):
    M, g = T * k + 5, gen(T + H)
    slots = some_slots(T, k, M, T)
    rows = torch.randn(M, H, device=DEV, generator=g).to(dtype)
    used = torch.zeros(M, dtype=torch.bool, device=DEV)
    used[slots[there(slots, M)].long()] = True
    rows[~used] = float("nan")  # rows of no pair are not read
    w = torch.randn(T, k, device=DEV, generator=g)
    w[~there(slots, M)] = float("inf")  # nor is the weight of a pair without a row
    add = torch.randn(T, H, device=DEV, generator=g).to(out)
    for weights in (w, None):
        for more in (add, None):
            buf = torch.full((T + 2, H), 7.0, dtype=out, device=DEV)
            got = qm.moe_combine_rows(rows, slots, weights, add=more, out=buf[1:T + 1])
            ref, mag = combine_ref(rows, slots, weights, more, H)
            check(f"combine {T} {k} {H} {dtype} {out}", got, ref, mag, k + 2)
            assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all())
    assert qm.moe_combine_rows(rows, slots).dtype == dtype


def test_combine_without_rows_and_shared_rows():
    """A token without rows gets add, or zeros; a row of two pairs counts for both; M = 0."""
    H = 64
    rows = torch.randn(6, H, device=DEV, generator=gen(1))
    slots = torch.tensor([[-1, 6], [2, 2], [5, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.0, 1], [0.5, 0.25], [2, float("nan")]], device=DEV)
    add = torch.randn(3, H, device=DEV, generator=gen(2))
    got = qm.moe_combine_rows(rows, slots, w, add=add)
    assert torch.equal(got[0], add[0])
    ref, mag = combine_ref(rows, slots, w, add, H)
    check("shared rows", got, ref, mag, 4)
    assert not qm.moe_combine_rows(rows, slots, w)[0].any()
    assert torch.equal(qm.moe_combine_rows(rows[:0], slots, w, add=add), add)
    assert not qm.moe_combine_rows(rows[:0], slots, w).any()
    dr, dw = qm.moe_combine_rows_grad(add, rows[:0], slots, w)
    assert dr.shape == (0, H) and not dw.any()


def test_values_that_are_not_finite():
    """A NaN or infinity in a row, a weight or add reaches its own token (and column) only."""
    T, k, H = 6, 2, 264
    rows = torch.ones(T * k, H, dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    w = torch.full((T, k), 0.5, device=DEV)
    rows[slots[1, 0], 3] = float("nan")
    rows[slots[2, 1], 5] = float("inf")
    w[4, 0] = float("inf")
    got = qm.moe_combine_rows(rows, slots, w).float()
    want = torch.ones(T, H, device=DEV)
    want[1, 3] = float("nan")
    want[2, 5] = want[4] = float("inf")
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    dout = torch.ones(T, H, device=DEV)
    dout[5, 7] = float("nan")
    dr, dw = qm.moe_combine_rows_grad(dout, rows, slots, w)
    assert dr[slots[5].long()].isnan().sum() == 2 and not dr[slots[:4].long()].isnan().any()
    assert dw[1, 0].isnan() and dw[5].isnan().all() and torch.isfinite(dw[[0, 3]]).all() and dw[2, 1] == float("inf")
    assert dw[4].tolist() == [264.0, 264.0]


# ------------------------------------------------------------------------------------------- gradients

@pytest.mark.parametrize("dout_type", BOTH, ids=str)
@pytest.mark.parametrize("dtype", BOTH, ids=str)
@pytest.mark.parametrize("T,k,H", [(1, 8, 2048), (1, 1, 8), (5, 3, 200), (101, 2, 264), (64, 8, 2056), (40, 70, 136),
                                   (33, 2, 8200)])
def test_combine_rows_grad(T, k, H, dtype, dout_type):
    M, g = T * k + 5, gen(T + H)
    slots = some_slots(T, k, M, T)
    ok = there(slots, M)
    rows = torch.randn(M, H, device=DEV, generator=g).to(dtype)
    dout = torch.randn(T, H, device=DEV, generator=g).to(dout_type)
    w = torch.randn(T, k, device=DEV, generator=g)
    buf = torch.full((M + 2, H), 7.0, dtype=dtype, device=DEV)
    wbuf = torch.full((T * k + 2,), 7.0, device=DEV)
    dr, dw = qm.moe_combine_rows_grad(dout, rows, slots, w, drows=buf[1:M + 1], dweights=wbuf[1:-1].view(T, k))
    token = torch.nonzero(ok)[:, 0]
    at = slots[ok].long()
    ref = w[ok].double()[:, None] * dout.double()[token]
    check("drows", dr[at], ref, ref.abs(), 1)
    idle = torch.ones(M, dtype=torch.bool, device=DEV)
    idle[at] = False
    assert bool((dr[idle] == 7).all()) and bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())
    terms = rows.double()[at] * dout.double()[token]
    check("dweights", dw[ok], terms.sum(1), terms.abs().sum(1), H)
    assert bool((dw[~ok] == 0).all()) and wbuf[0] == 7 and wbuf[-1] == 7


def test_gradients_against_differences():
    """The gradients of a scalar of the combined rows, by central differences in 64 bits of the same formula."""
    T, k, H = 4, 3, 16
    M, g = T * k, gen(3)
    slots = some_slots(T, k, M, 3)
    ok = there(slots, M)
    rows, w = torch.randn(M, H, device=DEV, generator=g), torch.randn(T, k, device=DEV, generator=g)
    dout = torch.randn(T, H, device=DEV, generator=g)
    dr, dw = qm.moe_combine_rows_grad(dout, rows, slots, w)

    def loss(r, v):
        return float((combine_ref(r, slots, v, None, H)[0] * dout.double()).sum())

    # the scalar is linear in each argument: a difference of step 1 is exact up to 64-bit rounding, and the kernel's
    # figures are off by at most H * 2^-23 of their terms
    for i, j in torch.nonzero(ok).tolist():
        up = w.double().clone()
        up[i, j] += 1
        terms = rows.double()[int(slots[i, j])] * dout.double()[i]
        assert abs(loss(rows, up) - loss(rows, w) - float(dw[i, j])) <= H * 2.0 ** -23 * float(terms.abs().sum()) + 1e-12
        for h in (0, 7, H - 1):
            up = rows.double().clone()
            up[int(slots[i, j]), h] += 1
            d = loss(up, w) - loss(rows, w)
            assert abs(d - float(dr[int(slots[i, j]), h])) <= 2.0 ** -23 * abs(d) + 1e-12


def test_gather_gradient_is_an_unweighted_combine():
    T, k, H = 50, 4, 136
    M, g = T * k + 3, gen(9)
    slots = some_slots(T, k, M, 9)
    ok = there(slots, M)
    drows = torch.randn(M, H, device=DEV, generator=g)
    x = torch.randn(T, H, dtype=torch.float64, device=DEV, requires_grad=True)
    x[torch.nonzero(ok)[:, 0]].backward(drows.double()[slots[ok].long()])
    ref, mag = combine_ref(drows, slots, None, None, H)
    assert torch.allclose(ref, x.grad, rtol=1e-14, atol=1e-14)
    check("gather gradient", qm.moe_combine_rows(drows, slots), x.grad, mag, k)


# ------------------------------------------------------------------------------------------- how they are called

def test_no_tokens_and_no_rows():
    s = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 64, device=DEV)
    assert qm.moe_gather_rows(x, s).shape == (0, 64)
    assert qm.moe_combine_rows(torch.ones(8, 64, device=DEV), s).shape == (0, 64)
    dr, dw = qm.moe_combine_rows_grad(x, torch.ones(8, 64, device=DEV), s, torch.empty(0, 4, device=DEV))
    assert dr.shape == (8, 64) and dw.shape == (0, 4)
    off = torch.zeros(9, dtype=torch.int32, device=DEV)
    assert qm.moe_pair_slots(s, torch.empty(0, dtype=torch.int32, device=DEV), off).shape == (0, 4)
    ids = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    got = qm.moe_pair_slots(ids, torch.empty(0, dtype=torch.int32, device=DEV), off)
    assert bool((got == -1).all())


def test_offsets_past_32_bits():
    """Rows whose byte offsets need more than 32 bits."""
    H, M = 8192, 300_000  # 4.9 GB of bf16 rows
    rows = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
    x = torch.randn(3, H, device=DEV, generator=gen(1)).to(torch.bfloat16)
    slots = torch.tensor([[M - 1], [0], [M - 2]], dtype=torch.int32, device=DEV)
    qm.moe_gather_rows(x, slots, out=rows)
    assert torch.equal(rows[slots.view(-1).long()], x)
    assert torch.equal(qm.moe_combine_rows(rows, slots), x)
    w = torch.full((3, 1), 2.0, device=DEV)
    _, dw = qm.moe_combine_rows_grad(x, rows, slots, w, drows=torch.empty_like(rows))
    ref = x.double().square().sum(1, keepdim=True)
    check("dweights of far rows", dw, ref, ref, H)


def test_run_of_them_captured_and_replayed():
    """Routing, alignment, slots, rows to the experts, their products, the rows back and the gradients, in a graph: every
    replay, on new inputs and with eager work between, gives what the calls give one by one."""
    T, k, E, H, I = 96, 4, 16, 256, 128
    g = gen(11)
    w1 = (torch.randn(E, I, H, device=DEV, generator=g) * 0.05).to(torch.bfloat16)
    w2 = (torch.randn(E, H, I, device=DEV, generator=g) * 0.05).to(torch.bfloat16)
    router = (torch.randn(E, H, device=DEV, generator=g) * 0.1).to(torch.bfloat16)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    dout = torch.empty(T, H, device=DEV)
    M = qm.moe_align_capacity(T, k, E, 16)

    def step():
        _, ids, wts = qm.moe_route(x, router, None, k)
        al = qm.moe_align(ids, E, 16)
        slots = qm.moe_pair_slots(ids, al.sorted_ids, al.offsets, al.counts)
        rows = qm.moe_gather_rows(x, slots, rows=M)
        a = qm.moe_grouped_mm(rows, w1, al.offsets, al.counts, T * k)
        y = qm.moe_grouped_mm(a, w2, al.offsets, al.counts, T * k)
        out = qm.moe_combine_rows(y, slots, wts, out_dtype=torch.float32)
        dy, dw = qm.moe_combine_rows_grad(dout, y, slots, wts)
        da = qm.moe_grouped_mm_dgrad(dy, w2, al.offsets, al.counts, T * k)
        dx = qm.moe_combine_rows(qm.moe_grouped_mm_dgrad(da, w1, al.offsets, al.counts, T * k), slots, out_dtype=torch.float32)
        return ids, wts, out, dw, dx

    def fill(seed):
        h = gen(seed)
        x.copy_(torch.randn(T, H, device=DEV, generator=h))
        dout.copy_(torch.randn(T, H, device=DEV, generator=h))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2, 3):
        fill(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), seed
    # the last step's values, against the formula: out and the gradients of sum(out * dout)
    ids, wts, out, dw, dx = outs
    assert bool((wts.sum(1) - 1).abs().max() < 1e-5)
    ref, dwr = torch.zeros(T, H, dtype=torch.float64, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
    scale = 0.0
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a = (x[t].double() @ w1[e].double().t()).to(torch.bfloat16).double()
        y = (a @ w2[e].double().t()).to(torch.bfloat16).double()
        ref.index_add_(0, t, y * wts[t, j].double()[:, None])
        dwr[t, j] = (y * dout[t].double()).sum(1)
    # a and y are rounded to bf16 twice on the way, from sums that may fall to either side of a rounding border: a step of
    # 2^-8 of y each, of terms that the largest of y bounds
    scale = float(y.abs().max())
    assert float((out.double() - ref).abs().max()) <= 4 * 2.0 ** -8 * max(scale, float(ref.abs().max()))
    assert float((dw.double() - dwr).abs().max()) <= 4 * 2.0 ** -8 * float(dout.abs().sum(1).max()) * max(scale, 1e-3)


def test_on_a_stream_of_its_own():
    """Calls with stream=S run behind S's own work, and what they allocate belongs to S."""
    T, k, H = 200, 4, 1024
    M, g = T * k, gen(4)
    x = torch.randn(T, H, device=DEV, generator=g)
    slots = some_slots(T, k, M, 4)
    w = torch.randn(T, k, device=DEV, generator=g)
    ids = routing(T, k, 8)
    al = aligned(ids, 8)
    tid = torch.from_numpy(ids).to(DEV)
    zero = torch.zeros(M, H, device=DEV)
    rows = qm.moe_gather_rows(x, slots, out=zero)

    def calls(stream):
        dr, dw = qm.moe_combine_rows_grad(x, rows, slots, w, drows=None, stream=stream)
        ok = there(slots, M)
        return [qm.moe_pair_slots(tid, al.sorted_ids, al.offsets, al.counts, stream=stream),
                qm.moe_gather_rows(x, slots, rows=M, stream=stream)[slots[ok].long()],
                qm.moe_combine_rows(rows, slots, w, stream=stream), dr[slots[ok].long()], dw]

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    S = torch.cuda.Stream()
    late = torch.zeros(T, H, device=DEV)
    with torch.cuda.stream(S):
        torch.cuda._sleep(50_000_000)
        late.copy_(x)
    got = qm.moe_gather_rows(late, slots, rows=M, stream=S)  # behind the copy
    S.synchronize()
    ok = there(slots, M)
    assert torch.equal(got[slots[ok].long()], want[1])
    with torch.cuda.stream(S):
        got = calls(S.cuda_stream)
    S.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_do_not_vary():
    T, k, H = 700, 8, 1024
    M, g = T * k, gen(6)
    rows = torch.randn(M, H, device=DEV, generator=g).to(torch.bfloat16)
    slots, w = some_slots(T, k, M, 6), torch.randn(T, k, device=DEV, generator=g)
    dout = torch.randn(T, H, device=DEV, generator=g)
    drows = torch.zeros_like(rows)
    a = [qm.moe_combine_rows(rows, slots, w), *qm.moe_combine_rows_grad(dout, rows, slots, w, drows=drows)]
    a = [t.clone() for t in a]
    for _ in range(5):
        b = [qm.moe_combine_rows(rows, slots, w), *qm.moe_combine_rows_grad(dout, rows, slots, w, drows=drows)]
        assert all(torch.equal(x, y) for x, y in zip(a, b))
