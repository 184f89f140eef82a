"""Calls of the rows' way and of MXFP4 with ``stream=S`` and no outputs: what the binding allocates belongs to S (as
tests/test_gpu_streams.py checks it for the other calls), and calls in flight at once on two streams."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import gen
from tests.test_gpu_mx import ROWS, group, operand, weights
from tests.test_gpu_rows import aligned, routing, some_slots
from tests.test_gpu_streams import check_on_another_stream

pytestmark = pytest.mark.gpu

DEV = "cuda"


def calls():
    T, k, H, E, N = 256, 4, 1024, 8, 512
    M, g = T * k, gen(5)
    ids = routing(T, k, E)
    al = aligned(ids, E)
    tid = torch.from_numpy(ids).to(DEV)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    rows = torch.randn(M, H, device=DEV, generator=g).to(torch.bfloat16)
    slots, w = some_slots(T, k, M, 5, lost=0.0), torch.rand(T, k, device=DEV, generator=g)  # every row has its pair
    xq, xb = operand(g, M, H, "binades")
    xs = group(xb)
    wq, ws, _ = weights(g, 1, N, H, "binades", ROWS)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    return {
        "moe_pair_slots": lambda s: [qm.moe_pair_slots(tid, al.sorted_ids, al.offsets, al.counts, stream=s)],
        "moe_gather_rows": lambda s: [qm.moe_gather_rows(x, slots, stream=s)],
        "moe_combine_rows": lambda s: [qm.moe_combine_rows(rows, slots, w, stream=s)],
        "moe_combine_rows_grad": lambda s: list(qm.moe_combine_rows_grad(x, rows, slots, w, stream=s)),
        "moe_quantize_mx": lambda s: list(qm.moe_quantize_mx(x, stream=s)),
        "moe_quantize_mx to slots": lambda s: list(qm.moe_quantize_mx(x, slots, stream=s)),
        "moe_dequantize_mx": lambda s: [qm.moe_dequantize_mx(xq, xs, stream=s)],
        "moe_mx_mm": lambda s: [qm.moe_mx_mm(xq, xs, wq[0], ws, stream=s)],
        "moe_grouped_mx_mm": lambda s: [qm.moe_grouped_mx_mm(xq, xs, wq, ws, off, stream=s)],
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["moe_pair_slots", "moe_gather_rows", "moe_combine_rows", "moe_combine_rows_grad",
                                  "moe_quantize_mx", "moe_quantize_mx to slots", "moe_dequantize_mx", "moe_mx_mm",
                                  "moe_grouped_mx_mm"])
def test_outputs_belong_to_the_stream(name, raw):
    check_on_another_stream(calls()[name], raw)


def test_two_streams_at_once():
    """Every call on two streams in flight together gives what it gives alone."""
    made = calls()
    want = {n: [t.clone() for t in f(None)] for n, f in made.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append({n: f(None) for n, f in made.items()})
    torch.cuda.synchronize()
    for one in got:
        for n, outs in one.items():
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want[n])), n
