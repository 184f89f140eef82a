"""Calls with ``stream=S`` and no output or workspace: what the binding allocates belongs to S.

Each call is made twice.  First with work queued on the current stream that will still write a block freed there (a
sleep, then a fill): an output that took that block would be overwritten by the fill.  Then with S asleep, so that the
call's kernels run late: memory that the call took from the current stream's pool and gave back would by then belong to
a new tensor there, and the kernels would write into it.  The queued fills and kernels are ordinary work inside live
allocations of the process; only values can come out wrong.
"""
import ctypes

import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import fp8_rows, fp8_weights, gen, ints, ranges

pytestmark = pytest.mark.gpu

DEV = "cuda"
SLEEP = 100_000_000  # cycles: some tens of milliseconds at least


def grouped_inputs():
    N, K = 1024, 512
    off, cnt, M = ranges([300, 0, 257, 467])
    g = gen(1)
    x, w, dy = ints(g, M, K), ints(g, 4, N, K), ints(g, M, N)
    xq, xs = fp8_rows(g, M, K, "ints")
    wq, ws = fp8_weights(g, 4, N, K, "ints")
    return {
        "moe_grouped_mm": lambda s: [qm.moe_grouped_mm(x, w, off, cnt, stream=s)],
        "moe_grouped_mm_dgrad": lambda s: [qm.moe_grouped_mm_dgrad(dy, w, off, cnt, stream=s)],
        "moe_grouped_mm_wgrad": lambda s: [qm.moe_grouped_mm_wgrad(dy, x, off, cnt, stream=s)],
        "moe_quantize_blocks": lambda s: list(qm.moe_quantize_blocks(x, stream=s)),
        "moe_block_mm": lambda s: [qm.moe_block_mm(xq, xs, wq[0], ws[0], stream=s)],
        "moe_grouped_block_mm": lambda s: [qm.moe_grouped_block_mm(xq, xs, wq, ws, off, cnt, stream=s)],
    }


def bits(ts):
    return [t.contiguous().view(torch.uint8) for t in ts]


def check_on_another_stream(call, raw, extra=()):
    """`extra`: sizes in bytes of temporary memory that the call takes besides its outputs."""
    S = torch.cuda.Stream()
    handle = S.cuda_stream if raw else S
    want = [t.clone() for t in bits(call(None))]
    sizes = [t.numel() for t in want] + list(extra)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda._sleep(SLEEP)
    for t in old:
        t.fill_(0xFF)
    del old, t
    got = call(handle)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(got), want)), "written by the current stream's earlier work"
    del got
    torch.cuda.empty_cache()
    with torch.cuda.stream(S):
        torch.cuda._sleep(SLEEP)
    got = call(handle)
    del got
    new = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x55) for n in sizes]
    torch.cuda.synchronize()
    assert all(bool((t == 0x55).all()) for t in new), "the call wrote into memory given to other work"


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", ["moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad",
                                       "moe_quantize_blocks", "moe_block_mm", "moe_grouped_block_mm"])
def test_outputs_belong_to_the_stream_of_the_call(name, raw):
    check_on_another_stream(grouped_inputs()[name], raw)


@pytest.mark.parametrize("handle", [0, ctypes.c_void_p(0), ctypes.c_void_p(None)], ids=["0", "pointer 0", "pointer None"])
def test_a_null_handle_is_the_default_stream(handle):
    """A raw handle of 0 names the default stream, for the kernels and for what the call allocates."""
    from quantized_moe_expert_topk_amd._streams import allocating_on
    call = grouped_inputs()["moe_grouped_mm"]
    want = call(None)[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with allocating_on(handle, torch.device("cuda", torch.cuda.current_device())):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        got = call(handle)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def layer_inputs():
    from synth import synth as S
    from tests.gpu_util import bf16_dev, device_bank
    T = 75
    cfg = S.LayerConfig(91, "small layer", "bf16", 256, 8, 2, 256, False, (T,), ((0, 256),))
    inp = S.layer_inputs(cfg, T)
    x, router, bank, rows = bf16_dev(inp.x), bf16_dev(inp.router), device_bank(inp.routed), device_bank(inp.routed, packed=False)
    logits, ids, wts, al = qm.moe_route_align(x, router, None, cfg.k, 16)

    def aligned(a):
        """The parts of an alignment that are written whatever the routing."""
        return [a.counts, a.offsets, a.total_padded]

    def route_align(s):
        *r, a = qm.moe_route_align(x, router, None, cfg.k, 16, stream=s)
        return [*r, *aligned(a)]

    def packed(s):
        b = qm.moe_pack_bank(rows, stream=s)
        return [b.gate_up, b.down]

    return {
        "moe_pack_bank": (packed, 0),
        "moe_route": (lambda s: list(qm.moe_route(x, router, None, cfg.k, stream=s)),
                      qm.moe_route_workspace_bytes(T, cfg.H, cfg.E)),
        "moe_route_from_logits": (lambda s: list(qm.moe_route_from_logits(logits, cfg.k, stream=s)), 0),
        "moe_align": (lambda s: aligned(qm.moe_align(ids, cfg.E, 16, stream=s)), qm.moe_align_workspace_bytes(T, cfg.k, cfg.E)),
        "moe_route_align": (route_align, qm.moe_route_align_workspace_bytes(T, cfg.H, cfg.E, cfg.k)),
        "moe_expert_forward": (lambda s: [qm.moe_expert_forward(bank, None, x, wts, al, 0, cfg.I, stream=s)],
                               qm.moe_workspace_bytes(bank, None, T, cfg.k, 16, 0, cfg.I)),
    }


@pytest.mark.parametrize("name", ["moe_pack_bank", "moe_route", "moe_route_from_logits", "moe_align", "moe_route_align",
                                  "moe_expert_forward"])
def test_memory_of_the_layer_calls_belongs_to_their_stream(name):
    call, workspace = layer_inputs()[name]
    check_on_another_stream(call, False, [workspace] if workspace else [])
