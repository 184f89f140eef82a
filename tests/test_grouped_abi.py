"""Refusals of the grouped products, the block quantiser and the fp8 block products, without a GPU: the C entry
points reject bad arguments before they touch a device, and the binding rejects bad tensors."""
import ctypes

import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from quantized_moe_expert_topk_amd import _lib as L


def at(n):
    """A distinct fake device address: validation never reads it."""
    return ctypes.c_void_p(n << 40)


def call(name, **change):
    """The entry point on valid arguments with some of them changed; returns (status, text)."""
    base = dict(a=at(1), b=at(2), off=at(3), cnt=None, E=8, M=64, rows=0, N=64, K=128, out=at(4), dt=1, acc=0,
                xs=at(5), ws=at(6), layout=0)
    v = {**base, **change}
    g = (v["off"], v["cnt"], v["E"], v["M"], v["rows"])
    args = {
        "moe_grouped_mm": (v["a"], v["b"], *g, v["N"], v["K"], v["out"], v["dt"], None),
        "moe_grouped_mm_dgrad": (v["a"], v["b"], *g, v["N"], v["K"], v["out"], v["dt"], None),
        "moe_grouped_mm_wgrad": (v["a"], v["b"], *g, v["N"], v["K"], v["out"], v["dt"], v["acc"], None),
        "moe_quantize_blocks": (v["a"], v["M"], v["K"], v["out"], v["xs"], None),
        "moe_block_mm": (v["a"], v["xs"], v["b"], v["ws"], v["layout"], v["M"], v["N"], v["K"], v["out"], v["dt"], None),
        "moe_grouped_block_mm": (v["a"], v["xs"], v["b"], v["ws"], v["layout"], *g, v["N"], v["K"], v["out"], v["dt"], None),
    }[name]
    rc = getattr(L.lib(), name)(*args)
    return rc, L.lib().moe_last_error().decode()


GROUPED = ("moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad", "moe_grouped_block_mm")
BF16 = GROUPED[:3]
FP8 = ("moe_block_mm", "moe_grouped_block_mm")
PRODUCTS = (*GROUPED, "moe_block_mm")
EVERY = (*PRODUCTS, "moe_quantize_blocks")

REFUSED = [
    (EVERY, dict(a=None), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(b=None), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(out=None), L.MOE_ERR_INVALID_ARG),
    (GROUPED, dict(off=None), L.MOE_ERR_INVALID_ARG),
    (GROUPED, dict(off=ctypes.c_void_p((3 << 40) + 2)), L.MOE_ERR_INVALID_ARG),
    (GROUPED, dict(cnt=ctypes.c_void_p((7 << 40) + 1)), L.MOE_ERR_INVALID_ARG),
    (GROUPED, dict(cnt=at(4)), L.MOE_ERR_INVALID_ARG),  # the output over the counts
    (GROUPED, dict(E=0), L.MOE_ERR_INVALID_ARG),
    (GROUPED, dict(E=1025), L.MOE_ERR_UNSUPPORTED),
    (GROUPED, dict(rows=-1), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(M=-1), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(N=0), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(K=0), L.MOE_ERR_INVALID_ARG),
    (BF16, dict(N=60), L.MOE_ERR_UNSUPPORTED),
    (BF16, dict(K=132), L.MOE_ERR_UNSUPPORTED),
    ((*FP8, "moe_quantize_blocks"), dict(K=136), L.MOE_ERR_UNSUPPORTED),
    (PRODUCTS, dict(K=1 << 22), L.MOE_ERR_UNSUPPORTED),
    (PRODUCTS, dict(N=1 << 22), L.MOE_ERR_UNSUPPORTED),
    (PRODUCTS, dict(dt=2), L.MOE_ERR_INVALID_ARG),
    (("moe_grouped_mm_wgrad",), dict(acc=1, dt=1), L.MOE_ERR_UNSUPPORTED),
    (FP8, dict(layout=2), L.MOE_ERR_UNSUPPORTED),
    (FP8, dict(layout=1, N=72), L.MOE_ERR_UNSUPPORTED),
    ((*FP8, "moe_quantize_blocks"), dict(xs=None), L.MOE_ERR_INVALID_ARG),
    (FP8, dict(ws=None), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(a=ctypes.c_void_p((1 << 40) + 8)), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(b=ctypes.c_void_p((2 << 40) + 2)), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(out=ctypes.c_void_p((4 << 40) + 4)), L.MOE_ERR_INVALID_ARG),
    (FP8, dict(xs=ctypes.c_void_p((5 << 40) + 2)), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(out=ctypes.c_void_p((1 << 40) + 16)), L.MOE_ERR_INVALID_ARG),  # inside an operand
    (PRODUCTS, dict(out=ctypes.c_void_p((2 << 40) + 64)), L.MOE_ERR_INVALID_ARG),
    (("moe_quantize_blocks",), dict(xs=at(4)), L.MOE_ERR_INVALID_ARG),  # codes and scales in one place
]


@pytest.mark.parametrize("names,change,status", REFUSED, ids=lambda v: str(v)[:60])
def test_refused_before_the_device(names, change, status):
    for name in names:
        rc, text = call(name, **change)
        assert rc == status, (name, rc, text)
        assert text.startswith(name), text


@pytest.mark.parametrize("name", EVERY)
def test_no_rows_need_no_device(name):
    """Nothing to do is a success without a device and with NULL matrices; wgrad without accumulate still has its
    zeros to write and is left out."""
    if name == "moe_grouped_mm_wgrad":
        assert call(name, M=0, a=None, b=None, acc=1, dt=0)[0] == L.MOE_OK
    else:
        assert call(name, M=0, a=None, b=None, xs=None, ws=None, out=None)[0] == L.MOE_OK


def test_binding_rejects_tensors():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    codes, f32 = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(1, 4)
    for f in (lambda: qm.moe_grouped_mm(x, w, off), lambda: qm.moe_grouped_mm_dgrad(x, w, off),
              lambda: qm.moe_grouped_mm_wgrad(x, x, off), lambda: qm.moe_quantize_blocks(x),
              lambda: qm.moe_block_mm(codes, f32, codes, f32),
              lambda: qm.moe_grouped_block_mm(codes, f32, codes[None], f32[None], off)):
        with pytest.raises(ValueError, match="cuda"):
            f()
    with pytest.raises(ValueError, match="dimensions"):
        qm.moe_grouped_mm(x[0], w, off)


def test_binding_checks_types_shapes_and_order():
    from quantized_moe_expert_topk_amd import grouped as G
    dev = torch.device("cpu")
    t = torch.zeros(4, 16, dtype=torch.bfloat16)
    for bad in (t.float(), t[:, ::2], t.t(), torch.zeros(16, 4, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="expected contiguous"):
            G._operand(bad, (torch.bfloat16,), (4, 16), dev, "x")
    for off, cnt in ((torch.zeros(3), None), (torch.zeros(2, dtype=torch.int32), None),
                     (torch.zeros(6, dtype=torch.int32)[::2], None),
                     (torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            G._ranges(off, cnt, 2, dev)
    G._ranges(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2, dev)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        G._output(torch.zeros(4, 4, dtype=torch.float16), None, (4, 4), dev)
    with pytest.raises(ValueError, match="out"):
        G._output(torch.zeros(4, 4), torch.bfloat16, (4, 4), dev)
