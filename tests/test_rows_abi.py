"""Refusals of the calls that take rows to the experts and back, without a GPU: the C entry points reject bad arguments
before they touch a device, and the binding rejects bad tensors."""
import ctypes

import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from quantized_moe_expert_topk_amd import _lib as L


def at(n, more=0):
    """A distinct fake device address: validation never reads it."""
    return ctypes.c_void_p((n << 40) + more)


def call(name, **change):
    """The entry point on valid arguments with some of them changed; returns (status, text)."""
    v = {**dict(ids=at(1), T=5, k=2, sorted=at(2), M=64, off=at(3), cnt=None, E=8, slots=at(4), x=at(5), width=64, out=at(6),
                rt=0, ot=1, w=at(7), add=None, H=16, dout=at(8), dt=1, dw=at(9)), **change}
    args = {
        "moe_pair_slots": (v["ids"], v["T"], v["k"], v["sorted"], v["M"], v["off"], v["cnt"], v["E"], v["slots"], None),
        "moe_gather_rows": (v["x"], v["T"], v["k"], v["slots"], v["width"], v["M"], v["out"], None),
        "moe_combine_rows": (v["x"], v["rt"], v["slots"], v["w"], v["add"], v["T"], v["k"], v["M"], v["H"], v["out"],
                             v["ot"], None),
        "moe_combine_rows_grad": (v["dout"], v["dt"], v["x"], v["rt"], v["slots"], v["w"], v["T"], v["k"], v["M"], v["H"],
                                  v["out"], v["dw"], None),
    }[name]
    rc = getattr(L.lib(), name)(*args)
    return rc, L.lib().moe_last_error().decode()


SLOTS, GATHER, COMBINE, GRAD = "moe_pair_slots", "moe_gather_rows", "moe_combine_rows", "moe_combine_rows_grad"
EVERY, ROWS, WIDE = (SLOTS, GATHER, COMBINE, GRAD), (GATHER, COMBINE, GRAD), (COMBINE, GRAD)

REFUSED = [
    (EVERY, dict(T=-1), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(k=0), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(T=1 << 30, k=2), L.MOE_ERR_UNSUPPORTED),
    (EVERY, dict(M=-1), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(M=0x7FFFFC01), L.MOE_ERR_UNSUPPORTED),
    (EVERY, dict(slots=None), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(slots=at(4, 2)), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(ids=None), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(ids=at(1, 1)), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(sorted=None), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(sorted=at(2, 2)), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(off=None), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(off=at(3, 2)), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(cnt=at(10, 2)), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(E=0), L.MOE_ERR_INVALID_ARG),
    ((SLOTS,), dict(E=1025), L.MOE_ERR_UNSUPPORTED),
    ((SLOTS,), dict(slots=at(1, 36)), L.MOE_ERR_INVALID_ARG),  # over the last id
    ((SLOTS,), dict(slots=at(3, 32)), L.MOE_ERR_INVALID_ARG),  # over the last offset
    ((SLOTS,), dict(cnt=at(10), slots=at(10)), L.MOE_ERR_INVALID_ARG),
    (ROWS, dict(x=None), L.MOE_ERR_INVALID_ARG),
    (ROWS, dict(x=at(5, 8)), L.MOE_ERR_INVALID_ARG),
    (ROWS, dict(out=None), L.MOE_ERR_INVALID_ARG),
    (ROWS, dict(out=at(6, 8)), L.MOE_ERR_INVALID_ARG),
    (ROWS, dict(out=at(5, 64)), L.MOE_ERR_INVALID_ARG),  # inside an operand
    (ROWS, dict(out=at(4, 32)), L.MOE_ERR_INVALID_ARG),  # over the slots
    ((GATHER,), dict(width=0), L.MOE_ERR_INVALID_ARG),
    ((GATHER,), dict(width=24), L.MOE_ERR_UNSUPPORTED),
    ((GATHER,), dict(width=1 << 24), L.MOE_ERR_UNSUPPORTED),
    (WIDE, dict(H=0), L.MOE_ERR_INVALID_ARG),
    (WIDE, dict(H=12), L.MOE_ERR_UNSUPPORTED),
    (WIDE, dict(H=1 << 22), L.MOE_ERR_UNSUPPORTED),
    (WIDE, dict(rt=2), L.MOE_ERR_INVALID_ARG),
    ((COMBINE,), dict(ot=2), L.MOE_ERR_INVALID_ARG),
    ((GRAD,), dict(dt=-1), L.MOE_ERR_INVALID_ARG),
    (WIDE, dict(w=at(7, 2)), L.MOE_ERR_INVALID_ARG),
    ((GRAD,), dict(w=None), L.MOE_ERR_INVALID_ARG),
    ((COMBINE,), dict(add=at(10, 8)), L.MOE_ERR_INVALID_ARG),
    ((COMBINE,), dict(add=at(6)), L.MOE_ERR_INVALID_ARG),  # in place
    ((GRAD,), dict(dout=None), L.MOE_ERR_INVALID_ARG),
    ((GRAD,), dict(dout=at(8, 4)), L.MOE_ERR_INVALID_ARG),
    ((GRAD,), dict(dw=None), L.MOE_ERR_INVALID_ARG),
    ((GRAD,), dict(dw=at(9, 2)), L.MOE_ERR_INVALID_ARG),
    ((GRAD,), dict(dw=at(6, 8)), L.MOE_ERR_INVALID_ARG),  # one output over the other
    ((GRAD,), dict(dw=at(7)), L.MOE_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("names,change,status", REFUSED, ids=lambda v: str(v)[:60])
def test_refused_before_the_device(names, change, status):
    for name in names:
        rc, text = call(name, **change)
        assert rc == status, (name, rc, text)
        assert text.startswith(name)


def test_no_tokens_needs_no_arrays():
    none = dict(T=0, ids=None, slots=None, x=None, out=None, w=None, dout=None, dw=None)
    for name in EVERY:
        assert call(name, **none)[0] == L.MOE_OK, name
    assert call(GATHER, M=0, out=None)[0] == L.MOE_OK  # no rows to write


class OnCuda(torch.Tensor):
    """A host tensor that says it is on a GPU: enough for the checks before a call."""
    @property
    def device(self):
        return torch.device("cuda", 0)


def fake(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnCuda)


def ints(*shape):
    return fake(*shape, dtype=torch.int32)


BAD = [
    (lambda: qm.moe_pair_slots(ints(4, 2).long().as_subclass(OnCuda), ints(16), ints(5)), "topk_ids"),
    (lambda: qm.moe_pair_slots(ints(8), ints(16), ints(5)), "topk_ids"),
    (lambda: qm.moe_pair_slots(ints(4, 2), ints(4, 4), ints(5)), "sorted_ids"),
    (lambda: qm.moe_pair_slots(ints(4, 2), ints(32)[::2], ints(5)), "sorted_ids"),
    (lambda: qm.moe_pair_slots(ints(4, 2), ints(16), ints(5, 2)), "offsets"),
    (lambda: qm.moe_pair_slots(ints(4, 2), ints(16), ints(3), ints(4)), "offsets"),
    (lambda: qm.moe_pair_slots(ints(4, 2), ints(16), ints(5), ints(4), slots=ints(4, 3)), "slots"),
    (lambda: qm.moe_gather_rows(torch.zeros(4, 8), ints(4, 2)), "x"),
    (lambda: qm.moe_gather_rows(fake(4, 8), ints(3, 2)), "slots"),
    (lambda: qm.moe_gather_rows(fake(4, 8), ints(2, 4).t()), "slots"),
    (lambda: qm.moe_gather_rows(fake(4, 8), ints(4, 2), rows=-1), "rows"),
    (lambda: qm.moe_gather_rows(fake(4, 8), ints(4, 2), out=fake(8, 16)), "out"),
    (lambda: qm.moe_gather_rows(fake(4, 8), ints(4, 2), out=fake(8, 8, dtype=torch.bfloat16)), "out"),
    (lambda: qm.moe_gather_rows(fake(4, 8).requires_grad_(), ints(4, 2)), "requires gradients"),
    (lambda: qm.moe_combine_rows(fake(8, 8, dtype=torch.float16), ints(4, 2)), "rows"),
    (lambda: qm.moe_combine_rows(fake(8, 8), ints(4, 2), fake(4, 3)), "weights"),
    (lambda: qm.moe_combine_rows(fake(8, 8), ints(4, 2), fake(4, 2, dtype=torch.bfloat16)), "weights"),
    (lambda: qm.moe_combine_rows(fake(8, 8), ints(4, 2), add=fake(4, 8), out=fake(4, 8, dtype=torch.bfloat16)), "add"),
    (lambda: qm.moe_combine_rows(fake(8, 8), ints(4, 2), out=fake(4, 16)), "out"),
    (lambda: qm.moe_combine_rows(fake(8, 8), ints(4, 2), out=fake(4, 8), out_dtype=torch.bfloat16), "out"),
    (lambda: qm.moe_combine_rows(fake(8, 8).requires_grad_(), ints(4, 2), out=fake(4, 8)), "requires gradients"),
    (lambda: qm.moe_combine_rows(fake(8, 8), ints(4, 2), fake(4, 2).requires_grad_(), out=fake(4, 8)), "requires gradients"),
    (lambda: qm.moe_combine_rows_grad(fake(4, 8), fake(8, 16), ints(4, 2), fake(4, 2)), "rows"),
    (lambda: qm.moe_combine_rows_grad(fake(4, 8), fake(8, 8), ints(5, 2), fake(5, 2)), "slots"),
    (lambda: qm.moe_combine_rows_grad(fake(4, 8), fake(8, 8), ints(4, 2), fake(4, 2), drows=fake(7, 8),
                                      dweights=fake(4, 2)), "drows"),
    (lambda: qm.moe_combine_rows_grad(fake(4, 8), fake(8, 8), ints(4, 2), fake(4, 2), drows=fake(8, 8),
                                      dweights=fake(4, 2, dtype=torch.bfloat16)), "dweights"),
]


@pytest.mark.parametrize("n", range(len(BAD)))
def test_binding_refuses(n):
    make, word = BAD[n]
    with pytest.raises(ValueError, match=word):
        make()
