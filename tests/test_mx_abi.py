"""Refusals of the MXFP4 quantiser and products, without a GPU: the C entry points reject bad arguments before they touch a
device, and the binding rejects bad tensors."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from quantized_moe_expert_topk_amd import _lib as L
from tests.test_rows_abi import at, fake, ints


def call(name, **change):
    """The entry point on valid arguments with some of them changed; returns (status, text)."""
    v = {**dict(a=at(1), xs=at(2), b=at(3), ws=at(4), layout=0, off=at(5), cnt=None, E=8, M=64, rows=0, N=48, K=160, out=at(6),
                dt=1, slots=at(7), T=20, k=3, q=at(8), s=at(9)), **change}
    args = {
        "moe_quantize_mx": (v["a"], v["slots"], v["T"], v["k"], v["M"], v["K"], v["q"], v["s"], None),
        "moe_dequantize_mx": (v["a"], v["xs"], v["M"], v["K"], v["out"], v["dt"], None),
        "moe_mx_mm": (v["a"], v["xs"], v["b"], v["ws"], v["layout"], v["M"], v["N"], v["K"], v["out"], v["dt"], None),
        "moe_grouped_mx_mm": (v["a"], v["xs"], v["b"], v["ws"], v["layout"], v["off"], v["cnt"], v["E"], v["M"], v["rows"],
                              v["N"], v["K"], v["out"], v["dt"], None),
    }[name]
    rc = getattr(L.lib(), name)(*args)
    return rc, L.lib().moe_last_error().decode()


QUANT, DEQUANT, MM, GROUPED = "moe_quantize_mx", "moe_dequantize_mx", "moe_mx_mm", "moe_grouped_mx_mm"
EVERY, PRODUCTS, READ = (QUANT, DEQUANT, MM, GROUPED), (MM, GROUPED), (DEQUANT, MM, GROUPED)

REFUSED = [
    (EVERY, dict(a=None), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(a=at(1, 8)), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(M=-1), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(M=0x7FFFFC01), L.MOE_ERR_UNSUPPORTED),
    (EVERY, dict(K=0), L.MOE_ERR_INVALID_ARG),
    (EVERY, dict(K=144), L.MOE_ERR_UNSUPPORTED),
    (EVERY, dict(K=1 << 22), L.MOE_ERR_UNSUPPORTED),
    (READ, dict(xs=None), L.MOE_ERR_INVALID_ARG),
    (READ, dict(xs=at(2, 2)), L.MOE_ERR_INVALID_ARG),
    (READ, dict(out=None), L.MOE_ERR_INVALID_ARG),
    (READ, dict(out=at(6, 4)), L.MOE_ERR_INVALID_ARG),
    (READ, dict(out=at(1, 16)), L.MOE_ERR_INVALID_ARG),  # inside an operand
    (READ, dict(out=at(2, 64 * 8 - 16)), L.MOE_ERR_INVALID_ARG),  # over the last scales
    (READ, dict(dt=2), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(b=None), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(b=at(3, 8)), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(ws=None), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(ws=at(4, 1)), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(N=0), L.MOE_ERR_INVALID_ARG),
    (PRODUCTS, dict(N=1 << 22), L.MOE_ERR_UNSUPPORTED),
    (PRODUCTS, dict(layout=2), L.MOE_ERR_UNSUPPORTED),
    (PRODUCTS, dict(layout=1, N=40), L.MOE_ERR_UNSUPPORTED),
    ((GROUPED,), dict(off=None), L.MOE_ERR_INVALID_ARG),
    ((GROUPED,), dict(off=at(5, 2)), L.MOE_ERR_INVALID_ARG),
    ((GROUPED,), dict(cnt=at(6)), L.MOE_ERR_INVALID_ARG),  # the output over the counts
    ((GROUPED,), dict(E=0), L.MOE_ERR_INVALID_ARG),
    ((GROUPED,), dict(E=1025), L.MOE_ERR_UNSUPPORTED),
    ((GROUPED,), dict(rows=-1), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(T=-1), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(k=0), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(T=1 << 30, k=2), L.MOE_ERR_UNSUPPORTED),
    ((QUANT,), dict(slots=None), L.MOE_ERR_INVALID_ARG),  # k and M are of slots
    ((QUANT,), dict(slots=None, k=1), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(slots=at(7, 2)), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(q=None), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(q=at(8, 8)), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(s=None), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(s=at(9, 2)), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(s=at(8, 64 * 80 - 4)), L.MOE_ERR_INVALID_ARG),  # one output over the other
    ((QUANT,), dict(q=at(1)), L.MOE_ERR_INVALID_ARG),
    ((QUANT,), dict(s=at(7)), L.MOE_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("names,change,status", REFUSED, ids=lambda v: str(v)[:60])
def test_refused_before_the_device(names, change, status):
    for name in names:
        rc, text = call(name, **change)
        assert rc == status, (name, rc, text)
        assert text.startswith(name)


def test_no_rows_needs_no_arrays():
    none = dict(M=0, T=0, a=None, xs=None, b=None, ws=None, out=None, slots=None, k=1, q=None, s=None)
    for name in EVERY:
        assert call(name, **none)[0] == L.MOE_OK, name
    assert call(QUANT, M=0, q=None, s=None)[0] == L.MOE_OK  # tokens without rows


def u8(*shape):
    return fake(*shape, dtype=torch.uint8)


def bf(*shape):
    return fake(*shape, dtype=torch.bfloat16)


Q, S = (64, 80), (2, 64, 4)  # 64 rows of 160 columns
BAD = [
    (lambda: qm.moe_quantize_mx(fake(4, 64)), "x"),
    (lambda: qm.moe_quantize_mx(torch.zeros(4, 64, dtype=torch.bfloat16)), "x"),
    (lambda: qm.moe_quantize_mx(bf(8, 128)[:, ::2]), "x"),
    (lambda: qm.moe_quantize_mx(bf(4, 64).requires_grad_(), q=u8(4, 32), scale=u8(1, 4, 4)), "requires gradients"),
    (lambda: qm.moe_quantize_mx(bf(4, 64), ints(5, 2)), "slots"),
    (lambda: qm.moe_quantize_mx(bf(4, 64), q=u8(4, 64), scale=u8(1, 4, 4)), "q"),
    (lambda: qm.moe_quantize_mx(bf(4, 64), q=u8(4, 32), scale=u8(4, 2)), "scale"),
    (lambda: qm.moe_quantize_mx(bf(4, 64), ints(4, 2), q=u8(9, 32), scale=u8(1, 8, 4)), "scale"),
    (lambda: qm.moe_quantize_mx(bf(4, 64), ints(4, 2), rows=-1), "rows"),
    (lambda: qm.moe_quantize_mx(bf(4, 64), rows=8), "rows"),
    (lambda: qm.moe_dequantize_mx(u8(*Q), u8(64, 5), out=bf(64, 160)), "scale"),
    (lambda: qm.moe_dequantize_mx(u8(*Q), u8(*S), out=bf(64, 80)), "out"),
    (lambda: qm.moe_dequantize_mx(u8(*Q), u8(*S), out=fake(64, 160, dtype=torch.float16)), "out"),
    (lambda: qm.moe_mx_mm(u8(*Q), u8(*S), u8(48, 64), u8(2, 48, 4), out=bf(64, 48)), "wq"),
    (lambda: qm.moe_mx_mm(u8(*Q), u8(*S), u8(48, 80), u8(48, 5), out=bf(64, 48)), "ws"),  # a bank's scales need its layout
    (lambda: qm.moe_mx_mm(u8(*Q), u8(*S), u8(48, 80), u8(2, 48, 4), layout=1, out=bf(64, 48)), "ws"),
    (lambda: qm.moe_mx_mm(u8(*Q), u8(64, 5), u8(48, 80), u8(2, 48, 4), out=bf(64, 48)), "xs"),
    (lambda: qm.moe_mx_mm(u8(*Q), u8(*S), u8(48, 80), u8(2, 48, 4), out=bf(48, 64)), "out"),
    (lambda: qm.moe_grouped_mx_mm(u8(*Q), u8(*S), u8(4, 48, 80), u8(2, 4, 48, 4), ints(5), out=bf(64, 48)), "ws"),
    (lambda: qm.moe_grouped_mx_mm(u8(*Q), u8(*S), u8(4, 48, 80), u8(2, 192, 4), ints(4), out=bf(64, 48)), "offsets"),
    (lambda: qm.moe_grouped_mx_mm(u8(*Q), u8(*S), u8(4, 48, 80), u8(2, 192, 4), ints(5), ints(3), out=bf(64, 48)), "counts"),
]


@pytest.mark.parametrize("n", range(len(BAD)))
def test_binding_refuses(n):
    make, word = BAD[n]
    with pytest.raises(ValueError, match=word):
        make()
