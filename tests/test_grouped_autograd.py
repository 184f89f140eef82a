"""Autograd and the grouped products: a tensor that requires gradients is refused while they are recorded, and
torch.autograd.Function's methods can call all of them."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from quantized_moe_expert_topk_amd import grouped as G


def test_tensors_that_require_gradients_are_refused():
    t = torch.zeros(4, 16, requires_grad=True)
    args = (torch.float32,), (4, 16), torch.device("cpu"), "x"
    with pytest.raises(ValueError, match="x: requires gradients"):
        G._operand(t, *args)
    with torch.no_grad():
        assert G._operand(t, *args) == t.data_ptr()
    assert G._operand(t.detach(), *args) == t.data_ptr()


@pytest.mark.gpu
def test_calls_refuse_what_they_would_not_record():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, dy = torch.zeros(4, 16, **bf), torch.zeros(2, 8, 16, **bf), torch.zeros(4, 8, **bf)
    leaf = lambda t: t.clone().requires_grad_()
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    xq, xs = qm.moe_quantize_blocks(x)
    wq, ws = torch.zeros(2, 8, 16, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, 1, device="cuda")
    calls = [lambda: qm.moe_grouped_mm(leaf(x), w, off), lambda: qm.moe_grouped_mm(x, leaf(w), off),
             lambda: qm.moe_grouped_mm_dgrad(leaf(dy), w, off), lambda: qm.moe_grouped_mm_dgrad(dy, leaf(w), off),
             lambda: qm.moe_grouped_mm_wgrad(leaf(dy), x, off), lambda: qm.moe_grouped_mm_wgrad(dy, leaf(x), off),
             lambda: qm.moe_grouped_mm(x, w, off, out=leaf(dy)), lambda: qm.moe_quantize_blocks(leaf(x)),
             lambda: qm.moe_block_mm(xq, leaf(xs), wq[0], ws[0]), lambda: qm.moe_block_mm(xq, xs, wq[0], leaf(ws[0])),
             lambda: qm.moe_grouped_block_mm(xq, xs, wq, leaf(ws), off)]
    for call in calls:
        with pytest.raises(ValueError, match="requires gradients"):
            call()
        with torch.no_grad():
            call()


@pytest.mark.gpu
def test_a_function_made_of_the_products():
    """Forward and both gradients inside torch.autograd.Function, rows of nobody zero: integers, so exact."""
    class Mm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, off, cnt):
            ctx.save_for_backward(x, w, off, cnt)
            return qm.moe_grouped_mm(x, w, off, cnt, out=torch.zeros(x.shape[0], w.shape[1], device=x.device))

        @staticmethod
        def backward(ctx, dy):
            x, w, off, cnt = ctx.saved_tensors
            dy = dy.to(torch.bfloat16).contiguous()
            return (qm.moe_grouped_mm_dgrad(dy, w, off, cnt, out=torch.zeros_like(x)),
                    qm.moe_grouped_mm_wgrad(dy, x, off, cnt), None, None)

    g = torch.Generator(device="cuda").manual_seed(0)
    ints = lambda *s: torch.randint(-1, 2, s, device="cuda", generator=g).to(torch.bfloat16)
    x, w, dy = ints(50, 24), ints(3, 16, 24), ints(50, 16)
    off = torch.tensor([2, 20, 20], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([15, 0, 27], dtype=torch.int32, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x, w)]
    Mm.apply(*leaves, off, cnt).backward(dy.float())
    dx, dw = torch.zeros(50, 24, dtype=torch.float64, device="cuda"), torch.zeros(3, 16, 24, dtype=torch.float64, device="cuda")
    for e, r in ((0, slice(2, 17)), (2, slice(20, 47))):  # sums of at most 27 products of +-1: exact in bf16
        dx[r], dw[e] = dy[r].double() @ w[e].double(), dy[r].double().t() @ x[r].double()
    assert torch.equal(leaves[0].grad.double(), dx) and torch.equal(leaves[1].grad.double(), dw)
