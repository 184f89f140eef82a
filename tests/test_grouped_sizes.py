"""Sizes that do not fit the C interface's 32-bit integers, and row ranges without experts, are refused by the binding
(a C integer would take their low bits): checked on tensors without memory."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from quantized_moe_expert_topk_amd import grouped as G


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32 + 5])
def test_more_rows_than_an_integer_holds(rows):
    off = torch.zeros(3, dtype=torch.int32)
    w, wq = meta(2, 8, 16), meta(2, 8, 16, dtype=torch.uint8)
    calls = [lambda: qm.moe_grouped_mm(meta(rows, 16), w, off), lambda: qm.moe_grouped_mm_dgrad(meta(rows, 8), w, off),
             lambda: qm.moe_grouped_mm_wgrad(meta(rows, 8), meta(rows, 16), off), lambda: qm.moe_quantize_blocks(meta(rows, 16)),
             lambda: qm.moe_block_mm(meta(rows, 16, dtype=torch.uint8), meta(1, rows), wq[0], meta(1, 1)),
             lambda: qm.moe_grouped_block_mm(meta(rows, 16, dtype=torch.uint8), meta(1, rows), wq, meta(2, 1, 1), off),
             lambda: qm.moe_quantize_blocks(meta(2, rows)), lambda: G._matrix(meta(2, rows, 16), 3, "w")]
    for call in calls:
        with pytest.raises(ValueError, match="too large"):
            call()


@pytest.mark.parametrize("rows,passed", [(None, 7), (0, 0), (5, 5), (10 ** 9, 10 ** 9), (2 ** 32, 2 ** 31 - 1), (2 ** 31 + 3, 2 ** 31 - 1),
                                         (-1, -1), (-2 ** 32, -1)])
def test_expected_rows_keeps_its_meaning(rows, passed):
    """A hint past 32 bits is as many rows as there can be, and a negative one stays negative (and is refused)."""
    assert G._rows_hint(rows, 7) == passed


@pytest.mark.parametrize("off,cnt", [(torch.zeros(0, dtype=torch.int32), None), (torch.zeros(1, dtype=torch.int32), None),
                                     (torch.zeros((), dtype=torch.int32), None),
                                     (torch.zeros(3, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)),
                                     (torch.zeros(3, dtype=torch.int32), torch.zeros((), dtype=torch.int32))])
def test_ranges_without_experts(off, cnt):
    """The number of experts of a weight gradient comes from its ranges."""
    with pytest.raises(ValueError, match="at least one expert"):
        G._experts(off, cnt)
    assert G._experts(torch.zeros(3, dtype=torch.int32), None) == 2
    assert G._experts(torch.zeros(9, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)) == 4
