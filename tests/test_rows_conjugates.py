"""Rows of complex numbers: torch conjugates a tensor lazily, by a flag beside bytes that stay as they were.  The rows are moved
by their bytes, so such a view is refused on either side (without a GPU: a refusal comes before the call)."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_rows_abi import fake, ints


def complex_rows(*shape):
    return fake(*shape, dtype=torch.complex64)


def test_a_lazily_conjugated_operand_is_refused():
    x = complex_rows(4, 8).conj()
    assert x.is_conj() and x.is_contiguous()
    with pytest.raises(ValueError, match="x: .*conjugate"):
        qm.moe_gather_rows(x, ints(4, 2), out=complex_rows(8, 8))


def test_a_lazily_conjugated_output_is_refused():
    with pytest.raises(ValueError, match="out: .*conjugate"):
        qm.moe_gather_rows(complex_rows(4, 8), ints(4, 2), out=complex_rows(8, 8).conj())


@pytest.mark.gpu
def test_rows_of_complex_numbers():
    x = torch.randn(5, 16, dtype=torch.complex64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    slots = torch.tensor([[3, -1], [9, 0], [1, 2], [8, 4], [5, 6]], dtype=torch.int32, device="cuda")
    for rows in (x, x.conj().resolve_conj()):
        got = qm.moe_gather_rows(rows, slots)
        for t, pair in enumerate(slots.tolist()):
            for s in pair:
                if s >= 0:
                    assert torch.equal(got[s], rows[t])
