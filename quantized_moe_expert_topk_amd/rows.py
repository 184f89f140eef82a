"""Python binding of the calls of ``include/qmoe.h`` that take token rows to their experts' row ranges and back:
argument checks and marshalling only.

``slots`` int32 [T, k] holds the row of every pair (token, choice) in the row matrices, as :func:`moe_pair_slots` makes
it of an alignment; a value outside the row matrix stands for a pair without a row.  Rows of no pair are left as they are
in an output that is passed, and undefined in one allocated here.  Streams, devices and autograd as in
:mod:`~quantized_moe_expert_topk_amd.grouped`.
"""
from __future__ import annotations

import torch

from ._streams import allocating_on
from .grouped import _INT_MAX, _OUT, _call, _matrix, _operand, _output, _ranges

_I32, _F32, _ROWS = (torch.int32,), (torch.float32,), (torch.float32, torch.bfloat16)


def _pairs(slots: torch.Tensor, T: int | None, device) -> tuple[int, int, int]:
    """(T, k, address) of a slots tensor of T tokens."""
    shape = _matrix(slots, 2, "slots")
    p = _operand(slots, _I32, shape if T is None else (T, shape[1]), device, "slots")
    return shape[0], shape[1], p


def _empty(shape, dtype, device, stream):
    with allocating_on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def moe_pair_slots(topk_ids: torch.Tensor, sorted_ids: torch.Tensor, offsets: torch.Tensor,
                   counts: torch.Tensor | None = None, slots: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The place of every pair in ``sorted_ids``, -1 for a pair that has none.  topk_ids int32 [T, k]; sorted_ids,
    offsets and counts as :func:`moe_align` gives them -> int32 [T, k]."""
    T, k = _matrix(topk_ids, 2, "topk_ids")
    dev = topk_ids.device
    ids = _operand(topk_ids, _I32, (T, k), dev, "topk_ids")
    M, = _matrix(sorted_ids, 1, "sorted_ids")
    E = counts.shape[0] if counts is not None and counts.dim() == 1 else max(offsets.numel() - 1, 0)
    off, cnt = _ranges(offsets, counts, E, dev)
    at = _operand(sorted_ids, _I32, (M,), dev, "sorted_ids")
    if slots is None:
        slots = _empty((T, k), torch.int32, dev, stream)
    _call("moe_pair_slots", dev, stream, ids, T, k, at, M, off, cnt, E, _operand(slots, _I32, (T, k), dev, "slots"))
    return slots


def _room(rows: int | None, out: torch.Tensor | None, T: int, k: int) -> int:
    """Rows of a row matrix that is allocated here, or passed."""
    if out is not None:
        return out.shape[0]
    if rows is None:
        return T * k
    if not 0 <= rows <= _INT_MAX:
        raise ValueError(f"rows: {rows} is not a number of rows")
    return rows


def moe_gather_rows(x: torch.Tensor, slots: torch.Tensor, rows: int | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """out[slots[t, j]] = x[t] for every pair.  x [T, H] of any type, rows of whole 16 bytes -> [rows, H] (``rows``: that
    of ``out``, else T * k).  Its gradient for x is :func:`moe_combine_rows` of the rows' gradients, without weights."""
    T, H = _matrix(x, 2, "x")
    dev = x.device
    px = _operand(x, (x.dtype,), (T, H), dev, "x")
    _, k, ps = _pairs(slots, T, dev)
    if out is not None:
        _matrix(out, 2, "out")
    M = _room(rows, out, T, k)
    if out is None:
        out = _empty((M, H), x.dtype, dev, stream)
    width = H * x.element_size()
    if width > _INT_MAX:
        raise ValueError(f"x: rows of {width} bytes are too large for 32-bit sizes")
    _call("moe_gather_rows", dev, stream, px, T, k, ps, width, M, _operand(out, (x.dtype,), (M, H), dev, "out"))
    return out


def moe_combine_rows(rows: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                     add: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * rows[slots[t, j]].  rows [M, H] bf16 or f32, weights f32 [T, k] (None:
    ones), add [T, H] of out's type -> [T, H] of ``out_dtype`` (rows' type if None)."""
    M, H = _matrix(rows, 2, "rows")
    dev = rows.device
    pr = _operand(rows, _ROWS, (M, H), dev, "rows")
    T, k, ps = _pairs(slots, None, dev)
    pw = _operand(weights, _F32, (T, k), dev, "weights") if weights is not None else None
    out, po, code = _output(out, out_dtype or (rows.dtype if out is None else None), (T, H), dev, stream)
    pa = _operand(add, (out.dtype,), (T, H), dev, "add") if add is not None else None
    _call("moe_combine_rows", dev, stream, pr, _OUT[rows.dtype], ps, pw, pa, T, k, M, H, po, code)
    return out


def moe_combine_rows_grad(dout: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
                          drows: torch.Tensor | None = None, dweights: torch.Tensor | None = None, stream=None):
    """The gradients of :func:`moe_combine_rows` with weights: drows[slots[t, j]] = weights[t, j] * dout[t] (of rows' shape
    and type) and dweights[t, j] = <rows[slots[t, j]], dout[t]> (f32 [T, k], 0 for pairs without a row)."""
    T, H = _matrix(dout, 2, "dout")
    M, _ = _matrix(rows, 2, "rows")
    dev = dout.device
    pd = _operand(dout, _ROWS, (T, H), dev, "dout")
    pr = _operand(rows, _ROWS, (M, H), dev, "rows")
    _, k, ps = _pairs(slots, T, dev)
    pw = _operand(weights, _F32, (T, k), dev, "weights")
    if drows is None:
        drows = _empty((M, H), rows.dtype, dev, stream)
    if dweights is None:
        dweights = _empty((T, k), torch.float32, dev, stream)
    _call("moe_combine_rows_grad", dev, stream, pd, _OUT[dout.dtype], pr, _OUT[rows.dtype], ps, pw, T, k, M, H,
          _operand(drows, (rows.dtype,), (M, H), dev, "drows"), _operand(dweights, _F32, (T, k), dev, "dweights"))
    return drows, dweights
