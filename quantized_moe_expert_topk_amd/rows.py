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

_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


# The checks of grouped.py, which a call of a few microseconds spends a good part of its time in: what is right is seen
# with fewer questions (a cuda device has an index), what is not goes on to those checks, which say what is wrong.

def _arg(t: torch.Tensor, dtype: torch.dtype, shape, device, name: str) -> int:
    if t.dtype is dtype and t.shape == shape and t.device == device and not t.requires_grad and t.is_contiguous():
        return t.data_ptr()
    return _operand(t, (dtype,), shape, device, name)


def _sizes(t: torch.Tensor, name: str):
    """The shape of a matrix on a cuda device."""
    shape = t.shape
    if len(shape) == 2 and 0 < t.numel() <= _INT_MAX and t.device.index is not None:
        return shape
    return _matrix(t, 2, name)


def _values(t: torch.Tensor, shape, device, name: str) -> tuple[int, int]:
    """(address, type code) of a bf16 or f32 matrix."""
    dtype = _BF16 if t.dtype is _BF16 else _F32
    return _arg(t, dtype, shape, device, name), _OUT[dtype]


def _runs(offsets: torch.Tensor, counts: torch.Tensor | None, E: int, device):
    """The addresses of the row ranges of E experts."""
    if offsets.dtype is _I32 and offsets.device == device and offsets.dim() == 1 and offsets.is_contiguous() \
            and offsets.shape[0] >= E + (counts is None):
        return offsets.data_ptr(), None if counts is None else _arg(counts, _I32, (E,), device, "counts")
    return _ranges(offsets, counts, E, device)


def _pairs(slots: torch.Tensor, T: int | None, device) -> tuple[int, int, int]:
    """(T, k, address) of a slots tensor of T tokens."""
    shape = _sizes(slots, "slots")
    p = _arg(slots, _I32, shape if T is None else (T, shape[1]), device, "slots")
    return shape[0], shape[1], p


def _empty(shape, dtype, device, stream):
    with allocating_on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def moe_pair_slots(topk_ids: torch.Tensor, sorted_ids: torch.Tensor, offsets: torch.Tensor,
                   counts: torch.Tensor | None = None, slots: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The place of every pair in ``sorted_ids``, -1 for a pair that has none.  topk_ids int32 [T, k]; sorted_ids,
    offsets and counts as :func:`moe_align` gives them -> int32 [T, k]."""
    T, k = shape = _sizes(topk_ids, "topk_ids")
    dev = topk_ids.device
    ids = _arg(topk_ids, _I32, shape, dev, "topk_ids")
    M, = _matrix(sorted_ids, 1, "sorted_ids")
    E = counts.shape[0] if counts is not None and counts.dim() == 1 else max(offsets.numel() - 1, 0)
    off, cnt = _runs(offsets, counts, E, dev)
    at = _arg(sorted_ids, _I32, (M,), dev, "sorted_ids")
    if slots is None:
        slots = _empty((T, k), torch.int32, dev, stream)
    _call("moe_pair_slots", dev, stream, ids, T, k, at, M, off, cnt, E, _arg(slots, _I32, shape, dev, "slots"))
    return slots


def _room(rows: int | None, T: int, k: int) -> int:
    """Rows of a row matrix that is allocated here."""
    if rows is None:
        return T * k
    if not 0 <= rows <= _INT_MAX:
        raise ValueError(f"rows: {rows} is not a number of rows")
    return rows


def moe_gather_rows(x: torch.Tensor, slots: torch.Tensor, rows: int | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """out[slots[t, j]] = x[t] for every pair.  x [T, H] of any type, rows of whole 16 bytes -> [rows, H] (``rows``: that
    of ``out``, else T * k).  The bytes are moved as they are: a lazily conjugated view (``resolve_conj()``) is refused.
    Its gradient for x is :func:`moe_combine_rows` of the rows' gradients, without weights."""
    T, H = shape = _sizes(x, "x")
    dev = x.device
    px = _arg(x, x.dtype, shape, dev, "x")
    _, k, ps = _pairs(slots, T, dev)
    if out is None:
        M = _room(rows, T, k)
        out = _empty((M, H), x.dtype, dev, stream)
    else:
        M = _sizes(out, "out")[0]
    if x.dtype.is_complex:
        for name, t in (("x", x), ("out", out)):
            if t.is_conj():
                raise ValueError(f"{name}: a conjugated view, whose bytes are not its values; call resolve_conj() first")
    width = H * x.element_size()
    if width > _INT_MAX:
        raise ValueError(f"x: rows of {width} bytes are too large for 32-bit sizes")
    _call("moe_gather_rows", dev, stream, px, T, k, ps, width, M, _arg(out, x.dtype, (M, H), dev, "out"))
    return out


def moe_combine_rows(rows: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                     add: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * rows[slots[t, j]].  rows [M, H] bf16 or f32, weights f32 [T, k] (None:
    ones), add [T, H] of out's type -> [T, H] of ``out_dtype`` (rows' type if None)."""
    M, H = shape = _sizes(rows, "rows")
    dev = rows.device
    pr, rt = _values(rows, shape, dev, "rows")
    T, k, ps = _pairs(slots, None, dev)
    pw = _arg(weights, _F32, (T, k), dev, "weights") if weights is not None else None
    if out is None or out_dtype is not None:
        out, po, code = _output(out, out_dtype or rows.dtype, (T, H), dev, stream)
    else:
        po, code = _values(out, (T, H), dev, "out")
    pa = _arg(add, out.dtype, (T, H), dev, "add") if add is not None else None
    _call("moe_combine_rows", dev, stream, pr, rt, ps, pw, pa, T, k, M, H, po, code)
    return out


def moe_combine_rows_grad(dout: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
                          drows: torch.Tensor | None = None, dweights: torch.Tensor | None = None, stream=None):
    """The gradients of :func:`moe_combine_rows` with weights: drows[slots[t, j]] = weights[t, j] * dout[t] (of rows' shape
    and type) and dweights[t, j] = <rows[slots[t, j]], dout[t]> (f32 [T, k], 0 for pairs without a row)."""
    T, H = _sizes(dout, "dout")
    M = _sizes(rows, "rows")[0]
    dev, shape = dout.device, (M, H)
    pd, dt = _values(dout, (T, H), dev, "dout")
    pr, rt = _values(rows, shape, dev, "rows")
    _, k, ps = _pairs(slots, T, dev)
    pw = _arg(weights, _F32, (T, k), dev, "weights")
    if drows is None:
        drows = _empty(shape, rows.dtype, dev, stream)
    if dweights is None:
        dweights = _empty((T, k), _F32, dev, stream)
    _call("moe_combine_rows_grad", dev, stream, pd, dt, pr, rt, ps, pw, T, k, M, H,
          _arg(drows, rows.dtype, shape, dev, "drows"), _arg(dweights, _F32, (T, k), dev, "dweights"))
    return drows, dweights
