"""Python binding of the MXFP4 quantiser and products of ``include/qmoe.h``: argument checks and marshalling only.

Quantised rows are two uint8 tensors: codes [M, K / 2], two a byte with the even column in the low nibble, and scales
[ceil(K / 128), M, 4], the e8m0 bytes of a row's four blocks of 32 together.  Row ranges, streams, devices and autograd as
in :mod:`~quantized_moe_expert_topk_amd.grouped`; ``slots`` as in :mod:`~quantized_moe_expert_topk_amd.rows`.
"""
from __future__ import annotations

import torch

from ._lib import MOE_LAYOUT_ROWS, MOE_LAYOUT_TILE16
from .grouped import _INT_MAX, _call, _matrix, _output, _rows_hint
from .rows import _BF16, _U8, _arg, _empty, _pairs, _room, _runs, _sizes, _values


def _out(out, out_dtype, shape, device, stream):
    if out is None or out_dtype is not None:
        return _output(out, out_dtype, shape, device, stream)
    return (out, *_values(out, shape, device, "out"))


def _width(codes: torch.Tensor, name: str) -> int:
    """K of a tensor of codes [.., K / 2]."""
    K = codes.shape[-1] * 2
    if K > _INT_MAX:
        raise ValueError(f"{name}: {K} columns are too many for 32-bit sizes")
    return K


def moe_quantize_mx(x: torch.Tensor, slots: torch.Tensor | None = None, rows: int | None = None,
                    q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """bf16 rows [T, K] to codes [M, K / 2] and scales [ceil(K / 128), M, 4]: the least power of two that leaves nothing of a
    block above the largest code (the OCP MX conversion takes half of it for some blocks, and saturates).  Without ``slots`` M is T; with slots
    [T, k] token t goes to rows slots[t], the other rows stay as they were, and M is that of ``q`` or ``scale``, else
    ``rows``, else T * k."""
    T, K = _sizes(x, "x")
    dev, G = x.device, (K + 127) // 128
    px = _arg(x, _BF16, (T, K), dev, "x")
    k, ps, M = 1, None, T
    if slots is None:
        if rows is not None and rows != T:
            raise ValueError(f"rows: without slots the {T} rows of x are quantised, not {rows}")
    else:
        _, k, ps = _pairs(slots, T, dev)
        if q is not None:
            M = _sizes(q, "q")[0]
        else:
            M = _room(rows, T, k) if scale is None else _matrix(scale, 3, "scale")[1]
    if q is None:
        q = _empty((M, K // 2), torch.uint8, dev, stream)
    if scale is None:
        scale = _empty((G, M, 4), torch.uint8, dev, stream)
    _call("moe_quantize_mx", dev, stream, px, ps, T, k, M, K, _arg(q, _U8, (M, K // 2), dev, "q"),
          _arg(scale, _U8, (G, M, 4), dev, "scale"))
    return q, scale


def moe_dequantize_mx(q: torch.Tensor, scale: torch.Tensor, out: torch.Tensor | None = None,
                      out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """The values [M, K], bf16 or f32, of quantised rows."""
    M, _ = _sizes(q, "q")
    K, dev = _width(q, "q"), q.device
    pq = _arg(q, _U8, (M, K // 2), dev, "q")
    ps = _arg(scale, _U8, ((K + 127) // 128, M, 4), dev, "scale")
    out, po, code = _out(out, out_dtype, (M, K), dev, stream)
    _call("moe_dequantize_mx", dev, stream, pq, ps, M, K, po, code)
    return out


def _scales(ws: torch.Tensor, layout: int, lead: tuple, N: int, K: int, device) -> int:
    """Scales of E * N weight rows; lead: (E,) or () of a dense product."""
    rows = N * (lead[0] if lead else 1)
    shape = (*lead, N, K // 32) if layout == MOE_LAYOUT_TILE16 else ((K + 127) // 128, rows, 4)
    return _arg(ws, _U8, shape, device, "ws")


def moe_mx_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, layout: int = MOE_LAYOUT_ROWS,
              out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """y = X @ W^T of the values X [M, K] and W [N, K] of two sets of quantised rows -> [M, N] bf16 or f32.  With ``layout``
    MOE_LAYOUT_TILE16, wq [N, K / 2] and ws [N, K / 32] are one matrix of a packed MXFP4 bank."""
    M, _ = _sizes(xq, "xq")
    N, _ = _sizes(wq, "wq")
    K, dev = _width(xq, "xq"), xq.device
    px, pxs = _arg(xq, _U8, (M, K // 2), dev, "xq"), _arg(xs, _U8, ((K + 127) // 128, M, 4), dev, "xs")
    pw, pws = _arg(wq, _U8, (N, K // 2), dev, "wq"), _scales(ws, layout, (), N, K, dev)
    out, po, code = _out(out, out_dtype, (M, N), dev, stream)
    _call("moe_mx_mm", dev, stream, px, pxs, pw, pws, layout, M, N, K, po, code)
    return out


def moe_grouped_mx_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, offsets: torch.Tensor,
                      counts: torch.Tensor | None = None, expected_rows: int | None = None,
                      layout: int = MOE_LAYOUT_ROWS, out: torch.Tensor | None = None,
                      out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """:func:`moe_mx_mm` by expert: wq [E, N, K / 2], with ws [ceil(K / 128), E * N, 4] as :func:`moe_quantize_mx` gives it
    for the E * N rows, or [E, N, K / 32] of a packed bank; row ranges as for the grouped products."""
    M, _ = _sizes(xq, "xq")
    E, N, _ = _matrix(wq, 3, "wq")
    K, dev = _width(xq, "xq"), xq.device
    px, pxs = _arg(xq, _U8, (M, K // 2), dev, "xq"), _arg(xs, _U8, ((K + 127) // 128, M, 4), dev, "xs")
    pw, pws = _arg(wq, _U8, (E, N, K // 2), dev, "wq"), _scales(ws, layout, (E,), N, K, dev)
    off, cnt = _runs(offsets, counts, E, dev)
    out, po, code = _out(out, out_dtype, (M, N), dev, stream)
    _call("moe_grouped_mx_mm", dev, stream, px, pxs, pw, pws, layout, off, cnt, E, M, _rows_hint(expected_rows, M), N, K,
          po, code)
    return out
