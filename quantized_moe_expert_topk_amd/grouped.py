"""Python binding of the grouped products by expert, their gradients, the block quantiser and the fp8
block products of ``include/qmoe.h``: argument checks and marshalling only.

Row ranges: ``offsets`` int32 [E + 1] alone, or ``offsets`` (at least E entries) with ``counts``
int32 [E]; ``AlignOut.offsets`` and ``AlignOut.counts`` are in this form.  ``expected_rows`` is about how
many rows the experts hold together (T * k; None: all rows).  Rows of no expert are left as they are in
``out``, and undefined in an output allocated here.

All tensors of a call are on one device, whose current stream the call uses unless ``stream`` is given.  Then the
caller sees to it that ``stream`` comes after the work that makes the operands, and outputs allocated here belong to
``stream``, as if the call were made under ``torch.cuda.stream(stream)``.

Nothing is recorded for autograd: tensors that require gradients are refused while gradients are recorded, as a result
without a history would be a silent loss.  Call under ``torch.no_grad()``, or from ``torch.autograd.Function``'s methods
(where nothing is recorded) with :func:`moe_grouped_mm_dgrad` and :func:`moe_grouped_mm_wgrad` as the backward.
"""
from __future__ import annotations

import torch

from ._lib import MOE_LAYOUT_ROWS, MOE_OUT_BF16, MOE_OUT_F32, check, lib
from ._streams import allocating_on

_OUT = {torch.float32: MOE_OUT_F32, torch.bfloat16: MOE_OUT_BF16}
_CODES = (torch.float8_e4m3fn, torch.uint8)
_INT_MAX = 2 ** 31 - 1  # of the C interface's sizes: ctypes would pass the low bits of a larger number


def _operand(t: torch.Tensor, dtypes, shape, device, name: str) -> int:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires gradients, which this call does not record; call it under torch.no_grad()")
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _matrix(t: torch.Tensor, dims: int, name: str):
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(t.shape)}")
    if not 0 < t.numel() <= _INT_MAX and max(t.shape) > _INT_MAX:  # (numel() is the cheaper one)
        raise ValueError(f"{name}: shape {tuple(t.shape)} is too large for 32-bit sizes")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: expected a cuda tensor, got one on {t.device}")
    return t.shape


def _ranges(offsets: torch.Tensor, counts: torch.Tensor | None, E: int, device):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.device != device \
            or offsets.shape[0] < E + (counts is None):
        raise ValueError(f"offsets: expected contiguous int32 [{E + 1}] on {device}, got {offsets.dtype} "
                         f"{tuple(offsets.shape)} on {offsets.device}")
    return offsets.data_ptr(), _operand(counts, (torch.int32,), (E,), device, "counts") if counts is not None else None


def _rows_hint(expected_rows: int | None, M: int) -> int:
    if expected_rows is None:
        return M
    return expected_rows if 0 <= expected_rows <= _INT_MAX else _INT_MAX if expected_rows > 0 else -1


def _experts(offsets: torch.Tensor, counts: torch.Tensor | None) -> int:
    """How many experts the row ranges are of."""
    t, rest = (offsets, 1) if counts is None else (counts, 0)
    if t.dim() != 1 or t.shape[0] <= rest:
        raise ValueError(f"{'offsets' if rest else 'counts'}: expected the ranges of at least one expert, got shape {tuple(t.shape)}")
    return t.shape[0] - rest


def _output(out, out_dtype, shape, device, stream=None):
    if out is None:
        with allocating_on(stream, device):
            out = torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out: expected {out_dtype}, got {out.dtype}")
    if out.dtype not in _OUT:
        raise ValueError(f"out: expected float32 or bfloat16, got {out.dtype}")
    return out, _operand(out, (out.dtype,), shape, device, "out"), _OUT[out.dtype]


_entries: dict = {}  # C functions by name


def _call(name: str, device, stream, *args) -> None:
    """The C call ``name`` on ``stream`` (default: the device's current one) of ``device``."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(lib(), name)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device.index)  # current_stream() builds an object: 1.7 us a call
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:  # launches go to the current device
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc:
        check(name, rc)


def _grouped(name, a, b, offsets, counts, expected_rows, E, N, K, out, out_dtype, shape, stream, *more):
    """a: the row matrix that the call is named by; b: the other operand, both checked."""
    dev = a.device
    off, cnt = _ranges(offsets, counts, E, dev)
    out, po, code = _output(out, out_dtype, shape, dev, stream)
    M = a.shape[0]
    _call(name, dev, stream, a.data_ptr(), b.data_ptr(), off, cnt, E, M,
          _rows_hint(expected_rows, M), N, K, po, code, *more)
    return out


_BF16 = (torch.bfloat16,)


def moe_grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, counts: torch.Tensor | None = None,
                   expected_rows: int | None = None, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """y[r] = w[e] @ x[r] for every row r of expert e.  x [M, K] bf16, w [E, N, K] bf16 -> [M, N] bf16 or f32."""
    M, K = _matrix(x, 2, "x")
    E, N, _ = _matrix(w, 3, "w")
    _operand(x, _BF16, (M, K), x.device, "x")
    _operand(w, _BF16, (E, N, K), x.device, "w")
    return _grouped("moe_grouped_mm", x, w, offsets, counts, expected_rows, E, N, K, out, out_dtype, (M, N), stream)


def moe_grouped_mm_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, counts: torch.Tensor | None = None,
                         expected_rows: int | None = None, out: torch.Tensor | None = None,
                         out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """The gradient of :func:`moe_grouped_mm` for x: dx[r] = w[e]^T @ dy[r].  dy [M, N], w [E, N, K] -> [M, K]."""
    M, N = _matrix(dy, 2, "dy")
    E, _, K = _matrix(w, 3, "w")
    _operand(dy, _BF16, (M, N), dy.device, "dy")
    _operand(w, _BF16, (E, N, K), dy.device, "w")
    return _grouped("moe_grouped_mm_dgrad", dy, w, offsets, counts, expected_rows, E, N, K, out, out_dtype, (M, K), stream)


def moe_grouped_mm_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, counts: torch.Tensor | None = None,
                         expected_rows: int | None = None, out: torch.Tensor | None = None,
                         out_dtype: torch.dtype | None = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """The gradient of :func:`moe_grouped_mm` for w: dw[e] = dy[rows of e]^T @ x[rows of e], zeros for an expert
    without rows.  dy [M, N], x [M, K] -> [E, N, K]; E is that of ``counts``, else of ``offsets``, less one.
    ``accumulate`` (f32 ``out`` only) adds to ``out``."""
    M, N = _matrix(dy, 2, "dy")
    _, K = _matrix(x, 2, "x")
    _operand(dy, _BF16, (M, N), dy.device, "dy")
    _operand(x, _BF16, (M, K), dy.device, "x")
    E = _experts(offsets, counts)
    if accumulate and out is None:
        raise ValueError("accumulate: needs the out to add to")
    return _grouped("moe_grouped_mm_wgrad", dy, x, offsets, counts, expected_rows, E, N, K, out, out_dtype, (E, N, K),
                    stream, int(accumulate))


def moe_quantize_blocks(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """bf16 rows [M, K] to e4m3 codes [M, K] and f32 scales [ceil(K / 128), M], one per row and 128 columns."""
    M, K = _matrix(x, 2, "x")
    dev, KB = x.device, (K + 127) // 128
    if q is None or scale is None:
        with allocating_on(stream, dev):
            q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev) if q is None else q
            scale = torch.empty((KB, M), dtype=torch.float32, device=dev) if scale is None else scale
    _call("moe_quantize_blocks", dev, stream, _operand(x, _BF16, (M, K), dev, "x"), M, K,
          _operand(q, _CODES, (M, K), dev, "q"), _operand(scale, (torch.float32,), (KB, M), dev, "scale"))
    return q, scale


def moe_block_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, layout: int = MOE_LAYOUT_ROWS,
                 out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """y = (xq * xs) @ (wq * ws)^T with one scale per row and 128 columns of xq and per 128 x 128 block of wq.
    xq [M, K] and xs as :func:`moe_quantize_blocks` gives them, wq e4m3 [N, K] (``layout`` MOE_LAYOUT_ROWS or
    MOE_LAYOUT_TILE16), ws f32 [ceil(N / 128), ceil(K / 128)] -> [M, N] bf16 or f32."""
    M, K = _matrix(xq, 2, "xq")
    N, _ = _matrix(wq, 2, "wq")
    dev, NB, KB = xq.device, (N + 127) // 128, (K + 127) // 128
    f32 = (torch.float32,)
    out, po, code = _output(out, out_dtype, (M, N), dev, stream)
    _call("moe_block_mm", dev, stream, _operand(xq, _CODES, (M, K), dev, "xq"), _operand(xs, f32, (KB, M), dev, "xs"),
          _operand(wq, _CODES, (N, K), dev, "wq"), _operand(ws, f32, (NB, KB), dev, "ws"), layout, M, N, K, po, code)
    return out


def moe_grouped_block_mm(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, offsets: torch.Tensor,
                         counts: torch.Tensor | None = None, expected_rows: int | None = None,
                         layout: int = MOE_LAYOUT_ROWS, out: torch.Tensor | None = None,
                         out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """:func:`moe_block_mm` by expert: wq [E, N, K], ws [E, ceil(N / 128), ceil(K / 128)], row ranges as above."""
    M, K = _matrix(xq, 2, "xq")
    E, N, _ = _matrix(wq, 3, "wq")
    dev, NB, KB = xq.device, (N + 127) // 128, (K + 127) // 128
    f32 = (torch.float32,)
    off, cnt = _ranges(offsets, counts, E, dev)
    out, po, code = _output(out, out_dtype, (M, N), dev, stream)
    _call("moe_grouped_block_mm", dev, stream, _operand(xq, _CODES, (M, K), dev, "xq"),
          _operand(xs, f32, (KB, M), dev, "xs"), _operand(wq, _CODES, (E, N, K), dev, "wq"),
          _operand(ws, f32, (E, NB, KB), dev, "ws"), layout, off, cnt, E, M, _rows_hint(expected_rows, M),
          N, K, po, code)
    return out
