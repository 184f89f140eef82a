"""The stream that memory allocated by the binding belongs to."""
from __future__ import annotations

import contextlib

import torch


def allocating_on(stream, device):
    """A context in which torch allocates on ``stream`` (a torch stream or a raw handle; None: leaves the current one).

    Memory belongs to the stream it was allocated on: work queued there before may still use it, and once it is freed
    goes to work queued there next.  What a call writes on ``stream`` is therefore allocated there."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        handle = int(getattr(stream, "value", stream) or 0)  # (an integer or a ctypes pointer)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)
