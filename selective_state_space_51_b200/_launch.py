"""What the operators' classes share: argument checks, the launch's stream and
device, buffers allocated where the launch will use them."""
from __future__ import annotations

import contextlib


def dtype_code(t):
    import torch
    from . import SSM_BF16, SSM_F32
    if t.dtype == torch.bfloat16:
        return SSM_BF16
    if t.dtype == torch.float32:
        return SSM_F32
    raise TypeError("activations must be float32 or bfloat16")


def dense(name, t, shape, dtype, device):
    """Raise unless t is None or a contiguous tensor of that description."""
    if t is None:
        return
    if (t.dtype != dtype or t.device != device or tuple(t.shape) != shape
            or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, shape, device))


def apart(**tensors):
    """Raise if two of the named tensors (None: left out) share memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(),
                    n) for n, t in tensors.items()
                   if t is not None and t.numel())
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError("%s and %s must not overlap" % (a, b))


@contextlib.contextmanager
def launching(device, stream):
    """The raw stream to launch on, with `device` current and torch's
    allocations made on that stream (so that a workspace or a result is never
    handed to, or taken from, work that another stream still has to do)."""
    import torch
    if stream is None:
        if torch.cuda.current_device() == device.index:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            with torch.cuda.device(device):
                yield torch.cuda.current_stream(device).cuda_stream
        return
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError("stream belongs to %s, not %s" % (stream.device,
                                                           device))
    with torch.cuda.stream(stream):   # also makes its device current
        yield stream.cuda_stream
