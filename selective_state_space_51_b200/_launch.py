"""What the operators' classes share: argument checks, the launch's stream and
device, buffers allocated where the launch will use them."""
from __future__ import annotations


def dtype_codes():
    """The activation types by torch's name."""
    import torch
    from . import SSM_BF16, SSM_F32
    return {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}


def dtype_error():
    return TypeError("activations must be float32 or bfloat16")


def dense(name, t, shape, dtype, device):
    """Raise unless t is None or a contiguous tensor of that description."""
    if t is None:
        return
    if (t.shape != shape or t.dtype != dtype or not t.is_contiguous()
            or t.device != device):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, tuple(shape), device))


def ptr(t):
    """Device address of a tensor, None for None."""
    return None if t is None else t.data_ptr()


def apart(**tensors):
    """Raise if two of the named tensors (None: left out) share memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(),
                    n) for n, t in tensors.items()
                   if t is not None and t.numel())
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError("%s and %s must not overlap" % (a, b))


def launch(torch, device, stream, call, *args):
    """call(raw stream, *args) with `device` current and torch's allocations
    made on that stream (so that a workspace or a result is never handed to,
    or taken from, work that another stream still has to do). stream: None
    for torch's current stream of the device, a torch stream or a raw one.

    On another stream than the current one the call comes behind what the
    current stream has been given so far, and the memory of the tensors among
    `args` is not given to anyone else before it is done. A raw stream may go
    before they do, so there the caller keeps them. A call that is captured on
    `stream` while the current stream is not being captured waits for nothing:
    a graph cannot depend on work outside."""
    index = device.index
    if stream is None:
        if torch.cuda.current_device() == index:
            return call(torch._C._cuda_getCurrentRawStream(index), *args)
        with torch.cuda.device(device):
            return call(torch._C._cuda_getCurrentRawStream(index), *args)
    raw = isinstance(stream, int)
    if raw:
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError("stream belongs to %s, not %s" % (stream.device,
                                                           device))
    here = torch.cuda.current_stream(device)
    if stream.cuda_stream == here.cuda_stream:
        with torch.cuda.device(device):
            return call(stream.cuda_stream, *args)
    with torch.cuda.stream(stream):   # also makes its device current
        if not torch.cuda.is_current_stream_capturing() or \
                _captured(torch, here):
            stream.wait_stream(here)
        result = call(stream.cuda_stream, *args)
    if not raw:
        for t in args:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return result


def _captured(torch, stream):
    """(The default stream cannot be, and asking may be an error.)"""
    if stream.cuda_stream == 0:
        return False
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()
