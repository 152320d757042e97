"""What the elementwise bindings share: tensor checks, and the device, stream and addresses of a
launch. Kept short: a decode step's kernel takes a few microseconds, and so should its binding."""
import contextlib

import torch

_NOTHING = contextlib.nullcontext()


def check(name, t, dev, dtype, shape):
    """``t`` must be a contiguous ``dtype`` tensor of ``shape`` on ``dev``."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s %s%s)"
                         % (name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape), t.device,
                            "" if t.is_contiguous() else ", not contiguous"))


def data_ptr(t):
    return None if t is None else t.data_ptr()


def scope(dev, stream):
    """Context of a launch and of its allocations: ``dev`` is the current device (a launch on a
    device's default stream goes to the device that is current), and with ``stream`` the current
    stream, so that the caching allocator ties the blocks to the stream the kernels run on."""
    here = dev.index is None or dev.index == torch.cuda.current_device()
    if stream is None and here:
        return _NOTHING
    both = contextlib.ExitStack()
    if not here:
        both.enter_context(torch.cuda.device(dev))
    if stream is not None:
        both.enter_context(torch.cuda.stream(stream))
    return both


def raw_stream(dev, stream):
    """The hipStream_t of ``stream``, or of the current stream of ``dev`` (without the Stream object
    that torch.cuda.current_stream makes: 2 us of a call's 10)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev.index is None else dev.index)
