"""What the elementwise bindings share: tensor checks, and the device, stream and addresses of a
launch. Kept short: a decode step's kernel takes a few microseconds, and so should its binding."""
import contextlib

import torch

_NOTHING = contextlib.nullcontext()
_current_device = getattr(torch._C, "_cuda_getDevice", None)            # torch.cuda.current_device without its wrappers
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # torch.cuda.current_stream without the Stream object


def check(name, t, index, dtype, shape):
    """``t`` must be a contiguous ``dtype`` tensor of ``shape`` on GPU ``index`` (-1: no GPU)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s %s%s)"
                         % (name, dtype, tuple(shape), "cuda:%d" % index if index >= 0 else "the inputs' device", t.dtype,
                            tuple(t.shape), t.device, "" if t.is_contiguous() else ", not contiguous"))


def on_gpu(fn, t):
    if not t.is_cuda:
        raise ValueError("%s runs on the GPU; got a tensor on %s" % (fn, t.device))


def ptr(t):
    return None if t is None else t.data_ptr()


def scope(index, stream):
    """Context of a launch and of its allocations: ``index`` is the current device (a launch on a
    device's default stream goes to the device that is current), and with ``stream`` the current
    stream, so that the caching allocator ties the blocks to the stream the kernels run on. A stream of
    another device is refused: its kernels would run there, on memory of this one."""
    if stream is not None and stream.device.index != index:
        raise ValueError("stream is on %s, the tensors on cuda:%d" % (stream.device, index))
    here = index == _current_device()
    if stream is None and here:
        return _NOTHING
    both = contextlib.ExitStack()
    if not here:
        both.enter_context(torch.cuda.device(index))
    if stream is not None:
        both.enter_context(torch.cuda.stream(stream))
    return both


def raw_stream(index, stream):
    """The hipStream_t of ``stream``, or of the current stream of GPU ``index``."""
    return _current_stream(index) if stream is None else stream.cuda_stream
