"""What the elementwise bindings share at a launch: raw addresses, the raw stream, the device."""
import contextlib

import torch


def data_ptr(t):
    return None if t is None else t.data_ptr()


def raw_stream(dev, stream):
    """The hipStream_t of ``stream``, or of the current stream of ``dev``."""
    return (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream


def on_device(dev):
    """Context in which ``dev`` is the current device: a launch on a device's default stream goes to
    the device that is current."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)
