"""What the bindings of the dense operators share: checks of 2-D tensors, and
where a call's stream, output and workspace come from.  The common way through a
call is csrc/call.cpp's; here is the full one, which it leaves to this module
for another stream or device and for arguments that do not fit."""
from __future__ import annotations

import torch

from . import DTYPES, _check

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def type_name(dtype):
    """"int8", "bf16" or "fp32", of a name or of its fconv_dtype code."""
    for name, code in DTYPES.items():
        if dtype == name or (type(dtype) is int and dtype == code):
            return name
    raise ValueError("dtype %r: %s, or their codes" % (dtype, ", ".join(DTYPES)))


def matrix(t, what, rows, cols, dtype):
    """Address and row stride (elements) of a GPU tensor that holds a
    [rows, cols] matrix: a 2-D tensor whose rows are dense (any row stride),
    or a contiguous tensor of another shape with rows * cols elements (an
    NHWC feature map, say)."""
    if t.dtype is not dtype:
        raise ValueError("%s: dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.shape == (rows, cols):
        step, one = t.stride()
        ld = step if rows > 1 else cols
        if (one != 1 and cols > 1) or ld < cols:
            raise ValueError("%s: rows must be dense and apart (strides %s)" % (what, tuple(t.stride())))
    elif t.numel() == rows * cols and t.is_contiguous():
        ld = cols
    else:
        raise ValueError("%s: shape %s, the plan needs [%d, %d]" % (what, tuple(t.shape), rows, cols))
    if not t.is_cuda:
        raise ValueError("%s: tensor must live on the GPU (got %s)" % (what, t.device))
    return t.data_ptr(), ld


def vector(t, what, numel, dtype):
    """Address of a dense GPU vector."""
    if t.dtype is not dtype:
        raise ValueError("%s: dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.numel() != numel:
        raise ValueError("%s: %d elements, the plan needs %d" % (what, t.numel(), numel))
    if not t.is_contiguous():
        raise ValueError("%s: tensor must be contiguous" % what)
    if not t.is_cuda:
        raise ValueError("%s: tensor must live on the GPU (got %s)" % (what, t.device))
    return t.data_ptr()


def same_device(first, *others):
    """The device of all of them (None: not given)."""
    at = first.get_device()
    if at < 0:
        raise ValueError("tensors must live on the GPU (got %s)" % first.device)
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError("tensors on different devices (%s and %s)" % (first.device, t.device))
    return first.device


def current_stream(device):
    """The handle of torch's current stream where `device` is the current one,
    else None."""
    at = device.index
    return torch._C._cuda_getCurrentRawStream(at) if at == torch._C._cuda_getDevice() else None


class Launch:
    """A call on `stream`, which may belong to another device than the current
    one and need not be the current stream.  Torch allocates the call's output
    and workspace for that stream, so their memory is not handed on while the
    call still uses it, and the call's inputs are held likewise."""

    def __init__(self, device, stream, inputs):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError("stream of %s, tensors on %s" % (stream.device, device))
        self.handle = stream.cuda_stream
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        self._scope = torch.cuda.stream(stream)  # switches the device too

    def __enter__(self):
        self._scope.__enter__()
        return self.handle

    def __exit__(self, *exc):
        return self._scope.__exit__(*exc)


def call(run, stream, *tensors):
    """run(handle, device): enqueues a call's work, and allocates what it needs,
    on `stream` (None: torch's current one).  tensors: what the call is given."""
    device = same_device(*tensors)
    if stream is None:
        handle = current_stream(device)
        if handle is not None:
            return run(handle, device)
    with Launch(device, stream, tensors) as handle:
        return run(handle, device)


def done(result, what):
    """What csrc/call.cpp's way has returned, unless it is a status."""
    if type(result) is int:
        _check(result, what)
    return result
