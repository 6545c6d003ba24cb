"""What the bindings of the dense operators share: checks of 2-D tensors, and
where a call's stream, output and workspace come from."""
from __future__ import annotations

import torch

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def matrix(t, what, rows, cols, dtype):
    """Address and row stride (elements) of a GPU tensor that holds a
    [rows, cols] matrix: a 2-D tensor whose rows are dense (any row stride),
    or a contiguous tensor of another shape with rows * cols elements (an
    NHWC feature map, say)."""
    if t.dtype != dtype:
        raise ValueError("%s: dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.dim() == 2 and t.shape[0] == rows and t.shape[1] == cols:
        ld = t.stride(0) if rows > 1 else cols
        if (cols > 1 and t.stride(1) != 1) or ld < cols:
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
    if t.dtype != dtype:
        raise ValueError("%s: dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.numel() != numel:
        raise ValueError("%s: %d elements, the plan needs %d" % (what, t.numel(), numel))
    if not t.is_contiguous():
        raise ValueError("%s: tensor must be contiguous" % what)
    if not t.is_cuda:
        raise ValueError("%s: tensor must live on the GPU (got %s)" % (what, t.device))
    return t.data_ptr()


class Launch:
    """The stream of one call and the device it is on.  With no stream given
    it is torch's current one.  With another one, torch allocates the call's
    output and workspace for that stream, so their memory is not handed on
    while the call still uses it, and the call's inputs are held likewise."""

    def __init__(self, device, stream, inputs):
        for t in inputs:
            if t is not None and t.device != device:
                raise ValueError("tensors on different devices (%s and %s)" % (device, t.device))
        self._scope = []
        if stream is None and device.index == torch.cuda.current_device():
            self.handle = torch.cuda.current_stream().cuda_stream
            return
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
        self._scope.append(torch.cuda.stream(stream))  # switches the device too

    def __enter__(self):
        for s in self._scope:
            s.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for s in self._scope:
            s.__exit__(*exc)
        return False
