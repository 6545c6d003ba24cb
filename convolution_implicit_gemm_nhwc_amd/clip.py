"""Norm of many gradients together and clipping by it: binding of
include/fconv_clip.h.

    p = ClipPlan([(g.numel(), "bf16") for g in grads])
    norm = p.clip(grads, max_norm)               # in place; norm is a 0-d fp32 tensor
    norm = p.norm(grads)
    p.clip(grads, max_norm, norm=norm, out=out)  # by a norm that is there already
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _abi
from . import DTYPES, _check, _whole
from ._dense import TORCH, call, done, type_name, vector

__all__ = ["ClipPlan"]


def _filled(t, what, numel, dtype):
    """Address of a GPU tensor whose elements fill their memory, in any order of
    its dimensions (a transposed or channels-last one, say)."""
    if t.dtype is not dtype:
        raise ValueError("%s: dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.numel() != numel:
        raise ValueError("%s: %d elements, the plan needs %d" % (what, t.numel(), numel))
    step = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if numel and stride != step:
            raise ValueError("%s: elements must lie one after another (strides %s)" % (what, tuple(t.stride())))
        step *= size
    if not t.is_cuda:
        raise ValueError("%s: tensor must live on the GPU (got %s)" % (what, t.device))
    return t.data_ptr()


class ClipPlan:
    """tensors: (numel, dtype) of each gradient (one at least), dtype "bf16" or
    "fp32"; eps is added to the norm that max_norm is divided by."""

    def __init__(self, tensors, eps=1e-6):
        sizes = [(_whole("numel", n, bits=64)[0], type_name(t)) for n, t in tensors]
        if not sizes:
            raise ValueError("a plan of no gradients")
        d = (_abi.ClipTensor * len(sizes))()
        for x, (n, t) in zip(d, sizes):
            x.numel, x.dtype = n, DTYPES[t]
        self.tensors = sizes
        self._h = ctypes.c_void_p()
        L = self._lib = _abi.clip_lib()
        self._destroy = L.fconv_clip_plan_destroy  # still at hand when the interpreter ends
        _check(L.fconv_clip_plan_create(d, len(sizes), eps, ctypes.byref(self._h)), "fconv_clip_plan_create")
        self.eps = ctypes.c_float(eps).value
        n = ctypes.c_size_t()
        _check(L.fconv_clip_plan_workspace_size(self._h, ctypes.byref(n)), "fconv_clip_plan_workspace_size")
        self.workspace_bytes = n.value
        self._call = _abi.native()
        rest = (self._h.value, _abi.address(L.fconv_clip_plan_tensors))
        self._norm = (_abi.address(L.fconv_clip_plan_norm),) + rest
        self._clip = (_abi.address(L.fconv_clip_plan_clip),) + rest

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._destroy(h)
            self._h = None

    def _addresses(self, tensors, what):
        if len(tensors) != len(self.tensors):
            raise ValueError("%s: %d tensors, the plan needs %d" % (what, len(tensors), len(self.tensors)))
        return (ctypes.c_void_p * len(tensors))(*(
            _filled(t, "%s[%d]" % (what, i), n, TORCH[dt])
            for i, (t, (n, dt)) in enumerate(zip(tensors, self.tensors))))

    def norm(self, grads, stream=None):
        """The norm of all gradients, a 0-d fp32 tensor."""
        return self._run(list(grads), None, None, None, stream)

    def clip(self, grads, max_norm, norm=None, out=None, stream=None):
        """Scales the gradients by min(1, max_norm / (norm + eps)), in place or into
        the tensors `out` (of the same shapes and strides), and returns the norm.
        With `norm` (a 0-d fp32 tensor on the GPU) that is taken instead of theirs."""
        max_norm = float(max_norm)
        if not max_norm >= 0.0:
            raise ValueError("max_norm %r: a number that is not negative" % max_norm)
        if math.isfinite(max_norm):  # past fp32 it would become an infinity, which clips nothing
            max_norm = min(max_norm, torch.finfo(torch.float32).max)
        return self._run(list(grads), max_norm, norm, None if out is None else list(out), stream)

    def _run(self, grads, max_norm, given, out, stream):
        clip = max_norm is not None
        what = "fconv_clip_plan_clip" if clip else "fconv_clip_plan_norm"
        if stream is None and given is None:
            r = self._call.clip(grads, out, *(self._clip if clip else self._norm), max_norm, self.workspace_bytes)
            if r is not None:
                return done(r, what)
        a = _abi.ClipArgs()
        a.in_ = self._addresses(grads, "grads")
        if clip:
            a.max_norm = max_norm
            a.out = a.in_ if out is None else self._addresses(out, "out")
            for i, (g, o) in enumerate(zip(grads, out or ())):
                if g.shape != o.shape or g.stride() != o.stride():
                    raise ValueError("out[%d]: shape %s and strides %s, the gradient has %s and %s"
                                     % (i, tuple(o.shape), o.stride(), tuple(g.shape), g.stride()))
        if given is not None:
            a.given_norm = vector(given, "norm", 1, torch.float32)

        def run(s, device):
            norm = given
            if norm is None:
                norm = torch.empty((), dtype=torch.float32, device=device)
                ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
                a.norm, a.workspace, a.workspace_bytes = norm.data_ptr(), ws.data_ptr(), self.workspace_bytes
            fn = self._lib.fconv_clip_plan_clip if clip else self._lib.fconv_clip_plan_norm
            _check(fn(self._h, s, ctypes.byref(a)), what)
            return norm
        return call(run, stream, *grads, given, *(out or ()))
