"""Embedding lookup and its gradient: binding of include/fconv_embed.h.

    p = EmbedPlan(T, D, V, "bf16", scale=D ** 0.5, ignore_index=-100)
    y = p.forward(w, token)             # scale w[token], [T, D]
    dw = p.backward(token, dy)          # [V, D], zeros in rows without a token
    p.backward(token, dy, dw=dw, accumulate=True)   # added to what dw holds
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from . import DTYPES, _check, _whole
from ._dense import TORCH, call, done, matrix, type_name, vector

__all__ = ["EmbedPlan"]


class EmbedPlan:
    """y[t] = scale w[token[t]], w [V, D] of dtype "bf16" or "fp32", token int64
    [T].  A token that is ignore_index has y = 0 and no gradient; another one
    outside [0, V) has a row of NaN and no gradient."""

    def __init__(self, T, D, V, dtype="bf16", scale=1.0, ignore_index=-100):
        dtype = type_name(dtype)
        d = _abi.EmbedDesc()
        d.T, d.D, d.V = T, D, V = _whole("T, D and V", T, D, V)
        d.dtype, d.scale = DTYPES[dtype], scale
        d.ignore_index, = _whole("ignore_index", ignore_index, bits=64)
        self.desc = d
        self.T, self.D, self.V, self.dtype, self.scale, self.ignore_index = T, D, V, dtype, d.scale, ignore_index
        self._h = ctypes.c_void_p()
        L = self._lib = _abi.embed_lib()
        self._destroy = L.fconv_embed_plan_destroy  # still at hand when the interpreter ends
        _check(L.fconv_embed_plan_create(ctypes.byref(d), ctypes.byref(self._h)), "fconv_embed_plan_create")
        self._torch = TORCH[dtype]
        n = ctypes.c_size_t()
        _check(L.fconv_embed_plan_workspace_size(self._h, ctypes.byref(n)), "fconv_embed_plan_workspace_size")
        self.workspace_bytes = n.value
        self._call = _abi.native()
        sizes = (self._h.value, T, D, V, d.dtype)
        self._forward = (_abi.address(L.fconv_embed_plan_forward),) + sizes
        self._backward = (_abi.address(L.fconv_embed_plan_backward),) + sizes + (self.workspace_bytes,)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._destroy(h)
            self._h = None

    def forward(self, w, token, y=None, stream=None):
        """y [T, D].  w and `y`, if given, may have rows apart."""
        if stream is None and y is None and self.T > 0:
            r = self._call.embed_forward(w, token, *self._forward)
            if r is not None:
                return done(r, "fconv_embed_plan_forward")
        a = _abi.EmbedArgs()
        a.w, a.ldw = matrix(w, "w", self.V, self.D, self._torch)
        a.token = vector(token, "token", self.T, torch.int64)

        def run(s, device):
            out = y
            if out is not None:
                a.y, a.ldy = matrix(out, "y", self.T, self.D, self._torch)
            else:
                out = torch.empty(self.T, self.D, dtype=self._torch, device=device)
                a.y, a.ldy = out.data_ptr(), self.D
            _check(self._lib.fconv_embed_plan_forward(self._h, s, ctypes.byref(a)), "fconv_embed_plan_forward")
            return out
        return call(run, stream, w, token, y)

    def backward(self, token, dy, dw=None, accumulate=False, stream=None):
        """dw [V, D] from the gradient dy [T, D] of y; in `dw` (whose rows may be
        apart) if given, added to what it holds with accumulate."""
        if accumulate and dw is None:
            raise ValueError("backward: accumulate needs the dw to add to")
        if stream is None and dw is None and self.T > 0:
            r = self._call.embed_backward(token, dy, *self._backward)
            if r is not None:
                return done(r, "fconv_embed_plan_backward")
        a = _abi.EmbedArgs()
        a.token = vector(token, "token", self.T, torch.int64)
        a.dy, a.lddy = matrix(dy, "dy", self.T, self.D, self._torch)
        a.run_flags = _abi.FCONV_EMBED_ADD if accumulate else 0

        def run(s, device):
            out = dw
            if out is not None:
                a.dw, a.lddw = matrix(out, "dw", self.V, self.D, self._torch)
            else:
                out = torch.empty(self.V, self.D, dtype=self._torch, device=device)
                a.dw, a.lddw = out.data_ptr(), self.D
            ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
            a.workspace, a.workspace_bytes = ws.data_ptr(), self.workspace_bytes
            _check(self._lib.fconv_embed_plan_backward(self._h, s, ctypes.byref(a)), "fconv_embed_plan_backward")
            return out
        return call(run, stream, token, dy, dw)
