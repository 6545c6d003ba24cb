"""Softmax cross entropy of a linear output layer and its gradient, without
keeping the logits: binding of include/fconv_xent.h.

    c = XentPlan(T, D, V, "bf16", ignore_index=-100)
    loss, lse = c.forward(h, w, target)              # fp32 [T] each
    dh, dw = c.backward(h, w, target, lse, dloss)    # dloss fp32 [T]
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from . import DTYPES, _check, _whole
from ._dense import TORCH, call, done, matrix, type_name, vector

__all__ = ["XentPlan"]


class XentPlan:
    """loss[t] = logsumexp_v(z[t, v]) - z[t, target[t]] with z = h w^T, h [T, D],
    w [V, D] of dtype "bf16" or "fp32", target int64 [T].  Tokens whose target is
    ignore_index have loss 0 and no gradient; a target outside [0, V) gives NaN."""

    def __init__(self, T, D, V, dtype="bf16", ignore_index=-100):
        dtype = type_name(dtype)
        d = _abi.XentDesc()
        d.T, d.D, d.V = T, D, V = _whole("T, D and V", T, D, V)
        d.dtype = DTYPES[dtype]
        d.ignore_index, = _whole("ignore_index", ignore_index, bits=64)
        self.desc = d
        self.T, self.D, self.V, self.dtype, self.ignore_index = T, D, V, dtype, ignore_index
        self._h = ctypes.c_void_p()
        L = self._lib = _abi.xent_lib()
        self._destroy = L.fconv_xent_plan_destroy  # still at hand when the interpreter ends
        _check(L.fconv_xent_plan_create(ctypes.byref(d), ctypes.byref(self._h)), "fconv_xent_plan_create")
        self._torch = TORCH[dtype]
        n = ctypes.c_size_t()
        _check(L.fconv_xent_plan_forward_workspace_size(self._h, ctypes.byref(n)),
               "fconv_xent_plan_forward_workspace_size")
        self.forward_workspace_bytes = n.value
        _check(L.fconv_xent_plan_backward_workspace_size(self._h, ctypes.byref(n)),
               "fconv_xent_plan_backward_workspace_size")
        self.backward_workspace_bytes = n.value
        self._call = _abi.native()
        sizes = (self._h.value, T, D, V, d.dtype)
        self._forward = (_abi.address(L.fconv_xent_plan_forward),) + sizes + (self.forward_workspace_bytes,)
        self._backward = (_abi.address(L.fconv_xent_plan_backward),) + sizes + (self.backward_workspace_bytes,)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._destroy(h)
            self._h = None

    def kernel_name(self, product):
        """Of "logits", "grad" (the backward pass's logits), "dh" or "dw"; None without tokens."""
        name = self._lib.fconv_xent_plan_kernel_name(self._h, _abi.XENT_PRODUCTS.index(product))
        return name and name.decode()

    def division(self, product):
        """(pieces of the vocabulary, ranges of the sum) of a product."""
        pieces, ranges = ctypes.c_int32(), ctypes.c_int32()
        _check(self._lib.fconv_xent_plan_division(self._h, _abi.XENT_PRODUCTS.index(product), ctypes.byref(pieces),
                                                  ctypes.byref(ranges)), "fconv_xent_plan_division")
        return pieces.value, ranges.value

    def _inputs(self, h, w, target):
        a = _abi.XentArgs()
        a.h, a.ldh = matrix(h, "h", self.T, self.D, self._torch)
        a.w, a.ldw = matrix(w, "w", self.V, self.D, self._torch)
        a.target = vector(target, "target", self.T, torch.int64)
        return a

    def forward(self, h, w, target, stream=None):
        """(loss, lse), fp32 [T].  h and w may have rows apart."""
        if stream is None:
            r = self._call.xent_forward(h, w, target, *self._forward)
            if r is not None:
                return done(r, "fconv_xent_plan_forward")
        a = self._inputs(h, w, target)

        def run(s, device):
            loss = torch.empty(self.T, dtype=torch.float32, device=device)
            lse = torch.empty(self.T, dtype=torch.float32, device=device)
            ws = torch.empty(self.forward_workspace_bytes, dtype=torch.uint8, device=device)
            a.loss, a.lse = loss.data_ptr(), lse.data_ptr()
            a.workspace, a.workspace_bytes = ws.data_ptr(), self.forward_workspace_bytes
            _check(self._lib.fconv_xent_plan_forward(self._h, s, ctypes.byref(a)), "fconv_xent_plan_forward")
            return loss, lse
        return call(run, stream, h, w, target)

    def backward(self, h, w, target, lse, dloss, dh=None, dw=None, need_dh=True, need_dw=True,
                 stream=None):
        """(dh [T, D], dw [V, D]) from the forward pass's lse and the gradient
        dloss [T] of the loss; in `dh` and `dw` (whose rows may be apart) if
        given, None where not needed."""
        if not (need_dh or need_dw):
            raise ValueError("backward: no gradient needed")
        if (dh is not None and not need_dh) or (dw is not None and not need_dw):
            raise ValueError("backward: an output given for a gradient that is not needed")
        # Of no tokens dh has no address: the full way.
        if stream is None and need_dh and need_dw and dh is None and dw is None and self.T > 0:
            r = self._call.xent_backward(h, w, target, lse, dloss, *self._backward)
            if r is not None:
                return done(r, "fconv_xent_plan_backward")
        a = self._inputs(h, w, target)
        a.lse = vector(lse, "lse", self.T, torch.float32)
        a.dloss = vector(dloss, "dloss", self.T, torch.float32)

        def run(s, device):
            gh, gw = dh, dw
            if gh is not None:
                a.dh, a.lddh = matrix(gh, "dh", self.T, self.D, self._torch)
            elif need_dh:
                gh = torch.empty(self.T, self.D, dtype=self._torch, device=device)
                a.dh, a.lddh = gh.data_ptr(), self.D
            if gw is not None:
                a.dw, a.lddw = matrix(gw, "dw", self.V, self.D, self._torch)
            elif need_dw:
                gw = torch.empty(self.V, self.D, dtype=self._torch, device=device)
                a.dw, a.lddw = gw.data_ptr(), self.D
            ws = torch.empty(self.backward_workspace_bytes, dtype=torch.uint8, device=device)
            a.workspace, a.workspace_bytes = ws.data_ptr(), self.backward_workspace_bytes
            # Of no tokens dh has no address, and dw is all there is to write.
            if a.dh or a.dw:
                _check(self._lib.fconv_xent_plan_backward(self._h, s, ctypes.byref(a)), "fconv_xent_plan_backward")
            return gh, gw
        return call(run, stream, h, w, target, lse, dloss, dh, dw)
