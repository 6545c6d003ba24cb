"""Gated feed-forward layer and its gradients: binding of include/fconv_gated.h.

    p = GatedPlan(T, D, F, "bf16", activation="silu")
    y = p.forward(x, w)                       # act(x w[:F]^T) (x w[F:]^T), [T, F]
    y, kept = p.forward(x, w, keep=True)      # for the gradients
    dx, dw = p.backward(x, w, kept, dy)
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from . import DTYPES, _check, _whole
from ._dense import TORCH, call, done, matrix, type_name, vector

__all__ = ["GatedPlan"]


class GatedPlan:
    """y = act(g) u with g = x w[:F]^T and u = x w[F:]^T, x [T, D], w [2 F, D] of
    dtype "bf16" or "fp32"; activation "silu", "gelu", "gelu_tanh" or "relu"."""

    def __init__(self, T, D, F, dtype="bf16", activation="silu"):
        dtype = type_name(dtype)
        if activation not in _abi.ACTIVATIONS:
            raise ValueError("activation %r: %s" % (activation, ", ".join(_abi.ACTIVATIONS)))
        d = _abi.GatedDesc()
        d.T, d.D, d.F = T, D, F = _whole("T, D and F", T, D, F)
        d.dtype, d.activation = DTYPES[dtype], _abi.ACTIVATIONS.index(activation)
        self.desc = d
        self.T, self.D, self.F, self.dtype, self.activation = T, D, F, dtype, activation
        self._h = ctypes.c_void_p()
        L = self._lib = _abi.gated_lib()
        self._destroy = L.fconv_gated_plan_destroy  # still at hand when the interpreter ends
        _check(L.fconv_gated_plan_create(ctypes.byref(d), ctypes.byref(self._h)), "fconv_gated_plan_create")
        self._torch = TORCH[dtype]
        self.kept_bytes = self._size("kept")
        self.forward_workspace_bytes = self._size("forward_workspace")
        self.backward_workspace_bytes = self._size("backward_workspace")
        self._kept = self.kept_bytes // 4  # fp32
        self._call = _abi.native()
        sizes = (self._h.value, T, D, F, d.dtype)
        self._forward = (_abi.address(L.fconv_gated_plan_forward),) + sizes + (self.forward_workspace_bytes,)
        self._backward = (_abi.address(L.fconv_gated_plan_backward),) + sizes + (self.backward_workspace_bytes,
                                                                                 self._kept)

    def _size(self, what):
        n, name = ctypes.c_size_t(), "fconv_gated_plan_%s_size" % what
        _check(getattr(self._lib, name)(self._h, ctypes.byref(n)), name)
        return n.value

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._destroy(h)
            self._h = None

    def kernel_name(self, product):
        """Of "forward", "dx" or "dw"; None without tokens."""
        name = self._lib.fconv_gated_plan_kernel_name(self._h, _abi.GATED_PRODUCTS.index(product))
        return name and name.decode()

    def ranges(self, product):
        """Ranges of a product's sum."""
        n = ctypes.c_int32()
        _check(self._lib.fconv_gated_plan_ranges(self._h, _abi.GATED_PRODUCTS.index(product), ctypes.byref(n)),
               "fconv_gated_plan_ranges")
        return n.value

    def _inputs(self, x, w):
        a = _abi.GatedArgs()
        a.x, a.ldx = matrix(x, "x", self.T, self.D, self._torch)
        a.w, a.ldw = matrix(w, "w", 2 * self.F, self.D, self._torch)
        return a

    def forward(self, x, w, keep=False, y=None, stream=None):
        """y [T, F], or (y, kept) with keep: what `backward` needs of this pass.
        x, w and `y`, if given, may have rows apart."""
        if stream is None and y is None and self.T > 0:
            r = self._call.gated_forward(x, w, *self._forward, self._kept if keep else 0)
            if r is not None:
                return done(r, "fconv_gated_plan_forward")
        a = self._inputs(x, w)

        def run(s, device):
            out = y
            if out is not None:
                a.y, a.ldy = matrix(out, "y", self.T, self.F, self._torch)
            else:
                out = torch.empty(self.T, self.F, dtype=self._torch, device=device)
                a.y, a.ldy = out.data_ptr(), self.F
            kept = torch.empty(self._kept, dtype=torch.float32, device=device) if keep else None
            ws = torch.empty(self.forward_workspace_bytes, dtype=torch.uint8, device=device)
            a.kept = kept.data_ptr() if keep else None
            a.workspace, a.workspace_bytes = ws.data_ptr(), self.forward_workspace_bytes
            _check(self._lib.fconv_gated_plan_forward(self._h, s, ctypes.byref(a)), "fconv_gated_plan_forward")
            return (out, kept) if keep else out
        return call(run, stream, x, w, y)

    def backward(self, x, w, kept, dy, dx=None, dw=None, need_dx=True, need_dw=True, stream=None):
        """(dx [T, D], dw [2 F, D]) from what the forward pass on the same x and w
        has kept and the gradient dy [T, F] of y; in `dx` and `dw` (whose rows may
        be apart) if given, None where not needed."""
        if not (need_dx or need_dw):
            raise ValueError("backward: no gradient needed")
        if (dx is not None and not need_dx) or (dw is not None and not need_dw):
            raise ValueError("backward: an output given for a gradient that is not needed")
        # Of no tokens dx has no address: the full way.
        if stream is None and need_dx and need_dw and dx is None and dw is None and self.T > 0:
            r = self._call.gated_backward(x, w, kept, dy, *self._backward)
            if r is not None:
                return done(r, "fconv_gated_plan_backward")
        a = self._inputs(x, w)
        a.kept = vector(kept, "kept", self._kept, torch.float32)
        a.dy, a.lddy = matrix(dy, "dy", self.T, self.F, self._torch)

        def run(s, device):
            gx, gw = dx, dw
            if gx is not None:
                a.dx, a.lddx = matrix(gx, "dx", self.T, self.D, self._torch)
            elif need_dx:
                gx = torch.empty(self.T, self.D, dtype=self._torch, device=device)
                a.dx, a.lddx = gx.data_ptr(), self.D
            if gw is not None:
                a.dw, a.lddw = matrix(gw, "dw", 2 * self.F, self.D, self._torch)
            elif need_dw:
                gw = torch.empty(2 * self.F, self.D, dtype=self._torch, device=device)
                a.dw, a.lddw = gw.data_ptr(), self.D
            ws = torch.empty(self.backward_workspace_bytes, dtype=torch.uint8, device=device)
            a.workspace, a.workspace_bytes = ws.data_ptr(), self.backward_workspace_bytes
            # Of no tokens dx has no address, and dw is all there is to write.
            if a.dx or a.dw:
                _check(self._lib.fconv_gated_plan_backward(self._h, s, ctypes.byref(a)), "fconv_gated_plan_backward")
            return gx, gw
        return call(run, stream, x, w, kept, dy, dx, dw)
