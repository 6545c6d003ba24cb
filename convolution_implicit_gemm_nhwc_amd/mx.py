"""MXFP4 (microscaled 4-bit floating point): binding of include/fconv_mx.h.

    q = MxQuantPlan(rows, cols, "bf16")
    t = q(x)                   # MxTensor: e2m1 codes, one e8m0 scale per 32
    x4 = q.dequantize(t)       # the values that t stands for

    w4 = MxTensor.from_codes(codes, scales, K)     # a 4-bit checkpoint
    y = MxPlan(M, N, K, "bf16", ops=("bias", "relu"))(x, w4, bias=b)

A quantised matrix is kept in the order in which the matrix cores read it
(the header says which); it is laid out once, when it is made.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from . import DTYPES, OPS, _check, _whole
from ._dense import TORCH, call, done, matrix, type_name, vector

__all__ = ["MxTensor", "MxQuantPlan", "MxPlan"]


def _mx_bytes(rows, cols):
    rows, cols = _whole("rows and cols", rows, cols)
    n = ctypes.c_size_t()
    _check(_abi.mx_lib().fconv_mx_bytes(rows, cols, ctypes.byref(n)), "fconv_mx_bytes")
    return n.value


class MxTensor:
    """A quantised [rows, cols] matrix: one uint8 GPU buffer `data` of
    fconv_mx_bytes(rows, cols) bytes, codes and then scales."""

    __slots__ = ("data", "rows", "cols")

    def __init__(self, data, rows, cols):
        self.data, self.rows, self.cols = data, rows, cols
        self.address(_mx_bytes(rows, cols))

    def address(self, nbytes):
        """Of the buffer, which has to hold `nbytes`: asked at each use, since a
        kernel reads that much whatever `data` has become."""
        data = self.data
        if data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() < nbytes:
            raise ValueError("data: %d bytes needed (uint8, contiguous), got %s of %s"
                             % (nbytes, tuple(data.shape), data.dtype))
        return data.data_ptr()

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.data.device

    @classmethod
    def from_codes(cls, codes, scales, cols, stream=None):
        """From row-major codes [rows, ceil(cols/32)*16] (uint8, two e2m1
        codes to a byte, low half first) and e8m0 scales [rows,
        ceil(cols/32)] (uint8)."""
        rows, nb = codes.shape[0], -(-cols // 32)
        nbytes = _mx_bytes(rows, cols)
        pc = vector(codes, "codes", rows * nb * 16, torch.uint8)
        ps = vector(scales, "scales", rows * nb, torch.uint8)

        def run(s, device):
            data = torch.empty(nbytes, dtype=torch.uint8, device=device)
            _check(_abi.mx_lib().fconv_mx_layout(s, pc, ps, rows, cols, data.data_ptr()),
                   "fconv_mx_layout")
            return data
        return cls(call(run, stream, codes, scales), rows, cols)

    @classmethod
    def _of(cls, data, rows, cols):
        """Of a buffer that a plan has just made."""
        t = cls.__new__(cls)
        t.data, t.rows, t.cols = data, rows, cols
        return t


class MxQuantPlan:
    """Quantises [rows, cols] matrices of dtype "bf16" or "fp32", and back."""

    def __init__(self, rows, cols, dtype="bf16"):
        rows, cols = _whole("rows and cols", rows, cols)
        dtype = type_name(dtype)
        self.rows, self.cols, self.dtype = rows, cols, dtype
        if dtype not in TORCH:
            raise ValueError("dtype %r: bf16 or fp32" % (dtype,))
        self._code, self._torch = DTYPES[dtype], TORCH[dtype]
        self.bytes = _mx_bytes(rows, cols)
        L = self._lib = _abi.mx_lib()
        self._call = _abi.native()
        sizes = (rows, cols, self._code, self.bytes)
        self._quantize = (_abi.address(L.fconv_mx_quantize),) + sizes
        self._dequantize = (_abi.address(L.fconv_mx_dequantize),) + sizes

    def __call__(self, x, stream=None):
        rows, cols = self.rows, self.cols
        if stream is None:
            data = self._call.quantize(x, *self._quantize)
            if data is not None:
                return MxTensor._of(done(data, "fconv_mx_quantize"), rows, cols)
        ptr, ld = matrix(x, "x", rows, cols, self._torch)

        def run(s, device):
            data = torch.empty(self.bytes, dtype=torch.uint8, device=device)
            _check(self._lib.fconv_mx_quantize(s, ptr, ld, rows, cols, self._code, data.data_ptr()),
                   "fconv_mx_quantize")
            return data
        return MxTensor._of(call(run, stream, x), rows, cols)

    def dequantize(self, t, stream=None):
        """The values of an MxTensor of this plan's size, in the plan's dtype."""
        rows, cols = self.rows, self.cols
        if t.rows != rows or t.cols != cols:
            raise ValueError("MxTensor of %s, the plan needs %s" % (t.shape, (rows, cols)))
        if stream is None:
            y = self._call.dequantize(t.data, *self._dequantize)
            if y is not None:
                return done(y, "fconv_mx_dequantize")
        ptr = t.address(self.bytes)

        def run(s, device):
            y = torch.empty(rows, cols, dtype=self._torch, device=device)
            _check(self._lib.fconv_mx_dequantize(s, ptr, rows, cols, self._code, y.data_ptr(), cols),
                   "fconv_mx_dequantize")
            return y
        return call(run, stream, t.data)


class MxPlan:
    """y[m, n] = act(sum_k X[m, k] W[n, k] + bias[n]) with X and W in MXFP4.
    A dense layer, or a 1x1 convolution over M = N*H*W pixels.  dtype is the
    type of x and y; ops: [bias], [relu | leaky_relu | clipped_relu | clamp].
    kernel_name is the kernel of a tensor x, quantized_kernel_name that of an
    MxTensor."""

    def __init__(self, M, N, K, dtype="bf16", ops=("bias",)):
        dtype = type_name(dtype)
        d = _abi.MxDesc()
        d.M, d.N, d.K = M, N, K = _whole("M, N and K", M, N, K)
        d.dtype = DTYPES[dtype]
        codes = [OPS[o] if isinstance(o, str) else int(o) for o in ops]
        if len(codes) > _abi.FCONV_MAX_OPS:
            raise ValueError("too many ops")
        d.n_ops = len(codes)
        for i, c in enumerate(codes):
            d.ops[i] = c
        self.desc = d
        self.M, self.N, self.K, self.dtype = M, N, K, dtype
        self._bias = _abi.OP_BIAS in codes
        self._h = ctypes.c_void_p()
        L = self._lib = _abi.mx_lib()
        self._destroy = L.fconv_mx_plan_destroy  # still at hand when the interpreter ends
        _check(L.fconv_mx_plan_create(ctypes.byref(d), ctypes.byref(self._h)), "fconv_mx_plan_create")
        self._torch = TORCH[dtype]
        n = ctypes.c_size_t()
        _check(L.fconv_mx_plan_workspace_size(self._h, ctypes.byref(n)), "fconv_mx_plan_workspace_size")
        self.workspace_bytes = n.value
        self.kernel_name = L.fconv_mx_plan_kernel_name(self._h).decode()
        self.quantized_kernel_name = L.fconv_mx_plan_quantized_kernel_name(self._h).decode()
        self._call = _abi.native()
        self._x_bytes, self._w_bytes = _mx_bytes(M, K), _mx_bytes(N, K)
        self._product = (_abi.address(L.fconv_mx_plan_run), self._h.value, M, N, K, d.dtype, self._w_bytes, n.value)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._destroy(h)
            self._h = None

    def __call__(self, x, w, bias=None, out=None, activ_alpha=0.0, activ_beta=0.0, stream=None):
        """x: a GPU tensor [M, K] (its rows may be apart) or an MxTensor; w: an
        MxTensor [N, K]; bias fp32 [N] with the bias op.  Returns y [M, N] (in
        `out`, whose rows may be apart, if given)."""
        short = stream is None and out is None and activ_alpha == 0.0 and activ_beta == 0.0
        if short and not isinstance(x, MxTensor) and isinstance(w, MxTensor) and w.rows == self.N and \
                w.cols == self.K and self._bias == (bias is not None):
            y = self._call.product(x, w.data, bias, *self._product)
            if y is not None:
                return done(y, "fconv_mx_plan_run")
        a = _abi.MxArgs()
        if isinstance(x, MxTensor):
            if x.rows != self.M or x.cols != self.K:
                raise ValueError("x: MxTensor of %s, the plan needs %s" % (x.shape, (self.M, self.K)))
            a.x_mx = x.address(self._x_bytes)
            x = x.data
        else:
            a.x, a.ldx = matrix(x, "x", self.M, self.K, self._torch)
        if not isinstance(w, MxTensor) or w.rows != self.N or w.cols != self.K:
            raise ValueError("w: an MxTensor of %s needed" % ((self.N, self.K),))
        if self._bias != (bias is not None):
            raise ValueError("bias: the plan has %s bias op" % ("a" if self._bias else "no"))
        a.w_mx = w.address(self._w_bytes)
        if bias is not None:
            a.bias = vector(bias, "bias", self.N, torch.float32)
        a.activ_alpha, a.activ_beta = activ_alpha, activ_beta

        def run(s, device):
            if out is None:
                y = torch.empty(self.M, self.N, dtype=self._torch, device=device)
                a.y, a.ldy = y.data_ptr(), self.N
            else:
                y = out
                a.y, a.ldy = matrix(out, "out", self.M, self.N, self._torch)
            if self.workspace_bytes:
                ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
                a.workspace, a.workspace_bytes = ws.data_ptr(), self.workspace_bytes
            _check(self._lib.fconv_mx_plan_run(self._h, s, ctypes.byref(a)), "fconv_mx_plan_run")
            return y
        return call(run, stream, x, w.data, bias, out)
