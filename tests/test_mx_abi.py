"""MXFP4, no GPU: the oracle's pins, the C ABI's host checks and the
binding's refusals (failing runs return before anything is enqueued, so the
fake device addresses are never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi
from oracle import mx as omx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = (
    _abi.FCONV_OK, _abi.FCONV_ERR_INVALID_ARG, _abi.FCONV_ERR_UNSUPPORTED, _abi.FCONV_ERR_WORKSPACE,
    _abi.FCONV_ERR_MISALIGNED)


# --- the oracle -----------------------------------------------------------

def test_oracle_rounds_to_nearest_even_code():
    # In a block whose largest value is 4 the scale is 1: values and codes by hand.
    x = np.zeros((1, 32))
    x[0, :16] = [4, 0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 1.74, 2.5, 2.51, 3.5, 3.49, -0.25, -5 / 2, -3.5]
    codes, scales = omx.quantize(x)
    assert scales[0, 0] == 127
    got = omx.values(codes, scales, 32)[0, :16]
    assert got.tolist() == [4, 0, 0.5, 1, 0.5, 1, 1.5, 2, 1.5, 2, 3, 4, 3, 0, -2, -4]


def test_oracle_saturates_between_six_and_eight():
    x = np.zeros((1, 32))
    x[0, :4] = [7.9, 5.0, 5.1, -7.0]
    assert omx.values(*omx.quantize(x), 4)[0].tolist() == [6, 4, 6, -6]


@pytest.mark.parametrize("v,byte", [(6.0, 127), (8.0, 128), (1.0, 125), (2.0 ** -126, 0), (2.0 ** -149, 0),
                                    (3.0e38, 252), (0.0, 0), (np.inf, 255), (np.nan, 255)])
def test_oracle_scale_bytes(v, byte):
    x = np.zeros((1, 32))
    x[0, 5] = v
    assert omx.quantize(x)[1][0, 0] == byte


def test_oracle_keeps_representable_values():
    rng = np.random.default_rng(0)
    v = rng.choice(omx.VALUES, (5, 96)) * rng.choice([-1, 1], (5, 96)) * 2.0 ** 9
    v[:, ::32] = 6 * 2.0 ** 9
    assert np.array_equal(omx.values(*omx.quantize(v), 96), v)


# --- the C ABI ------------------------------------------------------------

def test_header_and_exports_agree():
    text = open(os.path.join(ROOT, "include", "fconv_mx.h")).read()
    declared = set(re.findall(r"FCONV_API\s+[\w\s\*]+?\b(fconv_\w+)\s*\(", text))
    assert declared == set(_abi.MX_EXPORTS)
    lib = ctypes.CDLL(_abi.lib_path())
    for name in declared:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("rows,cols,n", [(1, 1, 1024 + 256), (16, 128, 1280), (17, 128, 2560),
                                         (16, 513, 5 * 1024 + 512), (0, 9, 0)])
def test_bytes(rows, cols, n):
    b = ctypes.c_size_t()
    assert _abi.mx_lib().fconv_mx_bytes(rows, cols, ctypes.byref(b)) == OK
    assert b.value == n


def test_bytes_refuses():
    L, b = _abi.mx_lib(), ctypes.c_size_t()
    assert L.fconv_mx_bytes(1, 0, ctypes.byref(b)) == INVALID
    assert L.fconv_mx_bytes(-1, 4, ctypes.byref(b)) == INVALID
    assert L.fconv_mx_bytes(1, 1, None) == INVALID
    assert L.fconv_mx_bytes(1, (1 << 22) + 1, ctypes.byref(b)) == UNSUPPORTED


@pytest.mark.parametrize("fn", ["fconv_mx_quantize", "fconv_mx_dequantize"])
def test_quantize_refuses(fn):
    def call(x=FAKE, ld=64, rows=4, cols=64, dtype=1, mx=FAKE * 2):
        L = _abi.mx_lib()
        if fn == "fconv_mx_quantize":
            return L.fconv_mx_quantize(None, x, ld, rows, cols, dtype, mx)
        return L.fconv_mx_dequantize(None, mx, rows, cols, dtype, x, ld)
    assert call(x=None) == INVALID
    assert call(mx=None) == INVALID
    assert call(ld=63) == INVALID
    assert call(rows=-1) == INVALID
    assert call(cols=0) == INVALID
    assert call(dtype=0) == UNSUPPORTED
    assert call(dtype=3) == UNSUPPORTED
    assert call(x=FAKE + 1) == MISALIGNED
    assert call(x=FAKE + 2, dtype=2) == MISALIGNED
    assert call(mx=FAKE * 2 + 8) == MISALIGNED
    assert call(mx=FAKE + 64) == INVALID  # overlap
    assert call(rows=2147483647, cols=1 << 22, ld=1 << 22) == UNSUPPORTED
    assert call(rows=0, mx=None) == OK


def test_layout_refuses():
    def call(codes=FAKE, scales=FAKE * 2, rows=4, cols=64, mx=FAKE * 4):
        return _abi.mx_lib().fconv_mx_layout(None, codes, scales, rows, cols, mx)
    assert call(codes=None) == INVALID
    assert call(scales=None) == INVALID
    assert call(mx=None) == INVALID
    assert call(rows=-1) == INVALID
    assert call(cols=0) == INVALID
    assert call(codes=FAKE + 2) == MISALIGNED
    assert call(mx=FAKE * 4 + 4) == MISALIGNED
    assert call(mx=FAKE) == INVALID
    assert call(mx=FAKE * 2) == INVALID
    assert call(rows=0) == OK


def _create(ops=(3,), **kw):
    d = _abi.MxDesc()
    for k, v in dict(dict(M=4, N=8, K=64, dtype=1, flags=0), **kw).items():
        setattr(d, k, v)
    d.n_ops = kw.get("n_ops", len(ops))
    for i, o in enumerate(ops[:8]):
        d.ops[i] = o
    h = ctypes.c_void_p()
    return _abi.mx_lib().fconv_mx_plan_create(ctypes.byref(d), ctypes.byref(h)), h


def test_plan_refuses():
    L = _abi.mx_lib()
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(n_ops=-1), dict(n_ops=9)):
        assert _create(**kw)[0] == INVALID, kw
    for kw in (dict(dtype=0), dict(dtype=5), dict(flags=1), dict(K=(1 << 22) + 1),
               dict(M=2147483647, N=2147483647), dict(ops=(5, 3)), dict(ops=(3, 4)), dict(ops=(1, 3)),
               dict(ops=(5, 6)), dict(ops=(3, 3))):
        assert _create(**kw)[0] == UNSUPPORTED, kw
    assert L.fconv_mx_plan_create(None, None) == INVALID
    assert L.fconv_mx_plan_destroy(None) == OK
    assert L.fconv_mx_plan_kernel_name(None) is None
    assert L.fconv_mx_plan_workspace_size(None, None) == INVALID


def test_run_refuses():
    L = _abi.mx_lib()
    st, h = _create(M=40, N=24, K=4096, ops=(3, 8))
    assert st == OK
    n = ctypes.c_size_t()
    assert L.fconv_mx_plan_workspace_size(h, ctypes.byref(n)) == OK and n.value > 0

    def run(**kw):
        a = _abi.MxArgs()
        base = dict(x=FAKE, ldx=4096, w_mx=2 * FAKE, bias=3 * FAKE, y=4 * FAKE, ldy=24, workspace=5 * FAKE,
                    workspace_bytes=n.value, activ_alpha=0.0, activ_beta=1.0)
        for k, v in dict(base, **kw).items():
            setattr(a, k, v)
        return L.fconv_mx_plan_run(h, None, ctypes.byref(a))
    for kw in (dict(x=None), dict(x_mx=6 * FAKE), dict(w_mx=None), dict(bias=None), dict(y=None),
               dict(ldx=4095), dict(ldy=23), dict(y=FAKE), dict(y=2 * FAKE), dict(y=3 * FAKE),
               dict(y=5 * FAKE), dict(workspace=FAKE), dict(activ_alpha=2.0),
               dict(activ_alpha=float("nan")), dict(activ_beta=float("inf"))):
        assert run(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 1), dict(y=4 * FAKE + 1), dict(w_mx=2 * FAKE + 8), dict(bias=3 * FAKE + 2),
               dict(workspace=5 * FAKE + 4)):
        assert run(**kw) == MISALIGNED, kw
    if n.value:
        assert run(workspace=None) == WORKSPACE
        assert run(workspace_bytes=n.value - 1) == WORKSPACE
    assert L.fconv_mx_plan_run(None, None, None) == INVALID
    assert L.fconv_mx_plan_destroy(h) == OK


def test_empty_product_is_a_no_op():
    st, h = _create(M=0)
    assert st == OK
    a = _abi.MxArgs()
    assert _abi.mx_lib().fconv_mx_plan_run(h, None, ctypes.byref(a)) == OK
    _abi.mx_lib().fconv_mx_plan_destroy(h)


# --- the binding ----------------------------------------------------------

def _mx(rows, cols):
    n = ctypes.c_size_t()
    _abi.mx_lib().fconv_mx_bytes(rows, cols, ctypes.byref(n))
    return fc.MxTensor(torch.zeros(n.value, dtype=torch.uint8), rows, cols)


def test_binding_refuses():
    q = fc.MxQuantPlan(4, 40, "fp32")
    with pytest.raises(ValueError, match="dtype"):
        q(torch.zeros(4, 40, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape"):
        q(torch.zeros(4, 41))
    with pytest.raises(ValueError, match="dense"):
        q(torch.zeros(40, 4).t())
    with pytest.raises(ValueError, match="dense"):
        q(torch.zeros(1, 40).expand(4, 40))
    with pytest.raises(ValueError, match="GPU"):
        q(torch.zeros(4, 40))
    with pytest.raises(ValueError, match="dtype"):
        fc.MxQuantPlan(4, 40, "int8")
    with pytest.raises(ValueError, match="MxTensor"):
        q.dequantize(_mx(4, 41))
    with pytest.raises(ValueError, match="bytes"):
        fc.MxTensor(torch.zeros(1279, dtype=torch.uint8), 1, 1)
    with pytest.raises(ValueError, match="codes"):
        fc.MxTensor.from_codes(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), 40)
    p = fc.MxPlan(4, 8, 40, "fp32", ops=("bias", "relu"))
    w, b = _mx(8, 40), torch.zeros(8)
    with pytest.raises(ValueError, match="bias"):
        p(_mx(4, 40), w)
    with pytest.raises(ValueError, match="w:"):
        p(_mx(4, 40), _mx(4, 40), bias=b)
    with pytest.raises(ValueError, match="x:"):
        p(_mx(4, 41), w, bias=b)
    with pytest.raises(ValueError, match="GPU"):
        p(torch.zeros(4, 40), w, bias=b)
    with pytest.raises(fc.FconvError):
        fc.MxPlan(4, 8, 40, "int8")
    with pytest.raises(fc.FconvError):
        fc.MxPlan(4, 0, 40)


# --- sizes at the ends of what the checks let through ----------------------

def test_strides_past_the_address_space_are_refused():
    far = (1 << 62) // 4
    L = _abi.mx_lib()
    assert L.fconv_mx_quantize(None, FAKE, far, 9, 64, 1, 2 * FAKE) == INVALID
    assert L.fconv_mx_dequantize(None, 2 * FAKE, 9, 64, 2, FAKE, far) == INVALID
    st, h = _create(M=40, N=24, K=96, ops=())
    assert st == OK
    a = _abi.MxArgs()
    a.x, a.w_mx, a.y, a.ldx, a.ldy = FAKE, 2 * FAKE, 4 * FAKE, far, 24
    assert L.fconv_mx_plan_run(h, None, ctypes.byref(a)) == INVALID
    a.ldx, a.ldy = 96, far
    assert L.fconv_mx_plan_run(h, None, ctypes.byref(a)) == INVALID
    L.fconv_mx_plan_destroy(h)


def test_few_rows_of_very_many_outputs_stay_a_legal_launch():
    # 2^29 outputs would be 2^24 workgroups of the few-rows kernel, 2^32 threads.
    st, h = _create(M=1, N=1 << 29, K=32, ops=())
    assert st == OK
    assert _abi.mx_lib().fconv_mx_plan_kernel_name(h) not in (b"mx_few", b"mx_few_raw")
    _abi.mx_lib().fconv_mx_plan_destroy(h)


def test_quantised_matrices_of_the_host_are_refused():
    p = fc.MxPlan(4, 8, 40, "fp32", ops=())
    with pytest.raises(ValueError, match="GPU"):
        p(_mx(4, 40), _mx(8, 40))
    with pytest.raises(ValueError, match="GPU"):
        fc.MxQuantPlan(4, 40, "fp32").dequantize(_mx(4, 40))
