"""Which sizes of the GPU tests take the tiled kernels, and what a plan says of
its products (CPU only)."""
import ctypes

import pytest

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi
from test_gpu_tiled_kernels import MX, PIECES, XENT, mx_selection, xent_selection


@pytest.mark.parametrize("row", XENT + PIECES, ids=lambda r: "%dx%dx%d" % r[0])
def test_cross_entropy(row):
    assert xent_selection(row[0])[1] == row


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("row", MX, ids=lambda r: "%dx%dx%d" % r[0])
def test_product(row, dtype):
    assert mx_selection(row[0], dtype)[1] == row


@pytest.mark.parametrize("size,dtype,names", [
    ((64, 452, 1024), "bf16", ("xent_few", "xent_few", "xent_few_grads", "xent_gen_64")),
    ((32, 512, 1000), "fp32", ("xent_few", "xent_few", "xent_few_grads", "xent_gen_64")),
    ((300, 16, 200), "bf16", ("xent_gen_64",) * 4),
    ((8192, 4096, 32768), "bf16", ("xent_tile_256",) * 4),
    ((8192, 4096, 32768), "fp32", ("xent_gen_64",) * 4),
    ((0, 64, 500), "bf16", (None,) * 4)])
def test_names(size, dtype, names):
    p = fc.XentPlan(*size, dtype)
    assert tuple(p.kernel_name(n) for n in ("logits", "grad", "dh", "dw")) == names
    pieces, ranges = p.division("logits")
    assert (pieces, ranges) == ((1, 1) if size[0] else (0, 0))


def test_refusals():
    L = _abi.xent_lib()
    p = fc.XentPlan(4, 40, 9)
    n, m = ctypes.c_int32(), ctypes.c_int32()
    for product in (-1, 4):
        assert L.fconv_xent_plan_kernel_name(p._h, product) is None
        assert L.fconv_xent_plan_division(p._h, product, ctypes.byref(n), ctypes.byref(m)) == _abi.FCONV_ERR_INVALID_ARG
    assert L.fconv_xent_plan_kernel_name(None, 0) is None
    for args in ((None, 0, ctypes.byref(n), ctypes.byref(m)), (p._h, 0, None, ctypes.byref(m)), (p._h, 0, ctypes.byref(n), None)):
        assert L.fconv_xent_plan_division(*args) == _abi.FCONV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        p.kernel_name("loss")
