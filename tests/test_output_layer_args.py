"""What the bindings of the output layer's operators accept and refuse before
the C ABI is called (CPU only: plans are host objects)."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi

MAKE = {"MxQuantPlan": lambda t: fc.MxQuantPlan(4, 40, t), "MxPlan": lambda t: fc.MxPlan(4, 8, 40, t),
        "XentPlan": lambda t: fc.XentPlan(4, 40, 9, t)}


@pytest.mark.parametrize("plan", MAKE)
@pytest.mark.parametrize("name,code,dtype", [("bf16", _abi.FCONV_BF16, torch.bfloat16),
                                             ("fp32", _abi.FCONV_FP32, torch.float32)])
def test_a_type_is_a_name_or_its_code(plan, name, code, dtype):
    for given in (name, code):
        p = MAKE[plan](given)
        assert p.dtype == name and p._torch is dtype
        # The plan takes tensors of that type: what is left to complain about is the device.
        x = torch.zeros(4, 40, dtype=dtype)
        with pytest.raises(ValueError, match="GPU"):
            if plan == "MxQuantPlan":
                p(x)
            elif plan == "MxPlan":
                p(x, fc.MxTensor(torch.zeros(1280, dtype=torch.uint8), 8, 40), bias=torch.zeros(8))
            else:
                p.forward(x, torch.zeros(9, 40, dtype=dtype), torch.zeros(4, dtype=torch.int64))


@pytest.mark.parametrize("plan", MAKE)
@pytest.mark.parametrize("bad", ["fp16", 7, -1, None, True, 1.0, (1 << 32) + 1])
def test_other_types_are_refused_by_name(plan, bad):
    with pytest.raises(ValueError, match="dtype"):
        MAKE[plan](bad)


@pytest.mark.parametrize("make", [
    lambda n: fc.MxQuantPlan(n, 40), lambda n: fc.MxQuantPlan(4, n),
    lambda n: fc.MxPlan(n, 8, 40), lambda n: fc.MxPlan(4, n, 40), lambda n: fc.MxPlan(4, 8, n),
    lambda n: fc.MxTensor(torch.zeros(1280, dtype=torch.uint8), n, 40),
    lambda n: fc.MxTensor.from_codes(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), n),
    lambda n: fc.XentPlan(n, 40, 9), lambda n: fc.XentPlan(4, n, 9), lambda n: fc.XentPlan(4, 40, n),
    lambda n: fc.Plan(n, 6, 5, 16, 24, 3, 3), lambda n: fc.Plan(2, 6, 5, 16, 24, 3, n),
    lambda n: fc.Plan(2, 6, 5, 16, 24, 3, 3, stride=(n, 1)), lambda n: fc.WgradPlan(n, 6, 5, 16, 24, 3, 3)])
def test_sizes_past_32_bits_are_refused(make):
    # The descriptors hold 32 bits: 2^32 + 1 was taken for 1.
    with pytest.raises(ValueError, match="32 bits"):
        make((1 << 32) + 1)
    with pytest.raises(ValueError, match="32 bits"):
        make(-(1 << 40))
    with pytest.raises(TypeError):
        make(3.0)


def test_ignore_index_past_64_bits_is_refused():
    assert fc.XentPlan(4, 40, 9, ignore_index=(1 << 63) - 1).ignore_index == (1 << 63) - 1
    with pytest.raises(ValueError, match="64 bits"):
        fc.XentPlan(4, 40, 9, ignore_index=(1 << 64) - 100)


def _mx(rows, cols, nbytes):
    return fc.MxTensor(torch.zeros(nbytes, dtype=torch.uint8), rows, cols)


@pytest.mark.parametrize("data", [torch.zeros(1279, dtype=torch.uint8), torch.zeros(1280, dtype=torch.int8),
                                  torch.zeros(2560, dtype=torch.uint8)[::2]])
def test_a_buffer_that_was_exchanged_is_looked_at_again(data):
    # The size was asked only when the MxTensor was made; kernels read it all.
    p = fc.MxPlan(4, 8, 40, "fp32", ops=())
    x, w = _mx(4, 40, 1280), _mx(8, 40, 1280)
    x.data = data
    with pytest.raises(ValueError, match="1280 bytes"):
        p(x, w)
    x, w.data = _mx(4, 40, 1280), data
    with pytest.raises(ValueError, match="1280 bytes"):
        p(x, w)
    with pytest.raises(ValueError, match="1280 bytes"):
        fc.MxQuantPlan(8, 40, "fp32").dequantize(w)


@pytest.mark.parametrize("M,N,K,given,quantized", [(1, 1000, 512, "mx_few_raw", "mx_few"), (500, 200, 512, "mx_rows", "mx_tile_128"),
                                                   (40, 100, 260, "mx_rows", "mx_few"), (32, 1024, 25088, "mx_few", "mx_few"),
                                                   (8192, 8192, 4096, "mx_tile_256", "mx_tile_256")])
def test_kernel_names_of_a_tensor_and_of_a_quantised_x(M, N, K, given, quantized):
    # A run whose x comes quantised was said to take a kernel that quantises x itself.
    p = fc.MxPlan(M, N, K, "bf16")
    assert (p.kernel_name, p.quantized_kernel_name) == (given, quantized)
    assert _abi.mx_lib().fconv_mx_plan_quantized_kernel_name(None) is None
