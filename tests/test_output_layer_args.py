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
