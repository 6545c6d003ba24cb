"""Every code under every scale byte, as a checkpoint may hold them: the values
are exact (numpy in 64 bits, rounded once to the output's type)."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from oracle import mx as omx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_code_under_every_scale(dtype):
    dev = device()
    say("codes and scales", dtype)
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    t = fc.MxTensor.from_codes(torch.from_numpy(omx.pack(codes)).to(dev), torch.from_numpy(scales).to(dev), 32)
    got = fc.MxQuantPlan(256, 32, dtype).dequantize(t)
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(omx.values(codes, scales, 32).astype(np.float32))  # past fp32's range: infinities
    assert torch.isinf(ref[253]).any() and torch.isinf(ref[254]).any() and torch.isnan(ref[255]).all()
    assert not torch.isinf(ref[:253]).any()
    ref = ref.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    assert np.array_equal(got.float().cpu().numpy(), ref.float().numpy(), equal_nan=True)


@pytest.mark.parametrize("M", [1, 16, 200])
def test_products_of_every_scale(M):
    # Row n of W has scale byte n and 32 codes of 1; x undoes the scale as far as fp32 goes.
    dev = device()
    say("product of every scale", M)
    codes = np.full((255, 32), 2, np.uint8)
    scales = np.arange(255, dtype=np.uint8).reshape(255, 1)
    w = fc.MxTensor.from_codes(torch.from_numpy(omx.pack(codes)).to(dev), torch.from_numpy(scales).to(dev), 32)
    plan = fc.MxPlan(M, 255, 32, "fp32", ops=())
    for e in (-100, 0, 100):
        y = plan(torch.full((M, 32), 2.0 ** e, device=dev), w)
        ref = 32.0 * np.exp2(np.arange(255) - 127.0 + e)
        live = (ref >= 2.0 ** -126) & (ref < 2.0 ** 128)  # beyond: the matrix cores' way with subnormals, infinities
        got = y.double().cpu().numpy()
        assert (got[:, live] == ref[live]).all()
        assert np.isinf(got[:, ref >= 2.0 ** 128]).all()
