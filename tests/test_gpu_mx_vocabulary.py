"""MXFP4 products of few tokens with the weights of a large vocabulary, past the
caches, in 64 bits on the GPU (tolerance: 4 u K s with u = 2^-24 and s the root
mean square of an output's products, half a step of bf16)."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from test_gpu_xent_pieces import sum_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K", [(128256, 4096), (65537, 16388)])
def test_few_tokens(N, K):
    dev = device()
    g = torch.Generator(device=dev).manual_seed(1)
    qw = fc.MxQuantPlan(N, K, "fp32")
    w = qw(torch.randn(N, K, generator=g, device=dev))
    wv = qw.dequantize(w)  # exact, see test_gpu_mx.py
    for M in (1, 3, 5, 16, 33, 64):
        plan = fc.MxPlan(M, N, K, "bf16", ops=())
        say("few tokens of a vocabulary", M, N, K, plan.kernel_name, plan.quantized_kernel_name)
        x = torch.randn(M, K, generator=g, device=dev).bfloat16()
        qx = fc.MxQuantPlan(M, K, "bf16")
        x4 = qx(x)
        y, y4 = plan(x, w), plan(x4, w)
        xv = qx.dequantize(x4).double()
        for n in range(0, N, 16384):
            s = slice(n, n + 16384)
            wd = wv[s].double().t()
            ref = torch.mm(xv, wd)
            bound = sum_error(xv, wd, K) + 2.0 ** -8 * ref.abs() + 1e-37
            assert bool(((y[:, s].double() - ref).abs() <= bound).all())
            assert bool(((y4[:, s].double() - ref).abs() <= bound).all())
