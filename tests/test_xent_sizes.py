"""Sizes that the linear softmax cross entropy takes and refuses, as
include/fconv_xent.h states them (CPU only: plans are host objects)."""
import pytest

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,V", [(4096, 8192, 262144), (4096, 12288, 256000), (1, 1024, 1 << 24),
                                   (131072, 4096, 262144), (0, 1 << 20, 1 << 24), (64, 1 << 20, 1 << 20),
                                   (65535 * 64, 2048, 65536), (1, 1 << 20, 1 << 24)])
def test_taken(T, D, V, dtype):
    p = fc.XentPlan(T, D, V, dtype)
    assert p.forward_workspace_bytes <= T * V // 4 + 4096 * T + (2 << 30)


@pytest.mark.parametrize("T,D,V", [(65535 * 64 + 1, 1, 1), (1, 1, (1 << 24) + 1), (1, (1 << 20) + 1, 1),
                                   (65535 * 64, 2049, 10), (1 << 22, 1, 1 << 19), ((1 << 20) + 64, 1, 1 << 20)])
def test_refused(T, D, V):
    with pytest.raises(fc.FconvError) as e:
        fc.XentPlan(T, D, V)
    assert e.value.status == _abi.FCONV_ERR_UNSUPPORTED
