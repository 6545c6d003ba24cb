"""What a gradient of the linear softmax cross entropy needs beside its inputs
and outputs (CPU only: plans are host objects)."""
import pytest

import convolution_implicit_gemm_nhwc_amd as fc

M = 512 << 20


def _round(n, m):
    return -(-n // m) * m


@pytest.mark.parametrize("dtype,es", [("bf16", 2), ("fp32", 4)])
@pytest.mark.parametrize("T,D,V", [(32768, 4096, 128256), (32768, 8192, 128256), (65536, 4096, 128256),
                                   (65536, 8192, 128256), (65536, 8192, 50021), (100000, 4096, 100000),
                                   (100000, 512, 100000), (16384, 4096, 128256), (8192, 512, 65536),
                                   (1000, 1000, 1000000), (64, 100, 1 << 24), (2048, 60000, 30000)])
def test_backward_workspace_is_linear_in_the_tokens(T, D, V, dtype, es):
    # A piece of q (at least 256 columns), h of the live tokens twice, one fp32 dh or its ranges, the ranges of
    # dw, a packed piece of w, and some scalars of each token.
    b = fc.XentPlan(T, D, V, dtype).backward_workspace_bytes
    q = max(M, T * 256 * es)
    dh = max(M, 4 * T * _round(D, 4))
    pack = 2 * M if D % 8 else 0
    assert b <= q + 2 * es * T * _round(D, 64) + dh + M + pack + 32 * T + (1 << 16)
    # Below the logits, which are not kept, wherever those are many to a token.
    if V >= 8 * D and T * V * es > 4 * M:
        assert b < T * V * es, (b, T * V * es)


def test_backward_workspace_of_a_long_batch_over_a_large_vocabulary():
    # 8.4 GB of bf16 logits; one dh for each piece of the vocabulary made this 18.8 GB.
    assert fc.XentPlan(32768, 8192, 128256).backward_workspace_bytes < 3 << 30
