"""Gradients of losses whose own gradient is infinite or NaN, as
include/fconv_xent.h states them: NaN in all of dw and in the token's dh, the
other tokens' dh as without it."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from test_gpu_xent_pieces import IGN, case

pytestmark = pytest.mark.gpu


# Few tokens with dh's own kernel and with the tiles', general tiles, tiles of 128 with ranges, of 256 without.
@pytest.mark.parametrize("T,D,V", [(1, 40, 90), (20, 64, 300), (40, 64, 9000), (90, 50, 300), (2000, 200, 5000),
                                   (7000, 1288, 1000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_dloss_not_finite(T, D, V, dtype, bad):
    dev = device()
    say("dloss", bad, T, D, V, dtype)
    h, w, t, dl = case(T, D, V, dtype, dev)
    t[0] = 3
    plan = fc.XentPlan(T, D, V, dtype, ignore_index=IGN)
    _, lse = plan.forward(h, w, t)
    dh, _ = plan.backward(h, w, t, lse, dl)
    dl2 = dl.clone()
    dl2[0] = bad
    dh2, dw2 = plan.backward(h, w, t, lse, dl2)
    assert torch.isnan(dw2).all()
    assert torch.isnan(dh2[0]).all()
    assert torch.equal(dh2[1:], dh[1:])
    # Of an ignored token it reaches nothing.
    t[0] = IGN
    _, lse = plan.forward(h, w, t)
    a, b = plan.backward(h, w, t, lse, dl)
    a2, b2 = plan.backward(h, w, t, lse, dl2)
    assert torch.equal(a, a2) and torch.equal(b, b2) and not torch.isnan(b).any()
