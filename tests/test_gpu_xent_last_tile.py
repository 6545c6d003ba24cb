"""Cross entropy by the general kernel where the last tile of 64 tokens is partly
empty, some of its waves wholly; errors as tests/test_gpu_xent.py derives them."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
import test_gpu_xent as tx
from gpu_helpers import device, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [1, 35, 200])
@pytest.mark.parametrize("T", [1, 16, 17, 32, 33, 48, 49, 64, 65, 80, 81, 112, 113, 129])
def test_every_number_of_empty_waves(T, D, dtype):
    # NaN behind the last token's row and its lse, target and dloss: no other row's answer may hold any of it.
    dev = device()
    V = 20011
    say("last tile", T, D, dtype)
    h, w, t, dl = tx._case(T, D, V, dtype, T + D, dev)
    t[0] = V - 1
    rows = torch.full((T + 70, D), float("nan"), dtype=h.dtype, device=dev)
    rows[:T] = h
    plan = fc.XentPlan(T, D, V, dtype, ignore_index=tx.IGN)
    if T > 64 and D < 200:
        assert plan.kernel_name("logits") == plan.kernel_name("grad") == "xent_gen_64"
    tx._check(rows[:T], w, t, dl, dtype, plan)
    # Each token by itself has the same loss, whatever tile and wave it is in.
    loss, lse = plan.forward(h, w, t)
    turned = torch.arange(T - 1, -1, -1, device=dev)
    loss2, lse2 = plan.forward(h[turned].contiguous(), w, t[turned])
    assert torch.equal(loss, loss2[turned]) and torch.equal(lse, lse2[turned])
