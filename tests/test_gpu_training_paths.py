"""Paths of the embedding lookup, the gated layer and clipping that a call takes
by its size, each shown to be taken: rows of x that end inside a piece of 16
bytes."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
import test_gpu_gated as tg
from gpu_helpers import device, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,F", [(1862, 76, 4346), (2458, 623, 1344), (171, 130, 15352)])
def test_rows_that_end_inside_a_piece(T, D, F):
    # Rows of x on 16 bytes, their length no whole pieces, NaN behind them and nothing behind the last one: dw's tiles
    # copy whole pieces.  The answer is that of dense rows, bit by bit (both are packed, and multiplied by one kernel).
    dev = device()
    say("rows' ends", T, D, F)
    x, w, dy = tg.case(T, D, F, "bf16", dev)
    p = fc.GatedPlan(T, D, F)
    assert p.kernel_name("dw").startswith("gemm_tile") and p.kernel_name("dw").endswith("_packed")
    y, kept = p.forward(x, w, keep=True)
    dx, dw = p.backward(x, w, kept, dy)
    ld = -(-D // 8) * 8
    memory = torch.full(((T - 1) * ld + D,), float("nan"), dtype=torch.bfloat16, device=dev)
    apart = memory.as_strided((T, D), (ld, 1))
    apart.copy_(x)
    assert torch.isnan(memory[D]) and apart.data_ptr() % 16 == 0
    dx2, dw2 = p.backward(apart, w, kept, dy)
    _, dw3 = p.backward(apart, w, kept, dy, need_dx=False)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(dw3, dw)
