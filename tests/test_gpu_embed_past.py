"""The lookup's gradient where dw and dy are more than the last-level cache
holds: rows of zeros then go past it, by 16 bytes from any element on, the last
piece of a row moved back to end with it."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
U = 2.0 ** -24
IGN = -100


# Tokens that a workgroup looks through for its rows, and more of them, which are sorted first; odd and even rows of dw
# at odd places, and dense ones.
@pytest.mark.parametrize("T,D,V,dtype,off,more", [(17000, 1001, 120000, "bf16", 1, 6), (17000, 1001, 120000, "bf16", 0, 0),
                                                  (40000, 501, 240000, "bf16", 3, 2), (40000, 264, 250001, "fp32", 1, 1),
                                                  (9000, 1003, 60001, "fp32", 2, 5)])
def test_zeros_past_the_cache(T, D, V, dtype, off, more):
    dev = device()
    es = 2 if dtype == "bf16" else 4
    assert T * D * es >= 32 << 20 and (T + V) * D * es >= 256 << 20  # where they go past it
    say("embed past", T, D, V, dtype, off, more)
    g = torch.Generator(device=dev).manual_seed(T + D)
    # Many of a few tokens, and rows of zeros between all others.
    token = torch.randint(0, V, (T,), generator=g, device=dev)
    token[::5] = torch.randint(0, 7, (len(token[::5]),), generator=g, device=dev) * (V // 7)
    token[3::11] = IGN
    token[5::13] = V
    dy = torch.randn(T, D, generator=g, device=dev).to(TDT[dtype])
    dy[3::11] = float("nan")
    whole = torch.full((V, off + D + more), 5.0, dtype=TDT[dtype], device=dev)
    dw = whole[:, off:off + D]
    plan = fc.EmbedPlan(T, D, V, dtype, scale=0.5, ignore_index=IGN)
    plan.backward(token, dy, dw=dw)
    again = plan.backward(token, dy)
    torch.cuda.synchronize()
    assert torch.equal(again, dw)
    assert (whole[:, :off] == 5.0).all() and (whole[:, off + D:] == 5.0).all()
    live = (token >= 0) & (token < V)
    at, rows = token[live], dy[live].double()
    count = torch.zeros(V, dtype=torch.float64, device=dev).index_add_(0, at, torch.ones(len(at), dtype=torch.float64, device=dev))
    assert (dw[count == 0].view(torch.int16 if dtype == "bf16" else torch.int32) == 0).all()
    used = torch.nonzero(count).squeeze(1)
    place = torch.full((V,), -1, dtype=torch.int64, device=dev)
    place[used] = torch.arange(len(used), device=dev)
    want = torch.zeros(len(used), D, dtype=torch.float64, device=dev).index_add_(0, place[at], rows) * 0.5
    size = torch.zeros(len(used), D, dtype=torch.float64, device=dev).index_add_(0, place[at], rows.abs()) * 0.5
    # A sum of n terms in fp32, in whatever order, is off by at most n steps of their sizes; then one rounding.
    err = count[used, None] * U * size + (HALF[dtype] + U) * want.abs() + 1e-40
    assert ((dw[used].double() - want).abs() <= err).all()
    # Added to what is there: rows without a token stay as they are.
    before = dw[used].double()
    keep = whole.clone()
    plan.backward(token, dy, dw=dw, accumulate=True)
    keep[used] = whole[used]
    assert torch.equal(keep, whole)
    total = before + want
    assert ((dw[used].double() - total).abs() <= err + (HALF[dtype] + U) * total.abs()).all()
