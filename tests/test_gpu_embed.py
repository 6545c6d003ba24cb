"""The embedding lookup and its gradient on the GPU against plain numpy in 64
bits (oracle/embed.py).

Tolerances, u = 2^-24 (half a step of fp32), r = half a step of the type (2^-8
of the value for bf16, u for fp32): a value of y is one fp32 product, rounded
to the type; a row's sum of n terms takes n - 1 additions in fp32, each off by u
of a partial sum that is no larger than the sum of the terms' sizes, then the
scale, then the type's rounding."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from oracle import embed as oe

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
IGN = -100


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def tokens(T, V, kind, seed=0):
    g = torch.Generator().manual_seed(seed + T + V)
    if kind == "even":
        t = torch.randint(0, V, (T,), generator=g)
    elif kind == "text":  # rank about even in its logarithm
        t = (V ** torch.rand(T, generator=g, dtype=torch.float64)).long().sub(1).clamp(0, V - 1)
    else:  # one token
        t = torch.full((T,), V // 2)
    t[torch.rand(T, generator=g) < 0.1] = IGN
    return t


def _half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else U


def check_backward(plan, token, dy, V, dtype, scale, before=None, **kw):
    dw = plan.backward(token, dy, **kw)
    torch.cuda.synchronize()
    t, d = token.cpu().numpy(), _np(dy)
    want = oe.backward(t, d, V, scale, IGN)
    size = oe.backward(t, np.abs(d), V, abs(scale), IGN)
    ok = (t >= 0) & (t < V) & (t != IGN)
    n = np.bincount(t[ok], minlength=V)[:, None]
    if before is not None:
        want = want + before
    err = (n + 2) * U * size + _half(dtype) * np.abs(want) + (U * np.abs(want) if before is not None else 0)
    off = np.abs(_np(dw) - want)
    assert (off <= err).all(), (float((off - err).max()), np.argwhere(~(off <= err))[:4])
    if before is None:
        assert (dw[torch.from_numpy(n[:, 0] == 0)] == 0).all()
    return dw


# One token; the last numbers that a workgroup sorts by itself and the first that it does not; ends of a ranked chunk
# and of sixteen of them; columns of less than 16 bytes, of one thread's, of a team's and of several workgroups'.
SIZES = [(1, 1, 1), (1, 64, 500), (2, 3, 7), (5, 8, 40), (64, 33, 100), (255, 72, 50), (256, 100, 1000), (257, 100, 1000),
         (300, 1, 9), (1000, 130, 333), (1999, 1000, 3201), (4095, 24, 700), (4096, 40, 5000), (4097, 40, 5000), (5000, 65, 1),
         (9000, 16, 30), (40, 2500, 300), (600, 5000, 70), (65536, 8, 2000), (65537, 5, 3000), (70001, 12, 100)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["even", "text", "one"])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_lookup_and_gradient(T, D, V, kind, dtype):
    dev = device()
    scale = 1.0 if T % 2 else 22.5
    say("embed", T, D, V, kind, dtype, scale)
    g = torch.Generator().manual_seed(T + D)
    w = torch.randn(V, D, generator=g).to(TDT[dtype]).to(dev)
    dy = torch.randn(T, D, generator=g).to(TDT[dtype]).to(dev)
    token = tokens(T, V, kind).to(dev)
    plan = fc.EmbedPlan(T, D, V, dtype, scale=scale, ignore_index=IGN)
    y = plan.forward(w, token)
    want = oe.forward(_np(w), token.cpu().numpy(), scale, IGN)
    assert (np.abs(_np(y) - want) <= (0 if scale == 1.0 else _half(dtype) + U) * np.abs(want)).all()
    # A row of an ignored token's dy reaches nothing.
    dy[(token == IGN)] = float("nan")
    d0 = torch.where((token == IGN)[:, None], torch.zeros_like(dy), dy)
    dw = plan.backward(token, dy)
    assert torch.equal(dw, check_backward(plan, token, d0, V, dtype, scale))
    # Added to what is there, rows without a token as they were.
    base = torch.randn(V, D, generator=g).to(TDT[dtype]).to(dev)
    kept = base.clone()
    check_backward(plan, token, d0, V, dtype, scale, before=_np(kept), dw=base, accumulate=True)
    idle = torch.ones(V, dtype=torch.bool, device=dev)
    idle[token[token != IGN]] = False
    assert torch.equal(base[idle], kept[idle])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [7, 700])
def test_tokens_outside_the_table(T, dtype):
    dev = device()
    say("embed outside", T, dtype)
    V, D = 50, 40
    token = tokens(T, V, "even")
    token[:5] = torch.tensor([-1, V, V + 3, -(1 << 40), (1 << 32) + 1])
    token = token.to(dev)
    w = torch.randn(V, D, device=dev).to(TDT[dtype])
    dy = torch.randn(T, D, device=dev).to(TDT[dtype])
    plan = fc.EmbedPlan(T, D, V, dtype, scale=2.0, ignore_index=IGN)
    y = plan.forward(w, token)
    assert torch.isnan(y[:5]).all() and not torch.isnan(y[5:]).any()
    check_backward(plan, token, dy, V, dtype, 2.0)


@pytest.mark.parametrize("T", [6, 600])
def test_ignore_index_of_the_table(T):
    # An ignore_index that is a row of the table: that row is neither read nor given a gradient.
    dev = device()
    say("embed padding row", T)
    V, D = 20, 24
    w = torch.randn(V, D, device=dev)
    w[0] = float("nan")
    token = torch.arange(T, device=dev) % V
    dy = torch.randn(T, D, device=dev)
    plan = fc.EmbedPlan(T, D, V, "fp32", ignore_index=0)
    y = plan.forward(w, token)
    assert (y[token == 0] == 0).all() and torch.equal(y[token != 0], w[token[token != 0]])
    dw = plan.backward(token, dy)
    assert (dw[0] == 0).all() and (dw[1] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [30, 900])
def test_rows_apart_unaligned_and_guards(T, dtype):
    dev = device()
    say("embed strided", T, dtype)
    V, D = 120, 77
    token = tokens(T, V, "text").to(dev)
    w = torch.randn(V, D + 4, device=dev).to(TDT[dtype])[:, 3:3 + D]
    dy = torch.randn(T, D + 6, device=dev).to(TDT[dtype])[:, 1:1 + D]
    by = torch.full((T, D + 8), 7.0, dtype=TDT[dtype], device=dev)
    bw = torch.full((V, D + 2), 7.0, dtype=TDT[dtype], device=dev)
    plan = fc.EmbedPlan(T, D, V, dtype, scale=0.5, ignore_index=IGN)
    plan.forward(w, token, y=by[:, 5:5 + D])
    want = oe.forward(_np(w), token.cpu().numpy(), 0.5, IGN)
    assert (np.abs(_np(by[:, 5:5 + D]) - want) <= (_half(dtype) + U) * np.abs(want)).all()
    assert (by[:, :5] == 7).all() and (by[:, 5 + D:] == 7).all()
    check_backward(plan, token, dy, V, dtype, 0.5, dw=bw[:, 1:1 + D])
    assert (bw[:, :1] == 7).all() and (bw[:, 1 + D:] == 7).all()
