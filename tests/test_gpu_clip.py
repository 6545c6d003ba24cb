"""The norm of many gradients and clipping by it on the GPU against plain numpy
in 64 bits (oracle/clip.py).

Tolerances, u = 2^-24 (half a step of fp32), r = half a step of the type (2^-8
of the value for bf16, u for fp32): squares and sums are in 64 bits, so the norm
is off by its own rounding, u, and by what n additions of 2^-53 make of it; the
factor by that and its own rounding; an output by that, its product's u and r."""
import math

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from oracle import clip as oc

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(sizes, dev, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    kinds = ("bf16", "fp32")
    dts = [kinds[(i * 7 + i // 3) % 2] for i in range(len(sizes))]
    grads = [(torch.randn(n, generator=g) * 10 ** (-spread * torch.rand((), generator=g))).to(TDT[d]).to(dev)
             for n, d in zip(sizes, dts)]
    return grads, dts


def check(plan, grads, dts, max_norm, place):
    values = [_np(g) for g in grads]
    n, want = oc.clip(values, max_norm)
    total = sum(g.numel() for g in grads)
    given = [g.clone() for g in grads]
    out = None if place else [torch.full_like(g, 9.0) for g in grads]
    norm = plan.clip(grads, max_norm, out=out)
    alone = plan.norm(given)
    torch.cuda.synchronize()
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - n) <= (1.01 * U + total * 2.0 ** -53) * n
    assert torch.equal(alone, norm)
    for i, (g, before, w, d) in enumerate(zip(out or grads, given, want, dts)):
        r = 2.0 ** -8 if d == "bf16" else U
        assert (np.abs(_np(g) - w) <= (1.01 * r + 4 * U) * np.abs(w) + 1e-40).all(), i
        if max_norm >= 2 * n:
            assert torch.equal(g, before)
        if not place:
            assert torch.equal(grads[i], before)
    return norm


# A single number; sizes about a thread's, a chunk's and several chunks' ends; empty tensors; more than one launch
# holds; more workgroups than sums that one adds up by itself.
SIZES = [[1], [7], [8, 0, 9], [8191, 8192, 8193], [4095, 4096, 4097, 0], [100000, 3, 1, 70000], [0, 5], [0, 0],
         [1000 + 17 * i for i in range(40)], [1 + i % 13 for i in range(128)], [3] * 129, [50 + i for i in range(300)],
         [5000000, 40], [9000000] * 5 + [20000] * 150]


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("share", [0.01, 0.9, 2.5])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
def test_norm_and_clip(sizes, share, place):
    dev = device()
    say("clip", len(sizes), max(sizes), share, place)
    grads, dts = make(sizes, dev, seed=len(sizes))
    n = oc.norm([_np(g) for g in grads])
    check(fc.ClipPlan([(g.numel(), d) for g, d in zip(grads, dts)]), grads, dts, n * share, place)


@pytest.mark.parametrize("offsets", [(1, 3), (2, 5), (7, 1)])
def test_unaligned_tensors_and_guards(offsets):
    dev = device()
    say("clip unaligned", offsets)
    for dt in ("bf16", "fp32"):
        a = torch.full((9001,), 7.0, dtype=TDT[dt], device=dev)
        b = torch.full((501,), 7.0, dtype=TDT[dt], device=dev)
        x, y = a[offsets[0]:offsets[0] + 8500], b[offsets[1]:offsets[1] + 333]
        x.normal_()
        y.normal_()
        check(fc.ClipPlan([(8500, dt), (333, dt)]), [x, y], [dt, dt], 1.0, True)
        for whole, at, n in ((a, offsets[0], 8500), (b, offsets[1], 333)):
            assert (whole[:at] == 7).all() and (whole[at + n:] == 7).all()


def test_any_order_of_dimensions():
    dev = device()
    say("clip strides")
    x = torch.randn(6, 5, 4, 3, device=dev).to(memory_format=torch.channels_last)
    y = torch.randn(40, 30, device=dev).t()
    out = [torch.empty_like(x), torch.empty_like(y)]
    assert out[0].stride() == x.stride() and out[1].stride() == y.stride()
    check(fc.ClipPlan([(x.numel(), "fp32"), (y.numel(), "fp32")]), [x, y], ["fp32"] * 2, 3.0, False)
    check(fc.ClipPlan([(x.numel(), "fp32"), (y.numel(), "fp32")]), [x, y], ["fp32"] * 2, 3.0, True)


@pytest.mark.parametrize("size", [1e30, 1e-30, 1e-38])
def test_squares_past_fp32(size):
    # Their squares leave fp32's range; the norm does not.
    dev = device()
    say("clip size", size)
    grads = [(torch.randn(5000, device=dev) * size).to(torch.bfloat16), torch.randn(77, device=dev) * size]
    values = [_np(g) for g in grads]
    plan = fc.ClipPlan([(5000, "bf16"), (77, "fp32")], eps=0.0)
    norm = plan.clip(grads, 0.5 * oc.norm(values))
    n = oc.norm(values)
    # A norm below 2^-126 is rounded to a multiple of 2^-149.
    assert abs(float(norm) - n) <= 1.01 * U * n + 2.0 ** -149
    for g, v in zip(grads, values):
        r = 2.0 ** -8 if g.dtype == torch.bfloat16 else U
        assert (np.abs(_np(g) - 0.5 * v) <= (1.01 * r + 4 * U) * np.abs(0.5 * v) + 2.0 ** -133).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite(bad):
    dev = device()
    say("clip", bad)
    x, y = torch.randn(1000, device=dev), torch.randn(50, device=dev).bfloat16()
    x[37] = bad
    plan = fc.ClipPlan([(1000, "fp32"), (50, "bf16")])
    a, b = torch.empty_like(x), torch.empty_like(y)
    norm = plan.clip([x, y], 1.0, out=[a, b])
    if math.isnan(bad):
        assert torch.isnan(norm) and torch.isnan(a).all() and torch.isnan(b).all()
    else:
        assert torch.isinf(norm) and norm > 0
        assert torch.isnan(a[37]) and (a[:37] == 0).all() and (a[38:] == 0).all() and (b == 0).all()
    norm = plan.clip([x, y], math.inf, out=[a, b])
    assert not torch.isfinite(norm)
    assert torch.equal(a.view(torch.int32), x.view(torch.int32)) and torch.equal(b, y)


def test_limits():
    dev = device()
    say("clip limits")
    x = torch.randn(3000, device=dev)
    plan = fc.ClipPlan([(3000, "fp32")])
    keep = x.clone()
    plan.clip([x], math.inf)
    plan.clip([x], 1e300)
    assert torch.equal(x, keep)
    plan.clip([x], 0.0)
    assert (x == 0).all()
    # Nothing to divide by: eps alone is the norm's share.
    assert float(plan.clip([x], 0.5)) == 0.0 and (x == 0).all()


def test_a_given_norm():
    # Two parts of a gradient, clipped by the norm of both.
    dev = device()
    say("clip given norm")
    x, y = torch.randn(70000, device=dev), torch.randn(90, device=dev).bfloat16()
    px, py = fc.ClipPlan([(70000, "fp32")]), fc.ClipPlan([(90, "bf16")])
    norm = torch.stack([px.norm([x]), py.norm([y])]).square().sum().sqrt()
    both = fc.ClipPlan([(70000, "fp32"), (90, "bf16")])
    n, (wx, wy) = oc.clip([_np(x), _np(y)], 3.0)
    out = [torch.empty_like(x), torch.empty_like(y)]
    both.clip([x, y], 3.0, out=out)
    assert px.clip([x], 3.0, norm=norm) is norm
    py.clip([y], 3.0, norm=norm)
    assert (np.abs(_np(x) - wx) <= 8 * U * np.abs(wx)).all()
    assert (np.abs(_np(y) - wy) <= (2.0 ** -8 * 1.01 + 8 * U) * np.abs(wy)).all()
    # By their own norm the answer is that of one call.
    given = [torch.empty_like(x), torch.empty_like(y)]
    keep = [o.clone() for o in out]
    both.clip(keep, 0.7, norm=both.norm(keep), out=given)
    both.clip(keep, 0.7)
    assert torch.equal(keep[0], given[0]) and torch.equal(keep[1], given[1])
