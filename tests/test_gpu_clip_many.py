"""Clipping so many gradients that their sums are added up by a launch of its
own before the scaling reads the norm; as tests/test_gpu_clip.py derives its
errors."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
import test_gpu_clip as tc
from gpu_helpers import device, say
from oracle import clip as oc

pytestmark = pytest.mark.gpu

# A launch holds 128 tensors and has up to 512 workgroups, each with a sum; every workgroup of the scaling adds up
# 2048 by itself, two rounds of eight of each of its 256 threads.
OWN = 2048
SIZES = [[70000] * 650, [64000 + 31 * i for i in range(520)], [200000] * 1300, [0, 70001] * 700]


def test_sums_are_more_than_a_workgroup_adds_up():
    for sizes in SIZES:
        plan = fc.ClipPlan([(n, "bf16") for n in sizes])
        assert plan.workspace_bytes > OWN * 8 + 16, len(sizes)
    # Past the first round of loads of such a launch, too.
    assert fc.ClipPlan([(200000, "bf16")] * 1300).workspace_bytes > 2 * OWN * 8 + 16


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("share", [0.3, 2.5])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
def test_norm_and_clip(sizes, share, place):
    dev = device()
    say("clip many", len(sizes), max(sizes), share, place)
    grads, dts = tc.make(sizes, dev, seed=len(sizes))
    plan = fc.ClipPlan([(g.numel(), d) for g, d in zip(grads, dts)])
    assert plan.workspace_bytes > OWN * 8 + 16
    n = oc.norm([tc._np(g) for g in grads])
    tc.check(plan, grads, dts, n * share, place)


def test_from_one_workgroup_to_all_of_them_by_itself():
    # Sums about a round of a workgroup's loads, and one more launch than it takes: 2048 and 2050 or more.
    dev = device()
    for count in (512, 513, 514):
        say("clip", count)
        sizes = [70000] * count
        grads = [torch.randn(n, device=dev).bfloat16() for n in sizes]
        plan = fc.ClipPlan([(n, "bf16") for n in sizes])
        sums = (plan.workspace_bytes - 16) // 8
        assert (sums <= OWN) == (count == 512)
        n = oc.norm([tc._np(g) for g in grads])
        tc.check(plan, grads, ["bf16"] * count, 0.5 * n, True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite(bad):
    dev = device()
    say("clip many", bad)
    grads = [torch.ones(70000, device=dev) for _ in range(650)]
    grads[649][69999] = bad
    plan = fc.ClipPlan([(70000, "fp32")] * 650)
    norm = plan.clip(grads, 1.0)
    if bad != bad:
        assert torch.isnan(norm) and all(bool(torch.isnan(g).all()) for g in (grads[0], grads[300], grads[649]))
    else:
        assert torch.isinf(norm) and (grads[0] == 0).all() and torch.isnan(grads[649][69999]) and (grads[649][:-1] == 0).all()


def test_same_bits_on_every_run_streams_and_graphs():
    dev = device()
    say("clip many, same bits")
    grads = [torch.randn(70000, device=dev).bfloat16() for _ in range(650)]
    plan = fc.ClipPlan([(70000, "bf16")] * 650)

    def run(stream=None):
        if stream is not None:
            torch.cuda.current_stream().synchronize()
        out = [torch.empty_like(g) for g in grads]
        norm = plan.clip(grads, 0.5, out=out, stream=stream)
        return norm, plan.norm(grads, stream=stream), out[0], out[649]
    want = run()

    def same(got):
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    same(run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    same(run(side))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    with torch.cuda.graph(other):
        out2 = run()
    for _ in range(3):
        graph.replay()
        same(run())
        other.replay()
        same(out)
        same(out2)
    for g in grads:
        g.mul_(0.5)
    want = run()
    graph.replay()
    same(out)
