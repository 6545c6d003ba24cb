"""Paths of the gated layer that a call takes by its size, each shown to be taken:
rows of x that end inside a piece of 16 bytes; packed rows, ranges and both
gradients in one launch of tiles, on streams, in graphs, at once and alone."""
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


# --- the same bits, of the paths that copies, ranges and joins make longest ---------

# Kernels of the forward pass, dx and dw, and the ranges of dx's sum (0: one).
PATHS = [(1862, 76, 4346, ("gemm_tile_128_packed",) * 3, True), (2458, 623, 1344, ("gemm_tile_128_packed",) * 3, False),
         (1999, 1000, 2731, ("gemm_tile_256",) * 3, True), (330, 32, 11350, ("gemm_tile_256", "gemm_tile_128", "gemm_tile_128"), True),
         (171, 130, 15352, ("gemm_gen_64", "gemm_tile_256_packed", "gemm_tile_256_packed"), True)]


def _path(T, D, F, names, parts):
    p = fc.GatedPlan(T, D, F, activation="gelu")
    assert tuple(p.kernel_name(n) for n in ("forward", "dx", "dw")) == names
    assert (p.ranges("dx") > 1) == parts
    return p


@pytest.mark.parametrize("T,D,F,names,parts", PATHS)
def test_same_bits_on_every_run_streams_and_graphs(T, D, F, names, parts):
    dev = device()
    say("same bits:", T, D, F, names)
    p = _path(T, D, F, names, parts)
    x, w, dy = tg.case(T, D, F, "bf16", dev)

    def run(stream=None):
        y, kept = p.forward(x, w, keep=True, stream=stream)
        dx, dw = p.backward(x, w, kept, dy, stream=stream)
        return y, dx, dw, p.forward(x, w, stream=stream)
    want = run()

    def same(got):
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    same(run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    same(run(side))
    same(run(side.cuda_stream))
    with torch.cuda.stream(side):
        same(run())
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
    for t in (x, w, dy):
        t.mul_(0.5)
    want = run()
    graph.replay()
    same(out)


@pytest.mark.parametrize("T,D,F,names,parts", PATHS)
def test_calls_at_once_on_two_streams(T, D, F, names, parts):
    # One plan, calls under way on two streams: each has its own outputs and workspace.
    dev = device()
    say("two streams:", T, D, F)
    p = _path(T, D, F, names, parts)
    x, w, dy = tg.case(T, D, F, "bf16", dev)

    def run():
        y, kept = p.forward(x, w, keep=True)
        return (y,) + p.backward(x, w, kept, dy)
    want = run()
    torch.cuda.synchronize()
    streams, got = (torch.cuda.Stream(), torch.cuda.Stream()), []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,D,F,names,parts", PATHS)
def test_one_gradient_alone(T, D, F, names, parts):
    dev = device()
    say("one gradient:", T, D, F)
    p = _path(T, D, F, names, parts)
    x, w, dy = tg.case(T, D, F, "bf16", dev)
    _, kept = p.forward(x, w, keep=True)
    dx, dw = p.backward(x, w, kept, dy)
    assert torch.equal(p.backward(x, w, kept, dy, need_dw=False)[0], dx)
    assert torch.equal(p.backward(x, w, kept, dy, need_dx=False)[1], dw)
