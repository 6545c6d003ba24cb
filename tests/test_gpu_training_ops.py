"""The embedding lookup, the gated layer and clipping: the same bits on every
run, stream and replay and by both ways through a call, rows far apart, values
at the ends of the range, one gradient alone, no tokens, gradients against
differences, and random sizes."""
import math
import random

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
import test_gpu_clip as tc
import test_gpu_embed as te
import test_gpu_gated as tg
from gpu_helpers import device, say
from oracle import clip as oc

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGN = -100


# --- the same bits ---------------------------------------------------------

def _embed(T, D, V, dtype, dev):
    w = torch.randn(V, D, device=dev).to(TDT[dtype])
    dy = torch.randn(T, D, device=dev).to(TDT[dtype])
    token = te.tokens(T, V, "text").to(dev)
    p = fc.EmbedPlan(T, D, V, dtype, scale=2.0, ignore_index=IGN)
    base = torch.randn(V, D, device=dev).to(TDT[dtype])

    def run(stream=None):
        added = base.clone()
        if stream is not None:        # the clone is work of the current stream
            torch.cuda.current_stream().synchronize()
        y, dw = p.forward(w, token, stream=stream), p.backward(token, dy, stream=stream)
        return y, dw, p.backward(token, dy, dw=added, accumulate=True, stream=stream)
    return run, (w, dy, base)


def _gated(T, D, F, dtype, dev):
    x, w, dy = tg.case(T, D, F, dtype, dev)
    p = fc.GatedPlan(T, D, F, dtype, "gelu")

    def run(stream=None):
        y, kept = p.forward(x, w, keep=True, stream=stream)
        dx, dw = p.backward(x, w, kept, dy, stream=stream)
        return y, dx, dw, p.forward(x, w, stream=stream)
    return run, (x, w, dy)


def _clip(n, dtype, dev):
    grads = [torch.randn(n + 7 * i, device=dev).to(TDT[dtype]) for i in range(140)]
    p = fc.ClipPlan([(g.numel(), dtype) for g in grads])

    def run(stream=None):
        out = [torch.empty_like(g) for g in grads]
        norm = p.clip(grads, 0.5, out=out, stream=stream)
        return norm, p.norm(grads, stream=stream), out[0], out[139]
    return run, tuple(grads)


CASES = {"embed tiny": lambda t, d: _embed(30, 40, 100, t, d), "embed": lambda t, d: _embed(900, 100, 333, t, d),
         "embed merged": lambda t, d: _embed(5000, 24, 100, t, d), "embed long": lambda t, d: _embed(40000, 16, 50, t, d),
         "gated few": lambda t, d: _gated(7, 64, 100, t, d), "gated small": lambda t, d: _gated(30, 300, 1500, t, d),
         "gated": lambda t, d: _gated(300, 96, 200, t, d), "gated tiles": lambda t, d: _gated(700, 512, 640, t, d),
         "gated packed": lambda t, d: _gated(2458, 203, 1344, t, d), "clip": lambda t, d: _clip(3000, t, d),
         "clip large": lambda t, d: _clip(100000, t, d)}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", CASES)
def test_same_bits_on_every_run_streams_and_graphs(name, dtype):
    dev = device()
    say("same bits:", name, dtype)
    run, inputs = CASES[name](dtype, dev)
    want = run()

    def same(got):
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    same(run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    same(run(side))                   # the full way through a call
    same(run(side.cuda_stream))
    with torch.cuda.stream(side):
        same(run())
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    with torch.cuda.graph(other):     # its own outputs and workspaces
        out2 = run()
    for _ in range(3):
        graph.replay()
        same(run())
        other.replay()
        same(out)
        same(out2)
    # Other inputs in the same places.
    for t in inputs:
        t.mul_(0.5)
    want = run()
    graph.replay()
    same(out)


def test_calls_at_once_on_two_streams():
    # One plan, two calls under way: each has its own outputs and workspace.
    dev = device()
    say("two streams")
    for name in ("embed merged", "gated tiles", "clip large"):
        run, _ = CASES[name]("bf16", dev)
        want = run()
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        got = []
        for _ in range(3):
            with torch.cuda.stream(a):
                got.append(run())
            with torch.cuda.stream(b):
                got.append(run())
        torch.cuda.synchronize()
        for g in got:
            for x, y in zip(g, want):
                assert torch.equal(x, y)


# --- rows far apart, past 32 bits -------------------------------------------

def _far(rows, cols, dtype, dev):
    """[rows, cols] with rows 2^21 elements apart."""
    ld = 1 << 21
    whole = torch.zeros((rows - 1) * ld + cols + 8, dtype=TDT[dtype], device=dev)
    return whole.as_strided((rows, cols), (ld, 1)), whole


def test_rows_past_32_bits():
    dev = device()
    say("rows past 2^31 elements")
    rows, D = 1100, 72  # 2.3e9 elements from the first row to the last
    far, whole = _far(rows, D, "bf16", dev)
    near = torch.randn(rows, D, device=dev).bfloat16()
    far.copy_(near)
    token = te.tokens(500, rows, "even").to(dev)
    token[0] = rows - 1
    p = fc.EmbedPlan(500, D, rows, scale=2.0, ignore_index=IGN)
    assert torch.equal(p.forward(far, token), p.forward(near, token))
    dy = torch.randn(500, D, device=dev).bfloat16()
    want = p.backward(token, dy)
    p.backward(token, dy, dw=far)
    assert torch.equal(far, want)
    p.backward(token, dy, dw=far, accumulate=True)
    assert torch.equal(far, p.backward(token, dy, dw=want, accumulate=True))
    for T in (8, 200, 2100):
        q = fc.GatedPlan(T, D, rows // 2)
        x, dy = torch.randn(T, D, device=dev).bfloat16(), torch.randn(T, rows // 2, device=dev).bfloat16()
        far.copy_(near / 8)
        w = far.contiguous()
        y, kept = q.forward(x, far, keep=True)
        y2, kept2 = q.forward(x, w, keep=True)
        assert torch.equal(y, y2)
        dx, dw = q.backward(x, far, kept, dy)
        dx2, dw2 = q.backward(x, w, kept2, dy)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        q.backward(x, w, kept, dy, dw=far)
        assert torch.equal(far, dw2)
    assert (whole[D:1 << 21] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_gradient_past_2_to_31_elements(dtype):
    # One tensor of 2^31 + 12345 elements, its last one found and scaled.
    dev = device()
    say("clip", dtype, "2^31 elements")
    n = (1 << 31) + 12345
    x = torch.zeros(n, dtype=TDT[dtype], device=dev)
    x[-1], x[0] = 4.0, 3.0
    p = fc.ClipPlan([(n, dtype)], eps=0.0)
    assert float(p.clip([x], 2.5)) == 5.0
    assert float(x[-1]) == 2.0 and float(x[0]) == 1.5 and float(p.norm([x])) == 2.5


# --- values ------------------------------------------------------------------

@pytest.mark.parametrize("T,D,F", [(5, 40, 60), (30, 64, 900), (200, 64, 90), (600, 256, 520)])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_and_special_gates(T, D, F, name, dtype):
    # A token of huge, one of NaN and one of zero values: the others' bits stay, no gate overflows to NaN.
    dev = device()
    say("gated special", T, D, F, name, dtype)
    x, w, dy = tg.case(T, D, F, dtype, dev)
    p = fc.GatedPlan(T, D, F, dtype, activation=name)
    y, kept = p.forward(x, w, keep=True)
    dx, _ = p.backward(x, w, kept, dy)
    x2 = x.clone()
    x2[0] = 1e4 * x[0]
    x2[1] = float("nan")
    x2[2] = 0.0
    y2, kept2 = p.forward(x2, w, keep=True)
    dx2, dw2 = p.backward(x2, w, kept2, dy)
    assert torch.equal(y2[3:], y[3:]) and torch.equal(dx2[3:], dx[3:])
    assert torch.isfinite(y2[0]).all() and torch.isfinite(dx2[0]).all()
    assert torch.isnan(y2[1]).all() and torch.isnan(dx2[1]).all()
    assert (y2[2] == 0).all() and torch.isnan(dw2).all()
    # Gates so large that their squares and cubes leave fp32.
    x3 = x.clone().float() * 1e16
    w3 = w.clone().float()
    w3[:F] *= 1e6
    w3[F:] *= 1e-16
    x3, w3 = x3.to(TDT[dtype]), w3.to(TDT[dtype])
    y3, kept3 = p.forward(x3, w3, keep=True)
    assert not torch.isnan(y3).any()
    g = x3.double().cpu() @ w3[:F].double().cpu().t()
    small = (g.abs() > 1e20).numpy()
    assert small.mean() > 0.9
    dx3, _ = p.backward(x3, w3, kept3, (1e-20 * dy.float()).to(TDT[dtype]))
    assert not torch.isnan(dx3).any()


def test_a_nan_weight_reaches_its_outputs_only():
    dev = device()
    say("gated NaN weight")
    for T in (9, 150, 520):
        x, w, dy = tg.case(T, 128, 200, "bf16", dev)
        p = fc.GatedPlan(T, 128, 200)
        y = p.forward(x, w)
        w[37], w[200 + 55] = float("nan"), float("inf")
        y2 = p.forward(x, w)
        keep = torch.ones(200, dtype=torch.bool, device=dev)
        keep[37] = keep[55] = False
        assert torch.equal(y2[:, keep], y[:, keep]) and torch.isnan(y2[:, 37]).all() and not torch.isfinite(y2[:, 55]).any()


# --- one gradient alone, no tokens -----------------------------------------------

@pytest.mark.parametrize("T,D,F", [(5, 40, 60), (30, 300, 1500), (200, 64, 90), (600, 512, 640), (2458, 203, 1344)])
def test_one_gradient_alone(T, D, F):
    dev = device()
    say("one gradient", T, D, F)
    x, w, dy = tg.case(T, D, F, "bf16", dev)
    p = fc.GatedPlan(T, D, F)
    _, kept = p.forward(x, w, keep=True)
    dx, dw = p.backward(x, w, kept, dy)
    a, none = p.backward(x, w, kept, dy, need_dw=False)
    none2, b = p.backward(x, w, kept, dy, need_dx=False)
    assert none is None and none2 is None and torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_tokens(dtype):
    dev = device()
    say("no tokens", dtype)
    e = torch.empty(0, 24, dtype=TDT[dtype], device=dev)
    token = torch.empty(0, dtype=torch.int64, device=dev)
    p = fc.EmbedPlan(0, 24, 50, dtype)
    w = torch.randn(50, 24, device=dev).to(TDT[dtype])
    assert p.forward(w, token).shape == (0, 24)
    assert (p.backward(token, e) == 0).all()
    assert torch.equal(p.backward(token, e, dw=w.clone(), accumulate=True), w)
    q = fc.GatedPlan(0, 24, 25, dtype)
    y, kept = q.forward(e, w, keep=True)
    assert y.shape == (0, 25)
    dx, dw = q.backward(e, w, kept, y)
    assert dx.shape == (0, 24) and (dw == 0).all() and dw.shape == (50, 24)


def test_all_tokens_ignored():
    dev = device()
    say("all ignored")
    for T in (5, 600, 5000):
        p = fc.EmbedPlan(T, 40, 70)
        token = torch.full((T,), IGN, device=dev)
        dy = torch.full((T, 40), float("nan"), dtype=torch.bfloat16, device=dev)
        w = torch.full((70, 40), float("nan"), dtype=torch.bfloat16, device=dev)
        assert (p.forward(w, token) == 0).all() and (p.backward(token, dy) == 0).all()


# --- against differences --------------------------------------------------------

@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradient_against_differences(name):
    # Along a random direction of x and of w, in fp32.  A difference of 2^-6 is off by its square times a third
    # derivative of about one: 1e-3 of the sum of the directions' sizes; the sums' own errors are below that.
    dev = device()
    say("differences", name)
    T, D, F, e = 40, 64, 90, 2.0 ** -6
    x, w, dy = tg.case(T, D, F, "fp32", dev)
    p = fc.GatedPlan(T, D, F, "fp32", activation=name)
    _, kept = p.forward(x, w, keep=True)
    dx, dw = p.backward(x, w, kept, dy)
    ux, uw = torch.randn_like(x), torch.randn_like(w) / 8
    for a, b, slope in ((ux, torch.zeros_like(w), (dx * ux).double().sum()), (torch.zeros_like(x), uw, (dw * uw).double().sum())):
        up, down = p.forward(x + e * a, w + e * b), p.forward(x - e * a, w - e * b)
        got = ((up.double() - down.double()) * dy.double()).sum() / (2 * e)
        size = float((dy.double().abs() * (up.double() - down.double()).abs()).sum() / (2 * e))
        assert abs(float(got - slope)) <= 1e-3 * size


# --- both ways, what is refused on the GPU ------------------------------------------

def test_bindings_on_the_gpu():
    dev = device()
    say("bindings")
    p = fc.EmbedPlan(4, 8, 20)
    w, token = torch.randn(20, 8, device=dev).bfloat16(), torch.arange(4, device=dev)
    with pytest.raises(ValueError, match="token: dtype"):
        p.forward(w, token.int())
    with pytest.raises(ValueError, match="different devices|GPU"):
        p.forward(w, token.cpu())
    # A [2, 2, 8] activation is one of four tokens.
    assert torch.equal(p.backward(token.view(2, 2), torch.ones(2, 2, 8, device=dev).bfloat16()),
                       p.backward(token, torch.ones(4, 8, device=dev).bfloat16()))
    with pytest.raises(fc.FconvError):
        p.forward(w, token, y=w[:4])  # overlaps
    q = fc.GatedPlan(4, 8, 10)
    x = torch.randn(4, 8, device=dev).bfloat16()
    y, kept = q.forward(x, w, keep=True)
    for bad in (kept[1:], kept[:-1], kept.bfloat16()):
        with pytest.raises((ValueError, fc.FconvError)):
            q.backward(x, w, bad, y)
    c = fc.ClipPlan([(160, "bf16"), (160, "bf16")])
    with pytest.raises(fc.FconvError):
        c.clip([w, w], 1.0)
    with pytest.raises(ValueError, match="shape"):
        c.clip([w, w.clone()], 1.0, out=[w.clone(), torch.empty(8, 20, device=dev).bfloat16()])
    with pytest.raises(fc.FconvError):
        c.clip([w, w.clone()], 1.0, out=[w, w])
    assert float(c.norm([w, w])) > 0  # read only: twice the same is as good as two


# --- random sizes -----------------------------------------------------------------

def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


@pytest.mark.parametrize("seed", range(60))
def test_random_layers(seed):
    dev = device()
    rng = random.Random(seed)
    while True:
        T, D, F = _size(rng, 1, 3000), _size(rng, 1, 2000), _size(rng, 1, 2000)
        if T * D * F <= 1 << 28:
            break
    dtype, name = rng.choice(("bf16", "bf16", "fp32")), rng.choice(tg.ACTS)
    x, w, dy = tg.case(T, D, F, dtype, dev, seed=seed)
    out = {}
    # Rows apart, at any element.
    for what in ("x", "w", "dy", "y", "dx", "dw"):
        if rng.random() < 0.3:
            rows, cols = {"x": (T, D), "w": (2 * F, D), "dy": (T, F), "y": (T, F), "dx": (T, D), "dw": (2 * F, D)}[what]
            off, more = rng.randrange(9), rng.randrange(9)
            b = torch.full((rows, cols + off + more), float("nan"), dtype=TDT[dtype], device=dev)[:, off:off + cols]
            if what in ("x", "w", "dy"):
                b.copy_({"x": x, "w": w, "dy": dy}[what])
                x, w, dy = (b if what == n else t for n, t in (("x", x), ("w", w), ("dy", dy)))
            else:
                out[what] = b
    say("gated", seed, T, D, F, dtype, name, sorted(out), x.stride(0), w.stride(0), dy.stride(0))
    tg.check(x, w, dy, dtype, name, **out)


@pytest.mark.parametrize("seed", range(40))
def test_random_lookups(seed):
    dev = device()
    rng = random.Random(1000 + seed)
    while True:
        T, D, V = _size(rng, 1, 70000), _size(rng, 1, 3000), _size(rng, 1, 20000)
        if (T + V) * D <= 1 << 23:
            break
    dtype, kind, scale = rng.choice(("bf16", "fp32")), rng.choice(("even", "text", "one")), rng.choice((1.0, -0.3, 64.0))
    say("embed", seed, T, D, V, dtype, kind, scale)
    token = te.tokens(T, V, kind, seed).to(dev)
    off, more = rng.randrange(9), rng.randrange(9)
    dy = torch.randn(T, D + off + more, device=dev).to(TDT[dtype])[:, off:off + D]
    base = torch.randn(V, D + off + more, device=dev).to(TDT[dtype])
    plan = fc.EmbedPlan(T, D, V, dtype, scale=scale, ignore_index=IGN)
    dw = te.check_backward(plan, token, dy, V, dtype, scale)
    at = base[:, more:more + D]
    te.check_backward(plan, token, dy, V, dtype, scale, dw=at)
    assert torch.equal(at, dw)
    at.normal_()
    te.check_backward(plan, token, dy, V, dtype, scale, before=te._np(at).copy(), dw=at, accumulate=True)
    y = plan.forward(base[:, more:more + D], token)
    row = torch.where(token == IGN, 0, token)
    want = torch.where((token == IGN)[:, None], 0.0, base[:, more:more + D].double()[row] * float(np.float32(scale)))
    half = 0 if scale == 1.0 else te._half(dtype) + te.U
    assert ((y.double() - want).abs() <= half * want.abs()).all()


@pytest.mark.parametrize("seed", range(25))
def test_random_gradients(seed):
    dev = device()
    rng = random.Random(2000 + seed)
    sizes = [rng.choice((0, 1, _size(rng, 1, 200000))) for _ in range(rng.choice((1, 3, 40, 128, 129, 260)))]
    say("clip", seed, len(sizes), max(sizes))
    grads, dts = tc.make(sizes, dev, seed=seed)
    # Some of them between aligned places.
    for i, g in enumerate(grads):
        if g.numel() and rng.random() < 0.3:
            off = rng.randrange(1, 9)
            grads[i] = torch.empty(g.numel() + 9, dtype=g.dtype, device=dev)[off:off + g.numel()].copy_(g)
    n = oc.norm([tc._np(g) for g in grads])
    tc.check(fc.ClipPlan([(g.numel(), d) for g, d in zip(grads, dts)]), grads, dts, n * rng.choice((0.0, 0.3, 3.0)), rng.random() < 0.5)
