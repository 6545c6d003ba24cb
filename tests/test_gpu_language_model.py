"""The lookup, the gated layer, the output layer and clipping as one step
(examples/language_model.py): its gradients against autograd in 64 bits, and
that it runs.

In fp32 every sum of n terms is off by about u n / 2.5 of their root mean square
at most (u = 2^-24), an activation and an exponential by some tens of u, and a
gradient passes three products one after another: 1e-5 of the gradient's norm is
a hundred times u with n of 64 .. 512.  In bf16 x, h, dh and dx are rounded between
the layers, dz and q within them, and every weight's gradient at the end: each by
2^-9 of itself on average, some eight of them one after another, amplified by
slopes of about one: 2^-9 * 8 = 0.016 of the norm."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import device, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def _act(name, g):
    f = torch.nn.functional
    return {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda x: f.gelu(x, approximate="tanh"), "relu": torch.relu}[name](g)


@pytest.mark.parametrize("dtype,most", [("fp32", 1e-5), ("bf16", 0.016)])
@pytest.mark.parametrize("T,D,V,act", [(1, 64, 90, "silu"), (40, 64, 200, "gelu"), (300, 72, 111, "gelu_tanh"), (1500, 128, 700, "silu"),
                                       (700, 65, 300, "gelu")])
def test_a_step(T, D, V, act, dtype, most):
    dev = device()
    say("language model", T, D, V, act, dtype)
    ex = _example()
    g = torch.Generator().manual_seed(T + D)
    table = (torch.randn(V, D, generator=g) / D ** 0.5).to(TDT[dtype])
    w = (torch.randn(2 * D, D, generator=g) / D ** 0.5).to(TDT[dtype])
    token, target = ex.batch(T, V, g, "cpu")
    token[0], target[0] = 1, 2
    live = target != ex.IGNORE
    dloss = live.float() / live.sum()

    a, b = table.double().requires_grad_(), w.double().requires_grad_()
    x = torch.where(live[:, None], a[torch.where(live, token, 0)], 0.0) * float(torch.tensor(D ** 0.5).float())
    h = _act(act, x @ b[:D].t()) * (x @ b[D:].t())
    want = torch.nn.functional.cross_entropy(h @ a.t(), target, ignore_index=ex.IGNORE, reduction="none")
    (want * dloss.double()).sum().backward()

    model = ex.Model(T, D, V, dtype, act)
    loss, dtable, dw = model.gradients(table.to(dev), w.to(dev), token.to(dev), target.to(dev), dloss.to(dev))
    off = (loss.cpu().double() - want.detach()).norm() / want.detach().norm()
    assert off <= most, float(off)
    for got, ref in ((dtable, a.grad), (dw, b.grad)):
        off = (got.cpu().double() - ref).norm() / ref.norm()
        assert off <= most, float(off)
    # Clipped to half of their norm.
    total = float(torch.stack([dtable.double().norm(), dw.double().norm()]).norm())
    keep = [dtable.clone(), dw.clone()]
    norm = model.clip.clip([dtable, dw], 0.5 * total)
    assert abs(float(norm) - total) <= 1e-6 * total
    for got, before in zip((dtable, dw), keep):
        assert (got.double() - 0.5 * before.double()).norm() <= (2.0 ** -8 if dtype == "bf16" else 1e-6) * before.double().norm()


def test_a_step_in_a_graph():
    # Captured with everything it allocates; replays between eager steps give the eager step's bits.
    dev = device()
    say("language model, captured")
    ex = _example()
    T, D, V = 700, 64, 300
    model = ex.Model(T, D, V)
    g = torch.Generator(device=dev).manual_seed(0)
    table = (torch.randn(V, D, generator=g, device=dev) / 8).bfloat16()
    w = (torch.randn(2 * D, D, generator=g, device=dev) / 8).bfloat16()
    token, target = ex.batch(T, V, g, dev)
    dloss = torch.full((T,), 1 / T, device=dev)

    def step():
        loss, dtable, dw = model.gradients(table, w, token, target, dloss)
        return loss, dtable, dw, model.clip.clip([dtable, dw], 0.01)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        g.manual_seed(seed)
        new = ex.batch(T, V, g, dev)
        token.copy_(new[0])
        target.copy_(new[1])
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,features,vocabulary", [(100, 64, 50), (600, 130, 333)])
def test_example_runs(tokens, features, vocabulary):
    device()
    say("language model example", tokens, features, vocabulary)
    r = _example().main(tokens, features, vocabulary, steps=3)
    assert len(r["loss"]) == 3 and all(x > 0 for x in r["norm"])
    assert all(0 <= t < vocabulary for t in r["said"]) and len(r["said"]) == 8
