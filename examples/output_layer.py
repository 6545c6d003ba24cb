"""A classifier's output layer, trained and then served in 4 bits.

    python examples/output_layer.py [--tokens T] [--features D] [--classes V] [--steps N]

Training: XentPlan gives the loss of a batch and both gradients without its
logits; dh is what the layers below would receive.  The weights are kept in
fp32 and rounded to bf16 for each step.  Serving: the weights are laid out once
in MXFP4, and MxPlan takes bf16 features to logits.  Features are synthetic: a
centre for each class and noise around it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_implicit_gemm_nhwc_amd as fc  # noqa: E402

IGNORE = -100


def batch(centres, tokens, noise, g):
    target = torch.randint(0, centres.shape[0], (tokens,), generator=g, device=centres.device)
    h = centres[target] + noise * torch.randn(tokens, centres.shape[1], generator=g, device=centres.device)
    return h.bfloat16(), target


def train(centres, tokens, steps, rate, noise, g):
    """Weights (fp32 [V, D]) and the mean loss before each step."""
    V, D = centres.shape
    xent = fc.XentPlan(tokens, D, V, "bf16", ignore_index=IGNORE)
    w, losses = torch.zeros(V, D, device=centres.device), []
    for _ in range(steps):
        h, target = batch(centres, tokens, noise, g)
        # Some tokens carry no loss, as padding does.
        target[torch.rand(tokens, generator=g, device=target.device) < 0.1] = IGNORE
        live = target != IGNORE
        mean = live.float() / live.sum().clamp_min(1)
        wb = w.bfloat16()
        loss, lse = xent.forward(h, wb, target)
        dh, dw = xent.backward(h, wb, target, lse, mean)
        losses.append((loss * mean).sum())
        w -= rate * dw.float()
    return w, torch.stack(losses).tolist()


def serve(w, h):
    """Logits of h by the 4-bit weights."""
    V, D = w.shape
    w4 = fc.MxQuantPlan(V, D, "fp32")(w)  # once, when the weights are loaded
    plan = fc.MxPlan(h.shape[0], V, D, "bf16", ops=())
    return plan(h, w4)


def main(tokens=2048, features=512, classes=1000, steps=8, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    centres = torch.randn(classes, features, generator=g, device="cuda")
    # A step moves a class's logit of its own centre by about rate * features / classes.
    w, losses = train(centres, tokens, steps, 20.0 * classes / features, 0.5, g)
    h, target = batch(centres, tokens, 0.5, g)
    full = (h.float() @ w.t()).argmax(1)
    four = serve(w, h).argmax(1)
    return {"loss": losses, "accuracy": (full == target).float().mean().item(),
            "accuracy_4bit": (four == target).float().mean().item()}


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("features", 512), ("classes", 1000), ("steps", 8), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=value)
    r = main(**vars(p.parse_args()))
    for i, loss in enumerate(r["loss"]):
        print("step %d: mean loss %.4f" % (i, loss))
    print("accuracy on a new batch: fp32 weights %.4f, MXFP4 weights and features %.4f"
          % (r["accuracy"], r["accuracy_4bit"]))
