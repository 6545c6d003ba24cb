"""A small language model with one table at both ends, trained and then served.

    python examples/language_model.py [--tokens T] [--features D] [--vocabulary V] [--steps N]

    x = sqrt(D) table[token]     EmbedPlan
    h = act(x wg^T) (x wu^T)     GatedPlan, as wide as the table
    loss of h table^T            XentPlan

Training: the output layer's gradient of the table and the lookup's go into one
tensor, all gradients are clipped by their norm together (ClipPlan), and the fp32
weights take a step.  Serving: one token at a time, the table once more in 4 bits
(MxPlan).  Tokens are synthetic: each is a fixed function of the one before it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_implicit_gemm_nhwc_amd as fc  # noqa: E402

IGNORE = -100


class Model:
    """The plans of a step of T tokens."""

    def __init__(self, T, D, V, dtype="bf16", activation="silu"):
        self.embed = fc.EmbedPlan(T, D, V, dtype, scale=D ** 0.5, ignore_index=IGNORE)
        self.gated = fc.GatedPlan(T, D, D, dtype, activation=activation)
        self.xent = fc.XentPlan(T, D, V, dtype, ignore_index=IGNORE)
        self.clip = fc.ClipPlan([(V * D, dtype), (2 * D * D, dtype)])

    def gradients(self, table, w, token, target, dloss):
        """(loss [T], gradient of the table, of the gated layer's weights)."""
        x = self.embed.forward(table, token)
        h, kept = self.gated.forward(x, w, keep=True)
        loss, lse = self.xent.forward(h, table, target)
        dh, dtable = self.xent.backward(h, table, target, lse, dloss)
        dx, dw = self.gated.backward(x, w, kept, dh)
        self.embed.backward(token, dx, dw=dtable, accumulate=True)
        return loss, dtable, dw


def batch(tokens, vocabulary, g, device):
    token = torch.randint(0, vocabulary, (tokens,), generator=g, device=device)
    target = (7 * token + 3) % vocabulary
    # Padding: neither looked up nor answered.
    pad = torch.rand(tokens, generator=g, device=device) < 0.1
    return torch.where(pad, IGNORE, token), torch.where(pad, IGNORE, target)


def train(tokens, features, vocabulary, steps, rate, max_norm, g, device="cuda"):
    """Weights (fp32), and of each step its mean loss and its gradients' norm."""
    model = Model(tokens, features, vocabulary)
    table = torch.randn(vocabulary, features, generator=g, device=device) / features ** 0.5
    w = torch.randn(2 * features, features, generator=g, device=device) / features ** 0.5
    log = []
    for _ in range(steps):
        token, target = batch(tokens, vocabulary, g, device)
        live = target != IGNORE
        dloss = live.float() / live.sum().clamp_min(1)
        loss, dtable, dw = model.gradients(table.bfloat16(), w.bfloat16(), token, target, dloss)
        norm = model.clip.clip([dtable, dw], max_norm)
        table -= rate * dtable.float()
        w -= rate * dw.float()
        log.append(((loss * dloss).sum(), norm))
    return table, w, [(a.item(), b.item()) for a, b in log]


class Server:
    """Logits of one token after another."""

    def __init__(self, table, w):
        V, D = table.shape
        self.table, self.w = table.bfloat16(), w.bfloat16()
        self.embed = fc.EmbedPlan(1, D, V, scale=D ** 0.5)
        self.gated = fc.GatedPlan(1, D, D)
        self.out, self.table4 = fc.MxPlan(1, V, D, ops=()), fc.MxQuantPlan(V, D, "fp32")(table)

    def __call__(self, token):
        return self.out(self.gated.forward(self.embed.forward(self.table, token), self.w), self.table4)


def main(tokens=2048, features=256, vocabulary=500, steps=20, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    table, w, log = train(tokens, features, vocabulary, steps, 1.0, 0.5, g)
    server, token, said = Server(table, w), torch.zeros(1, dtype=torch.int64, device="cuda"), []
    for _ in range(8):
        token = server(token).argmax(1)
        said.append(token)
    return {"loss": [a for a, _ in log], "norm": [b for _, b in log], "said": torch.cat(said).tolist()}


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("features", 256), ("vocabulary", 500), ("steps", 20), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=value)
    r = main(**vars(p.parse_args()))
    for i, (loss, norm) in enumerate(zip(r["loss"], r["norm"])):
        print("step %d: mean loss %.4f, norm of the gradients %.4f" % (i, loss, norm))
    print("tokens after 0:", *r["said"])
