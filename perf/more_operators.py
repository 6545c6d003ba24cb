"""Measured cases of the operators around the output layer: the embedding
lookup with its gradient, the gated feed-forward layer with its gradients, and
the norm and clipping of all gradients together.

``run`` computes a case either in plain torch operations (``own`` False) or
with the framework's entry points (``own`` True).

  lookup  y[t] = scale w[token[t]];  dw[v] = scale * sum of dy[t] over token[t] = v
  gated   g = x wg^T, u = x wu^T, y = act(g) u (wg: the first F rows of w, wu: the others)
          dg = dy u act'(g), du = dy act(g);  dx = dg wg + du wu;  dw = [dg du]^T x
  clip    norm = sqrt(sum of all gradients' squares);  gradients * min(1, max_norm / (norm + eps))
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGNORE = -100
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # Serving one token: the row of a large table, scaled by sqrt(D). Launch latency.
        {"name": "lookup_one_token", "op": "lookup", "T": 1, "D": 4096, "V": 32768, "dtype": "bf16", "scale": 64.0},
        # The tokens of a long batch of prompts, a large odd vocabulary: streaming.
        {"name": "lookup_prompts", "op": "lookup", "T": 32768, "D": 2048, "V": 50021, "dtype": "bf16", "scale": 1.0},
        # Training with odd sizes in fp32: a ragged batch over a middling vocabulary.
        {"name": "lookup_grad_ragged", "op": "lookup_grad", "T": 1999, "D": 1000, "V": 32001, "dtype": "fp32",
         "scale": 32.0},
        # Training a large table: most of the gradient's rows are zeros, a few tokens make up much of the batch.
        {"name": "lookup_grad_large", "op": "lookup_grad", "T": 16384, "D": 4096, "V": 65536, "dtype": "bf16",
         "scale": 64.0},
        # Serving one token: bound by reading both projections' weights.
        {"name": "gated_one_token", "op": "gated", "T": 1, "D": 4096, "F": 12288, "dtype": "bf16", "act": "silu"},
        # A prompt's feed-forward layer: bound by the matrix cores.
        {"name": "gated_prompt", "op": "gated", "T": 8192, "D": 4096, "F": 12288, "dtype": "bf16", "act": "silu"},
        # Training a small layer in fp32 (32 images, 512 features): latency.
        {"name": "gated_grad_small", "op": "gated_grad", "T": 32, "D": 512, "F": 1000, "dtype": "fp32", "act": "gelu"},
        # Training with odd sizes: a ragged batch of tokens, rows that are no multiple of 16 bytes.
        {"name": "gated_grad_ragged", "op": "gated_grad", "T": 1999, "D": 1000, "F": 2731, "dtype": "bf16",
         "act": "gelu_tanh"},
        # Training a large layer: bound by the matrix cores.
        {"name": "gated_grad_large", "op": "gated_grad", "T": 8192, "D": 4096, "F": 8192, "dtype": "bf16",
         "act": "silu"},
        # The gradients of a small convolutional classifier, clipped: launch latency.
        {"name": "clip_classifier", "op": "clip", "net": "conv", "depth": 4, "width": 64, "rows": 1000,
         "dtype": "fp32", "share": 0.5},
        # The gradients of a language model of 0.5 billion weights, clipped: streaming.
        {"name": "clip_model", "op": "clip", "net": "gated", "depth": 8, "width": 2048, "rows": 50021,
         "dtype": "bf16", "share": 0.25},
        # Gradients below the limit, as most steps have them: the norm alone is work, the gradients stay.
        {"name": "clip_not_needed", "op": "clip", "net": "gated", "depth": 12, "width": 1024, "rows": 32768,
         "dtype": "fp32", "share": 2.0},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even in its logarithm; rounded to a multiple
    of 64 half the time, left odd or even as it falls otherwise."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 128 and rng.random() < 0.5:
        n = (n + 32) // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(("lookup", "lookup_grad", "gated", "gated_grad", "clip"))
    while True:
        if op in ("lookup", "lookup_grad"):
            c = {"op": op, "T": _log(rng, 1, 65536), "D": _log(rng, 64, 8192), "V": _log(rng, 500, 131072),
                 "dtype": rng.choice(("bf16", "bf16", "fp32")), "scale": rng.choice((1.0, 0.5, 22.5, 64.0))}
            if (c["T"] + c["V"]) * c["D"] * (2 if c["dtype"] == "bf16" else 4) <= 1 << 29:
                return c
        elif op in ("gated", "gated_grad"):
            c = {"op": op, "T": _log(rng, 1, 8192), "D": _log(rng, 64, 4096), "F": _log(rng, 64, 16384),
                 "dtype": rng.choice(("bf16", "bf16", "bf16", "fp32")),
                 "act": rng.choice(("silu", "gelu", "gelu_tanh", "relu"))}
            if c["T"] * c["D"] * c["F"] <= (1 << 37 if c["dtype"] == "bf16" else 1 << 33):
                return c
        else:
            c = {"op": op, "net": rng.choice(("conv", "gated", "ragged")), "depth": _log(rng, 1, 64),
                 "width": _log(rng, 16, 2048), "rows": _log(rng, 10, 50000), "dtype": rng.choice(("bf16", "fp32", "mixed")),
                 "share": rng.choice((0.01, 0.5, 0.9, 2.0))}
            if sum(math.prod(s) for s, _ in _gradients(c)) <= 1 << 28:
                return c


def _gradients(case):
    """Shapes and types of a clipped network's gradients."""
    n, c, rows = case["depth"], case["width"], case["rows"]
    if case["net"] == "conv":
        # 3x3 and 1x1 filters in HWIO order, scale and shift of each, the classifier.
        shapes = []
        for _ in range(n):
            shapes += [(3, 3, c, c), (c,), (c,), (1, 1, c, 4 * c), (4 * c,), (4 * c,)]
        shapes += [(rows, 4 * c), (rows,)]
    elif case["net"] == "gated":
        # An embedding, and blocks of a gated layer, the projection after it and two norms.
        shapes = [(rows, c)]
        for _ in range(n):
            shapes += [(8 * c, c), (c, 4 * c), (c,), (c,)]
    else:
        # Tensors of any size, single numbers among them.
        rng = random.Random(n * 1000003 + c * 1009 + rows)
        shapes = [(_log(rng, 1, 64 * c),) for _ in range(4 * n)]
    kinds = {"bf16": ("bf16",), "fp32": ("fp32",), "mixed": ("bf16", "bf16", "fp32")}[case["dtype"]]
    return [(s, kinds[i % len(kinds)]) for i, s in enumerate(shapes)]


def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "lookup":
        # At most T different rows of the table are read.
        return {"bytes": case["D"] * e * (case["T"] + min(case["T"], case["V"])) + 8 * case["T"], "flops": 0}
    if case["op"] == "lookup_grad":
        return {"bytes": case["D"] * e * (case["T"] + case["V"]) + 8 * case["T"], "flops": 0}
    if case["op"] == "clip":
        n = sum(math.prod(s) * (2 if k == "bf16" else 4) for s, k in _gradients(case))
        return {"bytes": n if case["share"] > 1 else 2 * n, "flops": 0}
    T, D, F = case["T"], case["D"], case["F"]
    once = e * (T * D + 2 * F * D + T * F)
    if case["op"] == "gated":
        return {"bytes": once, "flops": 4 * T * D * F}
    # x, w and dy read, y, dx and dw written.
    return {"bytes": 2 * once, "flops": 12 * T * D * F}


# ---------------------------------------------------------------- plain forms

def _act(g, act):
    """act(g) and act'(g)."""
    if act == "silu":
        s = 1 / (1 + (-g).exp())
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * (-0.5 * g * g).exp() * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c, k = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(c * (g + k * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * k * g * g)
    return g.clamp_min(0), (g > 0).to(g.dtype)


def _plain_lookup(s):
    live = s["token"] != IGNORE
    rows = s["w"][torch.where(live, s["token"], torch.zeros_like(s["token"]))].float() * s["scale"]
    return torch.where(live.unsqueeze(1), rows, torch.zeros_like(rows)).to(s["w"].dtype)


def _plain_lookup_grad(s):
    V, D = s["V"], s["dy"].shape[1]
    # Ignored tokens go to a row behind the last one.
    at = torch.where(s["token"] != IGNORE, s["token"], torch.full_like(s["token"], V))
    dw = torch.zeros(V + 1, D, dtype=torch.float32, device=DEV)
    dw.index_add_(0, at, s["dy"].float())
    return (dw[:V] * s["scale"]).to(s["dy"].dtype)


def _plain_gated(s):
    x, w = s["x"].float(), s["w"].float()
    F = w.shape[0] // 2
    g, u = x @ w[:F].t(), x @ w[F:].t()
    a, da = _act(g, s["act"])
    y = (a * u).to(s["x"].dtype)
    if s["op"] == "gated":
        return y
    dy = s["dy"].float()
    dz = torch.cat((dy * u * da, dy * a), 1)
    return {"y": y, "dx": (dz @ w).to(s["x"].dtype), "dw": (dz.t() @ x).to(s["w"].dtype)}


def _plain_clip(s):
    # Squares in 64 bits: in 32 those of large and of tiny gradients leave the range.
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in s["grads"]:
        total = total + g.double().square().sum()
    norm = total.sqrt().float()
    by = (s["max_norm"] / (norm + EPS)).clamp_max(1.0)
    return [norm] + [(g.float() * by).to(g.dtype) for g in s["grads"]]


# ---------------------------------------------------------------- state

def _tokens(T, V, g):
    """Tokens as text has them: the rank of a token is about even in its
    logarithm, and ranks are spread over the table.  A tenth is padding."""
    rank = torch.exp(torch.rand(T, generator=g, device=DEV, dtype=torch.float64) * math.log(V)).long() - 1
    token = torch.randperm(V, generator=g, device=DEV)[rank.clamp(0, V - 1)]
    pad = torch.rand(T, generator=g, device=DEV) < 0.1
    pad[0] = False
    return torch.where(pad, torch.full_like(token, IGNORE), token)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * by).to(DTYPES[case["dtype"]])
    if case["op"] == "lookup":
        return {"token": _tokens(case["T"], case["V"], g), "w": normal(case["V"], case["D"]), "scale": case["scale"]}
    if case["op"] == "lookup_grad":
        return {"token": _tokens(case["T"], case["V"], g), "dy": normal(case["T"], case["D"], by=1 / case["T"]),
                "V": case["V"], "scale": case["scale"]}
    if case["op"] in ("gated", "gated_grad"):
        T, D, F = case["T"], case["D"], case["F"]
        s = {"x": normal(T, D), "w": normal(2 * F, D, by=1 / math.sqrt(D)), "act": case["act"]}
        if case["op"] == "gated_grad":
            s["dy"] = normal(T, F, by=1 / T)
        return s
    grads = []
    for shape, kind in _gradients(case):
        # Layers' gradients differ in size.
        size = 10 ** (-3 * torch.rand((), generator=g, device=DEV))
        grads.append((torch.randn(*shape, generator=g, device=DEV) * size).to(DTYPES[kind]))
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    # A limit of `share` of the norm, as a program has it: a number chosen beforehand.
    return {"grads": grads, "max_norm": float(torch.tensor(norm * case["share"], dtype=torch.float32))}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if own:
        import convolution_implicit_gemm_nhwc_amd as fc
        if case["op"] in ("lookup", "lookup_grad"):
            s["plan"] = fc.EmbedPlan(case["T"], case["D"], case["V"], case["dtype"], scale=case["scale"],
                                     ignore_index=IGNORE)
        elif case["op"] in ("gated", "gated_grad"):
            s["plan"] = fc.GatedPlan(case["T"], case["D"], case["F"], case["dtype"], activation=case["act"])
        else:
            s["plan"] = fc.ClipPlan([(t.numel(), k) for t, (_, k) in zip(s["grads"], _gradients(case))], eps=EPS)
            # Clipped gradients beside the given ones, so that a pass can be made again; where none is clipped in place.
            s["out"] = [torch.empty_like(t) for t in s["grads"]] if case["share"] <= 1 else None
    return s


def run(state):
    s = state
    if not own:
        return {"lookup": _plain_lookup, "lookup_grad": _plain_lookup_grad, "gated": _plain_gated,
                "gated_grad": _plain_gated, "clip": _plain_clip}[s["op"]](s)
    plan = s["plan"]
    if s["op"] == "lookup":
        return plan.forward(s["w"], s["token"])
    if s["op"] == "lookup_grad":
        return plan.backward(s["token"], s["dy"])
    if s["op"] == "gated":
        return plan.forward(s["x"], s["w"])
    if s["op"] == "gated_grad":
        y, kept = plan.forward(s["x"], s["w"], keep=True)
        dx, dw = plan.backward(s["x"], s["w"], kept, s["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    norm = plan.clip(s["grads"], s["max_norm"], out=s["out"])
    return [norm] + (s["grads"] if s["out"] is None else s["out"])


# ---------------------------------------------------------------- 64 bits

def _exact_act(g, act):
    """act(g) and act'(g) by the definitions' own terms."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # 0.5 (1 + tanh v) = sigmoid(2 v)
        v2 = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(v2)
        return g * s, s + g * s * torch.sigmoid(-v2) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g.square())
    return torch.relu(g), torch.heaviside(g, torch.zeros((), dtype=g.dtype, device=g.device))


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "lookup":
        y = torch.zeros(case["T"], case["D"], dtype=torch.float64, device=DEV)
        row = torch.nonzero(s["token"] != IGNORE).squeeze(1)
        y[row] = case["scale"] * s["w"].index_select(0, s["token"][row]).double()
        return y
    if case["op"] == "lookup_grad":
        dw = torch.zeros(case["V"], case["D"], dtype=torch.float64, device=DEV)
        row = torch.nonzero(s["token"] != IGNORE).squeeze(1)
        dw.index_put_((s["token"][row],), s["dy"][row].double(), accumulate=True)
        return dw.mul_(case["scale"])
    if case["op"] in ("gated", "gated_grad"):
        x, w = s["x"].double(), s["w"].double()
        z = torch.mm(x, w.t())
        g, u = z.chunk(2, 1)
        a, da = _exact_act(g, case["act"])
        y = a * u
        if case["op"] == "gated":
            return y
        dy = s["dy"].double()
        du, dg = a.mul_(dy), da.mul_(u).mul_(dy)
        F = case["F"]
        dx = torch.mm(dg, w[:F]).addmm_(du, w[F:])
        dw = torch.cat((torch.mm(dg.t(), x), torch.mm(du.t(), x)))
        return {"y": y, "dx": dx, "dw": dw}
    flat = [t.double() for t in s["grads"]]
    norm = torch.sqrt(torch.stack([torch.linalg.vector_norm(t) for t in flat]).square().sum())
    by = min(1.0, s["max_norm"] / (norm.item() + EPS))
    return [norm] + [t.mul_(by) for t in flat]
