"""Measured cases of the output-layer operators: MXFP4 quantisation, the MXFP4
product, and the linear softmax cross entropy with its gradient.

``run`` computes a case either in plain torch operations (``own`` False) or
with the framework's entry points (``own`` True).  MXFP4 is the 4-bit e2m1
format with one power-of-two scale (e8m0) per block of 32 values of a row.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGNORE = -100
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A small ragged activation (17 tokens of 1000 features) to 4 bits and back: launch latency.
        {"name": "quantise_ragged_fp32", "op": "quantise", "rows": 17, "cols": 1000, "dtype": "fp32"},
        # A long batch of activations to 4 bits and back: streaming.
        {"name": "quantise_large", "op": "quantise", "rows": 16384, "cols": 4096, "dtype": "bf16"},
        # Serving one token: a vocabulary-sized output layer, bound by reading the 4-bit weights.
        {"name": "product_one_token", "op": "product", "M": 1, "N": 32768, "K": 4096, "dtype": "bf16", "relu": False},
        # 32 images' last 7x7x512 feature map feeding 1024 outputs: few rows, a long reduction.
        {"name": "product_7x7x512", "op": "product", "M": 32, "N": 1024, "K": 25088, "dtype": "bf16", "relu": True},
        # A 1x1 convolution over 32 images of 56x56x256 -> 64: many rows, little work for each.
        {"name": "product_1x1", "op": "product", "M": 100352, "N": 64, "K": 256, "dtype": "bf16", "relu": True},
        # A dense layer on a long batch: bound by the matrix cores.
        {"name": "product_large", "op": "product", "M": 8192, "N": 8192, "K": 4096, "dtype": "bf16", "relu": False},
        # Classifier loss of a small batch (32 images, 512 features, 1000 classes): latency.
        {"name": "loss_classifier", "op": "loss", "T": 32, "D": 512, "V": 1000},
        # Evaluating a language model's loss: large odd vocabulary, forward only.
        {"name": "loss_vocabulary", "op": "loss", "T": 4096, "D": 2048, "V": 50021},
        # Training the classifier: loss and both gradients of the small batch.
        {"name": "grad_classifier", "op": "grad", "T": 32, "D": 512, "V": 1000},
        # Training with odd sizes: a ragged batch of tokens over a middling vocabulary.
        {"name": "grad_ragged", "op": "grad", "T": 1999, "D": 1000, "V": 32001},
        # Training a large output layer: bound by the matrix cores.
        {"name": "grad_large", "op": "grad", "T": 8192, "D": 4096, "V": 32768},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even in its logarithm; rounded to a multiple
    of 64 half the time, left odd or even as it falls otherwise."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 128 and rng.random() < 0.5:
        n = (n + 32) // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(("quantise", "product", "product", "loss", "grad"))
    while True:
        if op == "quantise":
            c = {"op": op, "rows": _log(rng, 1, 65536), "cols": _log(rng, 32, 16384),
                 "dtype": rng.choice(("bf16", "fp32"))}
            if c["rows"] * c["cols"] <= 1 << 25:
                return c
        elif op == "product":
            c = {"op": op, "M": _log(rng, 1, 65536), "N": _log(rng, 64, 65536), "K": _log(rng, 64, 25088),
                 "dtype": rng.choice(("bf16", "bf16", "fp32")), "relu": rng.random() < 0.5}
            if c["M"] * c["N"] * c["K"] <= 1 << 38 and c["N"] * c["K"] <= 1 << 27 and \
                    c["M"] * max(c["K"], c["N"]) <= 1 << 27:
                return c
        else:
            c = {"op": op, "T": _log(rng, 1, 8192), "D": _log(rng, 64, 4096), "V": _log(rng, 500, 65536)}
            if c["T"] * c["D"] * c["V"] <= 1 << 39:
                return c


def work(case):
    if case["op"] == "quantise":
        n, e = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        # x read, its values written; the 4-bit form between them written and read.
        return {"bytes": n * (2 * e + 2 * 17 / 32), "flops": 0}
    if case["op"] == "product":
        M, N, K, e = case["M"], case["N"], case["K"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * K * e + N * K * 17 / 32 + N * 4 + M * N * e, "flops": 2 * M * N * K}
    T, D, V = case["T"], case["D"], case["V"]
    if case["op"] == "loss":
        return {"bytes": 2 * (T * D + V * D) + 16 * T, "flops": 2 * T * D * V}
    # Without the logits kept, the gradient computes them a second time.
    return {"bytes": 4 * (T * D + V * D) + 20 * T, "flops": 8 * T * D * V}


# ---------------------------------------------------------------- plain forms

def _blocks(x):
    """x [rows, cols] in fp32 as blocks of 32 [rows, nb, 32], zeros past cols."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    p = torch.zeros(rows, nb * 32, dtype=torch.float32, device=x.device)
    p[:, :cols] = x
    return p.view(rows, nb, 32)


def _quantise(x):
    """e2m1 codes [rows, nb, 32] (uint8, sign in bit 3) and e8m0 scales [rows, nb]."""
    b = _blocks(x)
    amax = b.abs().amax(-1)
    # frexp: amax = f 2^k with f in [0.5, 1), so floor(log2 amax) = k - 1.
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    # Round to nearest, ties to the even code: each middle belongs to its even neighbour.
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    return code | ((b < 0).to(torch.uint8) << 3), (e + 127).to(torch.uint8)


def _values(codes, scales, cols):
    """The fp32 values [rows, cols] that codes and scales stand for."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    v = lut[codes.int()] * torch.exp2(scales.float() - 127).unsqueeze(-1)
    return v.reshape(codes.shape[0], -1)[:, :cols]


def _unpack(packed):
    """Packed e2m1 pairs (low half first) [rows, nb*16] to codes [rows, nb, 32]."""
    c = torch.stack((packed & 15, packed >> 4), -1)
    return c.reshape(packed.shape[0], -1, 32)


def _plain_product(s):
    x = _values(*_quantise(s["x"]), s["x"].shape[1])
    w = _values(_unpack(s["codes"]), s["scales"], s["x"].shape[1])
    y = x @ w.t() + s["bias"]
    if s["relu"]:
        y = y.relu()
    return y.to(s["x"].dtype)


def _plain_loss(s):
    logits = s["h"].float() @ s["w"].float().t()
    m = logits.amax(1, keepdim=True)
    lse = (m + (logits - m).exp().sum(1, keepdim=True).log()).squeeze(1)
    live = s["target"] != IGNORE
    at = torch.where(live, s["target"], torch.zeros_like(s["target"])).unsqueeze(1)
    loss = torch.where(live, lse - logits.gather(1, at).squeeze(1), torch.zeros_like(lse))
    return logits, lse, loss, live, at


def _plain_grad(s):
    logits, lse, loss, live, at = _plain_loss(s)
    g = (logits - lse.unsqueeze(1)).exp()
    g.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    g *= torch.where(live, s["dloss"], torch.zeros_like(s["dloss"])).unsqueeze(1)
    dh = g @ s["w"].float()
    dw = g.t() @ s["h"].float()
    return {"loss": loss, "lse": lse, "dh": dh.to(s["h"].dtype), "dw": dw.to(s["w"].dtype)}


# ---------------------------------------------------------------- state

def _activations(rows, cols, dtype, g):
    """Activations as they leave a layer: normal values whose size differs from
    feature to feature, with a few features much larger than the others."""
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    size = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 16 * size, size)
    return (torch.randn(rows, cols, generator=g, device=DEV) * size).to(dtype)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "quantise":
        return {"x": _activations(case["rows"], case["cols"], DTYPES[case["dtype"]], g)}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        w = torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)
        codes, scales = _quantise(w)
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        return {"x": _activations(M, K, DTYPES[case["dtype"]], g), "codes": packed.reshape(N, -1),
                "scales": scales, "bias": torch.randn(N, generator=g, device=DEV), "relu": case["relu"]}
    T, D, V = case["T"], case["D"], case["V"]
    s = {"h": torch.randn(T, D, generator=g, device=DEV).to(torch.bfloat16),
         "w": (torch.randn(V, D, generator=g, device=DEV) * (2 / math.sqrt(D))).to(torch.bfloat16),
         "target": torch.randint(0, V, (T,), generator=g, device=DEV)}
    # Padding and prompt tokens carry no loss; the first token always does.
    pad = torch.rand(T, generator=g, device=DEV) < 0.1
    pad[0] = False
    s["target"] = torch.where(pad, torch.full_like(s["target"], IGNORE), s["target"])
    s["dloss"] = (~pad).float() / (~pad).sum()  # the mean over the tokens that count
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if own:
        import convolution_implicit_gemm_nhwc_amd as fc
        if case["op"] == "quantise":
            s["plan"] = fc.MxQuantPlan(case["rows"], case["cols"], case["dtype"])
        elif case["op"] == "product":
            ops = ("bias", "relu") if case["relu"] else ("bias",)
            s["plan"] = fc.MxPlan(case["M"], case["N"], case["K"], case["dtype"], ops=ops)
            # A served layer's weights are laid out once, from the 4-bit checkpoint.
            s["weight"] = fc.MxTensor.from_codes(s["codes"], s["scales"], case["K"])
        else:
            s["plan"] = fc.XentPlan(case["T"], case["D"], case["V"], "bf16", ignore_index=IGNORE)
    return s


def run(state):
    s = state
    if not own:
        if s["op"] == "quantise":
            return _values(*_quantise(s["x"]), s["x"].shape[1]).to(s["x"].dtype)
        if s["op"] == "product":
            return _plain_product(s)
        if s["op"] == "loss":
            _, lse, loss, _, _ = _plain_loss(s)
            return {"loss": loss, "lse": lse}
        return _plain_grad(s)
    plan = s["plan"]
    if s["op"] == "quantise":
        return plan.dequantize(plan(s["x"]))
    if s["op"] == "product":
        return plan(s["x"], s["weight"], bias=s["bias"])
    loss, lse = plan.forward(s["h"], s["w"], s["target"])
    if s["op"] == "loss":
        return {"loss": loss, "lse": lse}
    dh, dw = plan.backward(s["h"], s["w"], s["target"], lse, s["dloss"])
    return {"loss": loss, "lse": lse, "dh": dh, "dw": dw}


# ---------------------------------------------------------------- 64 bits

def _exact_values(x):
    """The values that x's MXFP4 form stands for, in 64 bits: each block's
    nearest representable values by distance, ties to the even code."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    out = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    lut = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 22) // (nb * 32))
    for r in range(0, rows, step):
        part = x[r:r + step].double()
        b = torch.zeros(part.shape[0], nb * 32, dtype=torch.float64, device=x.device)
        b[:, :cols] = part
        b = b.view(-1, nb, 32)
        amax = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))) - 2
        scale = torch.exp2(e.clamp(-127, 127))
        far = ((b.abs() / scale).unsqueeze(-1) - lut).abs()
        near = far.amin(-1, keepdim=True)
        # Of two equally near codes the even one.
        code = torch.arange(8, device=x.device)
        pick = torch.where(far == near, code + 8 * (code % 2), torch.full_like(far, 99, dtype=torch.int64)).argmin(-1)
        out[r:r + step] = (torch.sign(b) * lut[pick] * scale).view(-1, nb * 32)
    return out[:, :cols]


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quantise":
        return _exact_values(s["x"])
    if case["op"] == "product":
        K = case["K"]
        codes = s["codes"].long()
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        w = torch.zeros(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=DEV)
        for half in (0, 1):
            nib = codes >> 4 if half else codes & 15
            w[:, half::2] = torch.where(nib >= 8, -mag[nib % 8], mag[nib % 8])
        w *= torch.pow(2.0, s["scales"].double() - 127).repeat_interleave(32, 1)
        y = torch.addmm(s["bias"].double(), _exact_values(s["x"]), w[:, :K].t())
        return y.clamp_min(0) if case["relu"] else y
    h, w, t = s["h"].double(), s["w"].double(), s["target"]
    logits = torch.mm(h, w.t())
    lse = torch.logsumexp(logits, 1)
    row = torch.arange(t.numel(), device=DEV)[t != IGNORE]
    loss = torch.zeros_like(lse)
    loss[row] = lse[row] - logits[row, t[row]]
    if case["op"] == "loss":
        return {"loss": loss, "lse": lse}
    p = logits.sub_(lse.unsqueeze(1)).exp_()
    p[row, t[row]] -= 1
    scale = torch.zeros_like(lse)
    scale[row] = s["dloss"].double()[row]
    p *= scale.unsqueeze(1)
    return {"loss": loss, "lse": lse, "dh": torch.mm(p, w), "dw": torch.mm(p.t(), h)}
