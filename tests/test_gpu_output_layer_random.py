"""The output layer's operators at random sizes, types, strides, offsets,
masks and outputs, against 64 bits on the GPU (tolerances of
test_gpu_xent_pieces.py; of the product: 4 u K s with u = 2^-24 and s the root
mean square of an output's products, the bias's addition, half a step of bf16)."""
import math
import random

import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from test_gpu_xent_pieces import IGN, TDT, U, case, check, sum_error

pytestmark = pytest.mark.gpu


def _size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 16 and rng.random() < 0.4:
        n = (n + 4) // 8 * 8
    return max(lo, min(hi, n))


def _apart(rng, t, dev):
    """t, its rows sometimes apart and off their boundaries, NaN around them."""
    if rng.random() < 0.5:
        return t
    rows, cols = t.shape
    off, gap = rng.choice((0, 1, 3, 8)), rng.choice((0, 1, 5, 8))
    b = torch.full((rows, off + cols + gap), float("nan"), dtype=t.dtype, device=dev)
    b[:, off:off + cols] = t
    return b[:, off:off + cols]


def _out(rng, rows, cols, dtype, dev):
    """None, or a place for an output inside a larger buffer of sevens."""
    if rng.random() < 0.5:
        return None, None
    off, gap = rng.choice((0, 1, 4, 8)), rng.choice((0, 3, 8))
    b = torch.full((rows, off + cols + gap), 7.0, dtype=dtype, device=dev)
    return b, b[:, off:off + cols]


def _clean(b, out):
    if b is None:
        return True
    b = b.clone()
    off = (out.storage_offset()) % b.shape[1] if b.shape[0] else 0
    b[:, off:off + out.shape[1]] = 7
    return bool((b == 7).all())


def run_xent(seed):
    dev, rng = device(), random.Random(seed)
    while True:
        T, D, V = _size(rng, 1, 6000), _size(rng, 1, 2500), _size(rng, 1, 40000)
        if T * D * V <= 1 << 33 and T * V <= 1 << 26:
            break
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    h, w, t, dl = case(T, D, V, dtype, dev, seed)
    mask = rng.choice(("some", "none", "all", "ends"))
    if mask == "none":
        t = torch.where(t == IGN, 0, t)
    elif mask == "all":
        t.fill_(IGN)
    elif mask == "ends":
        t[: T // 3] = IGN
        t[T - T // 4:] = IGN
    dl = rng.choice((dl, torch.full_like(dl, 1.0 / T), dl * 1e-20))
    h, w = _apart(rng, h, dev), _apart(rng, w, dev)
    (bh, oh), (bw, ow) = _out(rng, T, D, h.dtype, dev), _out(rng, V, D, h.dtype, dev)
    plan = fc.XentPlan(T, D, V, dtype, ignore_index=IGN)
    say("xent", seed, T, D, V, dtype, mask, [plan.kernel_name(k) for k in ("logits", "grad", "dh", "dw")],
        h.stride(), h.storage_offset(), w.stride(), w.storage_offset(), bh is None, bw is None)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl, dh=oh, dw=ow)
    check(h, w, t, dl, loss, lse, dh, dw, dtype, 3000)
    assert _clean(bh, dh) and _clean(bw, dw)
    a, none = plan.backward(h, w, t, lse, dl, need_dw=False)
    assert none is None and torch.equal(a, dh)
    none, b = plan.backward(h, w, t, lse, dl, need_dh=False)
    assert none is None and torch.equal(b, dw)


def run_mx(seed):
    dev, rng = device(), random.Random(1000000 + seed)
    while True:
        M, N, K = _size(rng, 1, 20000), _size(rng, 1, 20000), _size(rng, 1, 20000)
        if M * N * K <= 1 << 34 and max(M * N, M * K, N * K) <= 1 << 27:
            break
    dtype = rng.choice(("bf16", "fp32"))
    act = rng.choice((None, None, "relu", "leaky_relu", "clipped_relu", "clamp"))
    ops = (("bias",) if rng.random() < 0.5 else ()) + ((act,) if act else ())
    plan = fc.MxPlan(M, N, K, dtype, ops=ops)
    g = torch.Generator(device=dev).manual_seed(seed)
    x = _apart(rng, torch.randn(M, K, generator=g, device=dev).to(TDT[dtype]), dev)
    w = _apart(rng, torch.randn(N, K, generator=g, device=dev), dev)
    bias = torch.randn(N, generator=g, device=dev) if "bias" in ops else None
    say("mx", seed, M, N, K, dtype, ops, plan.kernel_name, plan.quantized_kernel_name, x.stride(), x.storage_offset())
    qw, qx = fc.MxQuantPlan(N, K, "fp32"), fc.MxQuantPlan(M, K, dtype)
    w4, x4 = qw(w), qx(x)
    xv, wv = fc.MxQuantPlan(M, K, "fp32").dequantize(x4).double(), qw.dequantize(w4).double().t()
    al, be = (-0.5, 1.0) if act == "clamp" else (0.25, 0.0)
    ref = torch.mm(xv, wv)
    if bias is not None:
        ref += bias.double()
    bound = sum_error(xv, wv, K) + U * ref.abs() + (2.0 ** -8 * ref.abs() if dtype == "bf16" else 0) + 1e-37
    ref = {"relu": lambda v: v.clamp_min(0), "leaky_relu": lambda v: torch.where(v > 0, v, al * v),
           "clipped_relu": lambda v: v.clamp(0, al), "clamp": lambda v: v.clamp(al, be)}.get(act, lambda v: v)(ref)
    for given in (x, x4):
        b, out = _out(rng, M, N, TDT[dtype], dev)
        y = plan(given, w4, bias=bias, out=out, activ_alpha=al, activ_beta=be)
        assert bool(((y.double() - ref).abs() <= bound).all())
        assert _clean(b, y)


@pytest.mark.parametrize("seed", range(60))
def test_cross_entropy(seed):
    run_xent(seed)


@pytest.mark.parametrize("seed", range(60))
def test_product(seed):
    run_mx(seed)
