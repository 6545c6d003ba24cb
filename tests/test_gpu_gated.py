"""The gated feed-forward layer and its gradients on the GPU against plain
numpy in 64 bits (oracle/gated.py).

Tolerances, u = 2^-24 (half a step of fp32), r = half a step of the type (2^-8
of the value for bf16, u for fp32):
* g and u sum D products, exact or once rounded, in fp32; with products of root
  mean square s their errors add up to about u D s / 2.5, and 4 u D s is ten of
  those (`_sum_error`);
* an activation's slope is at most 1.13 and its second derivative below 1
  (relu's slope jumps at 0: there the whole slope may be wrong within g's
  error); its own evaluation rounds an exponent's argument, off by
  (|g| + g^2 + |g|^3 / 10) u, and some ten steps of the result: `_own`;
* g and u are kept in fp32; dg and du are rounded by r, and so is every output."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from oracle import gated as og

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def case(T, D, F, dtype, dev, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed + T + D + F)
    x = torch.randn(T, D, generator=g).to(TDT[dtype])
    w = (torch.randn(2 * F, D, generator=g) * (spread / D ** 0.5)).to(TDT[dtype])
    dy = torch.randn(T, F, generator=g).to(TDT[dtype])
    return x.to(dev), w.to(dev), dy.to(dev)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _sum_error(a, b):
    n = a.shape[1]
    return 4 * U * n * np.sqrt((a ** 2) @ (b ** 2) / max(n, 1))


def _own(g):
    g = np.abs(g)
    return (16 + 4 * g + 4 * g ** 2 + g ** 3) * U


class Ref:
    def __init__(self, x, w, dy, dtype, name):
        x, w, dy = _np(x), _np(w), _np(dy)
        F = w.shape[0] // 2
        r = 2.0 ** -8 if dtype == "bf16" else U
        self.y, g, u = og.forward(x, w, name)
        self.dx, self.dw, dz = og.backward(x, w, g, u, dy, name)
        a, da = og.act(g, name)
        ez = _sum_error(x, w.T)
        eg, eu = ez[:, :F], ez[:, F:]
        self.e_y = 1.01 * (np.abs(u) * (1.13 * eg + _own(g) * np.abs(a)) + np.abs(a) * eu + (r + 3 * U) * np.abs(self.y)) + 1e-37
        slope = np.where(np.abs(g) <= eg, 1.0, 0.0) if name == "relu" else eg
        edg = np.abs(dy) * (eu * np.abs(da) + np.abs(u) * (slope + 2 * _own(g))) + (r + 4 * U) * np.abs(dz[:, :F])
        edu = np.abs(dy) * (1.13 * eg + _own(g) * np.abs(a)) + (r + 3 * U) * np.abs(dz[:, F:])
        edz = 1.02 * np.concatenate((edg, edu), 1)
        self.e_dx = edz @ np.abs(w) + _sum_error(dz, w) + r * np.abs(self.dx) + 1e-37
        self.e_dw = edz.T @ np.abs(x) + _sum_error(dz.T, x) + r * np.abs(self.dw) + 1e-37


def check(x, w, dy, dtype, name, plan=None, y=None, **out):
    T, D = x.shape
    F = w.shape[0] // 2
    plan = plan or fc.GatedPlan(T, D, F, dtype, activation=name)
    got, kept = plan.forward(x, w, keep=True, y=y)
    dx, dw = plan.backward(x, w, kept, dy, **out)
    alone = plan.forward(x, w)
    torch.cuda.synchronize()
    assert torch.equal(alone, got)
    ref = Ref(x, w, dy, dtype, name)
    for what, value, want, err in (("y", got, ref.y, ref.e_y), ("dx", dx, ref.dx, ref.e_dx), ("dw", dw, ref.dw, ref.e_dw)):
        off = np.abs(_np(value) - want)
        assert (off <= err).all(), (what, float((off / err).max()), np.argwhere(~(off <= err))[:4])
    return got, dx, dw


# One token up to the few-token kernel's end; k below eight, of less than a step, of whole steps and a rest; f below
# sixteen and odd; general tiles; tiled kernels of 128 and 256 with and without ranges; rows packed to 16 bytes.
SIZES = [(1, 1, 1), (1, 64, 16), (1, 4096, 40), (2, 5, 3), (3, 33, 17), (5, 257, 100), (16, 128, 48), (17, 1000, 203), (31, 72, 65),
         (32, 512, 1000), (33, 127, 31), (48, 1024, 77), (64, 200, 129), (64, 576, 300), (65, 64, 8), (66, 7, 9),
         (100, 513, 200), (130, 130, 130), (257, 40, 33), (200, 96, 700), (300, 520, 333), (513, 1001, 1400), (700, 260, 2500),
         (1500, 72, 520), (2049, 264, 1029), (40, 2048, 1024), (1100, 512, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_layer_and_gradients(T, D, F, dtype):
    dev = device()
    name = ACTS[(T + D + F) % 4]
    say("gated", T, D, F, dtype, name)
    check(*case(T, D, F, dtype, dev), dtype, name)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,F", [(7, 40, 50), (90, 64, 100), (600, 512, 640)])
def test_every_activation(T, D, F, dtype, name):
    # Gates far into both tails.
    dev = device()
    say("gated", name, T, D, F, dtype)
    check(*case(T, D, F, dtype, dev, seed=1, spread=6.0), dtype, name)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,F", [(70, 33, 21), (200, 101, 333), (960, 72, 119), (500, 5, 7), (130, 250, 43)])
@pytest.mark.parametrize("gap", [1, 7, 40])
def test_what_lies_between_rows_reaches_nothing(T, D, F, gap, dtype):
    # Loads of a row's last elements may read what follows them.
    dev = device()
    say("between rows:", T, D, F, gap, dtype)
    x, w, dy = case(T, D, F, dtype, dev)
    p = fc.GatedPlan(T, D, F, dtype, "silu")
    y, kept = p.forward(x, w, keep=True)
    dx, dw = p.backward(x, w, kept, dy)

    def apart(t):
        whole = torch.full((t.shape[0], t.shape[1] + gap), float("nan"), dtype=t.dtype, device=dev)
        whole[:, :t.shape[1]] = t
        return whole[:, :t.shape[1]]
    x2, w2, dy2 = apart(x), apart(w), apart(dy)
    y2, kept2 = p.forward(x2, w2, keep=True)
    out = [torch.full((r, D + gap), 5.0, dtype=x.dtype, device=dev) for r in (T, 2 * F)]
    dx2, dw2 = p.backward(x2, w2, kept2, dy2, dx=out[0][:, :D], dw=out[1][:, :D])
    # Rows elsewhere in memory may be multiplied by another kernel: off by its order of
    # the sum, then one rounding more.
    for a, b, n in ((y, y2, D), (dx, dx2, 2 * F), (dw, dw2, T)):
        eps = torch.finfo(x.dtype).eps + 4 * n * torch.finfo(torch.float32).eps
        assert not torch.isnan(b).any()
        assert (a.double() - b.double()).norm() <= eps * a.double().norm()
    for o in out:
        assert (o[:, D:] == 5.0).all()
