"""The gated layer's tiled kernels, each chosen by its size and named, against
torch products in 64 bits on the GPU; errors as tests/test_gpu_gated.py derives
them.  Sizes past the caches, weights past 128 MB for a few tokens, and more than
a million tokens of the lookup, whose keys are merged three times."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from test_gpu_gated import TDT, U, case

pytestmark = pytest.mark.gpu


def _act(g):  # silu and its derivative
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    return g * s, s + g * s * c


def _sum_error(a, b):
    n = a.shape[1]
    return 4 * U * n * ((a * a) @ (b * b) / max(n, 1)).sqrt()


def _own(g):
    g = g.abs()
    return (16 + 4 * g + 4 * g ** 2 + g ** 3) * U


def _within(what, got, want, err):
    off = (got.double() - want).abs()
    assert bool((off <= err).all()), (what, float((off / err).max()))


def check(T, D, F, dev, dtype="bf16", x_off=0, w_off=0):
    x, w, dy = case(T, D, F, dtype, dev)
    if x_off:
        x = torch.cat((x, x[:, :8]), 1)[:, :D] if x_off == 8 else torch.nn.functional.pad(x, (x_off, 3))[:, x_off:x_off + D]
    if w_off:
        w = torch.nn.functional.pad(w, (w_off, 2))[:, w_off:w_off + D]
    plan = fc.GatedPlan(T, D, F, dtype)
    y, kept = plan.forward(x, w, keep=True)
    dx, dw = plan.backward(x, w, kept, dy)
    assert torch.equal(plan.forward(x, w), y)
    only_x, _ = plan.backward(x, w, kept, dy, need_dw=False)
    _, only_w = plan.backward(x, w, kept, dy, need_dx=False)
    assert torch.equal(only_x, dx) and torch.equal(only_w, dw)
    r = 2.0 ** -8 if dtype == "bf16" else U
    x, w, dy = x.double(), w.double(), dy.double()
    z, ez = x @ w.t().contiguous(), _sum_error(x, w.t().contiguous())
    g, u, eg, eu = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
    a, da = _act(g)
    want = a * u
    _within("y", y, want, 1.01 * (u.abs() * (1.13 * eg + _own(g) * a.abs()) + a.abs() * eu + (r + 3 * U) * want.abs()) + 1e-37)
    dz = torch.cat((dy * u * da, dy * a), 1)
    edg = dy.abs() * (eu * da.abs() + u.abs() * (eg + 2 * _own(g))) + (r + 4 * U) * dz[:, :F].abs()
    edu = dy.abs() * (1.13 * eg + _own(g) * a.abs()) + (r + 3 * U) * dz[:, F:].abs()
    e = 1.02 * torch.cat((edg, edu), 1)
    want = dz @ w
    _within("dx", dx, want, e @ w.abs() + _sum_error(dz, w) + r * want.abs() + 1e-37)
    dzt, et = dz.t().contiguous(), e.t().contiguous()
    want = dzt @ x
    _within("dw", dw, want, et @ x.abs() + _sum_error(dzt, x) + r * want.abs() + 1e-37)
    return plan


def _names(plan):
    return tuple((plan.kernel_name(n), plan.ranges(n) > 1) for n in ("forward", "dx", "dw"))


SIZES = [  # with the kernels of the forward pass, dx and dw, and whether their sums are divided
    (330, 32, 11350, "gemm_tile_256", "gemm_tile_128", True, "gemm_tile_128", False),
    (2283, 34, 2990, "gemm_tile_256_packed", None, None, None, None),
    (1862, 76, 4346, "gemm_tile_128_packed", None, None, None, None),
    (171, 130, 15352, None, "gemm_tile_256_packed", True, "gemm_tile_256_packed", False),
    (5695, 1480, 8, None, "gemm_tile_256", False, None, None),
    (6600, 1459, 8, None, "gemm_tile_256_packed", False, None, None),
    (4332, 40, 9, None, None, None, "gemm_tile_128", True),
    (7127, 136, 4211, "gemm_tile_256", None, None, "gemm_tile_256", True),
    (1999, 1000, 731, None, None, None, None, None),
    (2048, 1024, 2816, "gemm_tile_256", None, None, None, None),
    (300, 2048, 4099, None, None, None, None, None),
]


@pytest.mark.parametrize("T,D,F,fwd,dx,dx_parts,dw,dw_parts", SIZES)
def test_tiled_kernels(T, D, F, fwd, dx, dx_parts, dw, dw_parts):
    dev = device()
    say("gated tiles", T, D, F)
    names = _names(check(T, D, F, dev))
    say(names)
    for got, want in zip((names[0][0],) + names[1] + names[2], (fwd, dx, dx_parts, dw, dw_parts)):
        assert want is None or got == want, (names, want)


@pytest.mark.parametrize("T", [20, 500, 2100])
@pytest.mark.parametrize("x_off,w_off", [(1, 0), (0, 1), (3, 2), (8, 0)])
def test_rows_that_the_tiles_cannot_copy(T, x_off, w_off):
    # Whole eights, but from addresses or at distances that are no multiple of 16 bytes.
    dev = device()
    say("gated, rows between", T, x_off, w_off)
    check(T, 256, 1040, dev, x_off=x_off, w_off=w_off)


def test_weights_past_the_caches():
    # dw of 64 MB goes past the caches; a few tokens of a 134 MB layer are read by eight waves.
    dev = device()
    say("gated, large w")
    check(700, 2048, 8192, dev)
    for T, dtype in ((1, "bf16"), (3, "fp32"), (8, "bf16")):
        check(T, 4096, 8200 if dtype == "bf16" else 4200, dev, dtype)


def test_a_million_tokens():
    dev = device()
    T, D, V = 1100003, 3, 70000
    say("embed", T)
    g = torch.Generator(device=dev).manual_seed(0)
    token = torch.exp(torch.rand(T, generator=g, device=dev, dtype=torch.float64) * np.log(V)).long() - 1
    token[::7] = -100
    dy = torch.randn(T, D, generator=g, device=dev)
    p = fc.EmbedPlan(T, D, V, "fp32")
    dw = p.backward(token, dy)
    assert torch.equal(dw, p.backward(token, dy))
    live = token != -100
    at = torch.where(live, token, V)
    want = torch.zeros(V + 1, D, dtype=torch.float64, device=dev).index_add_(0, at, dy.double())[:V]
    size = torch.zeros(V + 1, D, dtype=torch.float64, device=dev).index_add_(0, at, dy.double().abs())[:V]
    # Sixty-four terms of a piece one after another, then the pieces': four waves, eight loads, some hundreds in a row.
    n = torch.bincount(at, minlength=V + 1)[:V, None].double()
    steps = torch.minimum(n, torch.full_like(n, 64.0)) + n / 64 / 4 + 8
    _within("dw", dw, want, steps * U * size)
    y = p.forward(dw, torch.where(live, token, 0))
    assert torch.equal(y, dw[torch.where(live, token, 0)])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,F", [(65, 4096, 20), (128, 8192, 33), (300, 1024, 300), (271, 3689, 88), (1000, 515, 50),
                                   (513, 1001, 16), (64, 2048, 17), (40, 3001, 100), (1999, 260, 40)])
def test_long_rows_of_few_outputs(T, D, F, dtype):
    # Workgroups share the tokens, by 16, 32 or 64 of them, past those that one can take.
    dev = device()
    say("gated, few outputs", T, D, F, dtype)
    assert check(T, D, F, dev, dtype).kernel_name("forward") == "gated_few"
    check(T, D, F, dev, dtype, x_off=1, w_off=3)  # rows between dwords: fewer tokens in a workgroup
