"""Gradients whose q = softmax - onehot is made in several pieces of the
vocabulary (more than 512 MB of it), against 64 bits on the GPU in chunks of
tokens.

Tolerances (u = 2^-24): a logit's error is at most 4 u D s with s the root mean
square of its products (ten times what fp32 sums of that many gather), lse's
the same and three steps of lse; so p is off by p (2 ez + 8 u |lse|), q in bf16 by
2^-8 of itself, r h by 2^-8 of itself (fp32: 2 u).  dh and dw sum such terms
in fp32, n of them: 4 u n s again, and are off by 2^-8 of themselves in bf16."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
IGN = -100


def case(T, D, V, dtype, dev, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.randn(T, D, generator=g, device=dev).to(TDT[dtype])
    w = (torch.randn(V, D, generator=g, device=dev) * (2 / D ** 0.5)).to(TDT[dtype])
    t = torch.randint(0, V, (T,), generator=g, device=dev)
    t[torch.rand(T, generator=g, device=dev) < 0.2] = IGN
    dl = torch.randn(T, generator=g, device=dev)
    return h, w, t, dl


def sum_error(a, b, n):
    """4 u n s of a [m, n] times b [n, k], s the root mean square of a sum's products."""
    return 4 * U * n * torch.mm(a * a, b * b).div_(max(n, 1)).sqrt_()


def check(h, w, t, dl, loss, lse, dh, dw, dtype, chunk):
    """All of loss, lse, dh and dw of the tokens t (IGN ignored)."""
    T, D = h.shape
    V = w.shape[0]
    wd = w.double()
    rh = 2.0 ** -8 if dtype == "bf16" else 2 * U
    ro = 2.0 ** -8 if dtype == "bf16" else U
    rq = 2.0 ** -8 if dtype == "bf16" else 2 * U
    rdw = torch.zeros(V, D, dtype=torch.float64, device=h.device)
    edw, sdw = torch.zeros_like(rdw), torch.zeros_like(rdw)
    for i in range(0, T, chunk):
        s = slice(i, min(T, i + chunk))
        hd, keep = h[s].double(), t[s] != IGN
        z = torch.mm(hd, wd.t())
        l = torch.logsumexp(z, 1)
        ez = sum_error(hd, wd.t(), D)
        p = (z - l.unsqueeze(1)).exp_()
        # exp's argument: two roundings of z - max; the sum of V terms is tree-like.
        el = (p * ez).sum(1) * 1.01 + (p * (2 * (z - z.amax(1, keepdim=True)).abs() + 4)).sum(1) * U \
            + (24 + V / 256) * U + 3 * U * l.abs()
        assert bool(((lse[s].double() - l).abs() <= el).all())
        at = torch.where(keep, t[s], 0).unsqueeze(1)
        rl = torch.where(keep, l - z.gather(1, at).squeeze(1), 0)
        assert bool(((loss[s].double() - rl).abs() <= torch.where(keep, el + ez.gather(1, at).squeeze(1)
                                                                  + U * rl.abs(), 0)).all())
        ep = p * (ez + el.unsqueeze(1) + (2 * (z - l.unsqueeze(1)).abs() + 4) * U) + 2 * U * p
        del z, ez
        q = p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
        d = torch.where(keep, dl[s].double(), 0).unsqueeze(1)
        eq = (ep * 1.01 + (rq + 2 * U) * q.abs()) * d.abs()
        g = q * d
        rdh = torch.mm(g, wd)
        edh = 1.01 * torch.mm(eq, wd.abs()) + sum_error(g, wd, V) + ro * rdh.abs() + 1e-37
        assert bool(((dh[s].double() - rdh).abs() <= edh).all())
        hk = torch.where(keep.unsqueeze(1), hd, 0)
        rdw += torch.mm(g.t(), hk)
        edw += torch.mm((eq + rh * g.abs()).t(), hk.abs())
        sdw += torch.mm((g * g).t(), hk * hk)
    edw = 1.01 * edw + 4 * U * T * (sdw / T).sqrt() + ro * rdw.abs() + 1e-37
    assert bool(((dw.double() - rdw).abs() <= edw).all())


def run(T, D, V, dtype, chunk):
    dev = device()
    say("pieces", T, D, V, dtype)
    h, w, t, dl = case(T, D, V, dtype, dev)
    plan = fc.XentPlan(T, D, V, dtype, ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    check(h, w, t, dl, loss, lse, dh, dw, dtype, chunk)
    # The order of the pieces' sums is fixed.
    dh2, dw2 = plan.backward(h, w, t, lse, dl)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2)


# Two and five pieces, few and many tokens; D of whole and ragged tiles, below and above a tile, rows between
# dwords (general kernel) and rows that are packed.
@pytest.mark.parametrize("T,D,V", [(20000, 264, 16500), (70001, 600, 9001), (9000, 72, 40000), (30000, 65, 10007),
                                   (2000, 513, 140001)])
def test_bf16(T, D, V):
    run(T, D, V, "bf16", 4000)


@pytest.mark.parametrize("T,D,V", [(20000, 100, 16500), (40001, 33, 9001)])
def test_fp32(T, D, V):
    run(T, D, V, "fp32", 4000)


def test_few_tokens_of_a_vocabulary_past_a_piece():
    run(40, 16, 4200001, "bf16", 4)
