"""Linear softmax cross entropy and its gradient on the GPU against plain
numpy in 64 bits (oracle/xent.py).

Tolerances, u = 2^-24 (half a step of fp32):
* a logit sums D exact (bf16) or once-rounded (fp32) products in fp32; with
  products of root mean square s the errors add up to about u D s / 2.5, and
  4 u D s is ten of those (`_sum_error`);
* an exponential's argument z - m takes two roundings, its value one step:
  relative error (2 |z - m| + 4) u, weighted by its share p of the sum; the
  sum of V terms is tree-like: at most 16 additions in a lane, 8 joins and one
  addition for every fourth tile; the logarithm adds two steps of lse;
* g = dloss (p - onehot): p is off by p (error of z + error of lse + the
  exponential's), the subtraction by u, p - onehot in bf16 by 2^-8 of itself;
* dh and dw sum products of g, each off by that much, in fp32 (4 u n s again);
  dw's h, scaled by dloss / max |dloss|, is off by 2^-8 of itself in bf16 (by
  2 u in fp32); a bf16 output is off by another 2^-8 of itself."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from oracle import xent as ox

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
IGN = -100


def _case(T, D, V, dtype, seed, dev, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D, generator=g).to(TDT[dtype])
    w = (torch.randn(V, D, generator=g) * (spread / D ** 0.5)).to(TDT[dtype])
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < 0.2] = IGN
    dl = torch.randn(T, generator=g)
    return h.to(dev), w.to(dev), t.to(dev), dl.to(dev)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _sum_error(a, b):
    """4 u n s for a [m, n] times b [n, k]."""
    n = a.shape[1]
    return 4 * U * n * np.sqrt((a ** 2) @ (b ** 2) / max(n, 1))


class Ref:
    def __init__(self, h, w, target, dloss, dtype):
        h, w, t, dl = _np(h), _np(w), target.cpu().numpy(), _np(dloss)
        keep = t != IGN
        self.loss, self.lse, z = ox.forward(h, w, t, IGN)
        self.dh, self.dw, g = ox.backward(h, w, t, self.lse, dl, IGN)
        T, V = z.shape
        p = np.exp(z - self.lse[:, None])
        ez = _sum_error(h, w.T)
        x = np.abs(z - z.max(1, keepdims=True))
        elog = (p * (2 * x + 4)).sum(1) * U + (24 + V / 256) * U
        self.e_lse = (p * ez).sum(1) * 1.01 + elog + 3 * U * np.abs(self.lse)
        at = np.where(keep, t, 0)
        rows = np.arange(T)
        self.e_loss = self.e_lse + ez[rows, at] + U * np.abs(self.loss)
        eg = np.abs(dl)[:, None] * (p * (ez + self.e_lse[:, None] + (2 * np.abs(z - self.lse[:, None]) + 4) * U)
                                    + 2 * U) + 2 * U * np.abs(g)
        r = 2.0 ** -8 if dtype == "bf16" else U
        if dtype == "bf16":
            eg = eg * 1.01 + r * np.abs(g)
        eg[~keep] = 0
        self.e_dh = 1.01 * eg @ np.abs(w) + _sum_error(g, w) + r * np.abs(self.dh) + 1e-37
        gk, hk = g[keep], h[keep]
        eh = r if dtype == "bf16" else 2 * U
        self.e_dw = 1.01 * (eg[keep] + eh * np.abs(gk)).T @ np.abs(hk) + _sum_error(gk.T, hk) + r * np.abs(self.dw) + 1e-37


def _check(h, w, t, dl, dtype, plan=None, **kw):
    T, D = h.shape
    V = w.shape[0]
    plan = plan or fc.XentPlan(T, D, V, dtype, ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl, **kw)
    torch.cuda.synchronize()
    r = Ref(h, w, t, dl, dtype)
    assert (np.abs(_np(lse) - r.lse) <= r.e_lse).all()
    assert (np.abs(_np(loss) - r.loss) <= np.where(t.cpu().numpy() == IGN, 0, r.e_loss)).all()
    assert (np.abs(_np(dh) - r.dh) <= r.e_dh).all()
    assert (np.abs(_np(dw) - r.dw) <= r.e_dw).all()
    return loss, lse, dh, dw


SIZES = [(1, 1, 1), (1, 64, 500), (2, 8, 70), (3, 33, 17), (16, 100, 300), (17, 1000, 1003), (32, 512, 1000),
         (64, 64, 64), (65, 130, 257), (130, 511, 129), (33, 8, 5000), (200, 96, 700), (300, 520, 1100),
         (700, 64, 600), (1500, 72, 520)]
# At most 64 tokens, and the first number above; k of less than a step, whole steps, a ragged rest; many groups of v.
SIZES += [(16, 64, 33), (33, 127, 40), (48, 257, 65), (63, 1000, 999), (64, 576, 2000), (66, 576, 2000), (5, 40, 70001),
          (30, 64, 140000), (3, 1024, 70000)]
# Few tokens and k of less than eight, of eight and a little, of whole steps and a ragged end; a vocabulary of dh's own kernel.
SIZES += [(2, 3, 40), (9, 9, 1000), (20, 71, 300), (34, 199, 2048), (64, 452, 1024), (17, 600, 2049), (40, 515, 1025)]
# Tokens counted in blocks, gathered by four and by sixteen; many ranges of few outputs.
SIZES += [(2049, 40, 300), (4100, 24, 260), (3, 40, 60000), (20, 72, 40000)]
# Rows that are no multiple of 16 bytes, packed for the tiled kernel.
SIZES += [(513, 1001, 3000), (700, 260, 5000), (1100, 513, 2500)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_loss_and_gradient(T, D, V, dtype):
    dev = device()
    say("xent", T, D, V, dtype)
    _check(*_case(T, D, V, dtype, T + D + V, dev), dtype)


@pytest.mark.parametrize("T,D,V,hoff,woff", [(5, 64, 90, 1, 0), (40, 128, 200, 0, 1), (40, 130, 200, 1, 1), (64, 77, 70, 3, 2),
                                           (90, 128, 200, 1, 0), (90, 65, 300, 0, 3), (90, 192, 130, 2, 1)])
def test_rows_between_dwords(T, D, V, hoff, woff):
    # bf16 rows that begin at any element, with an odd and an even distance, of both operands.
    dev = device()
    say("odd rows", T, D, V, hoff, woff)
    for extra in (0, 1):
        h, w, t, dl = _case(T, D, V, "bf16", 3, dev)
        hb = torch.full((T, D + hoff + extra), float("nan"), dtype=torch.bfloat16, device=dev)
        wb = torch.full((V, D + woff + extra), float("nan"), dtype=torch.bfloat16, device=dev)
        hb[:, hoff:hoff + D], wb[:, woff:woff + D] = h, w
        _check(hb[:, hoff:hoff + D], wb[:, woff:woff + D], t, dl, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_logits(dtype):
    # Logits of some hundreds: most exponentials underflow.
    dev = device()
    say("large logits", dtype)
    _check(*_case(70, 64, 600, dtype, 4, dev, spread=300.0), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,V", [(40, 50, 333), (300, 128, 600)])
def test_strided_unaligned_rows_and_guards(T, D, V, dtype):
    dev = device()
    say("strided", T, D, V, dtype)
    h, w, t, dl = _case(T, D + 5, V, dtype, 3, dev)
    h, w = h[:, 3:3 + D], w[:, 1:1 + D]
    bh = torch.full((T, D + 9), 7.0, dtype=TDT[dtype], device=dev)
    bw = torch.full((V, D + 3), 7.0, dtype=TDT[dtype], device=dev)
    _check(h, w, t, dl, dtype, dh=bh[:, 5:5 + D], dw=bw[:, 1:1 + D])
    assert (bh[:, :5] == 7).all() and (bh[:, 5 + D:] == 7).all()
    assert (bw[:, :1] == 7).all() and (bw[:, 1 + D:] == 7).all()


@pytest.mark.parametrize("T,D,V", [(1, 64, 500), (37, 40, 300), (600, 256, 600)])
def test_ignored_tokens_hold_anything(T, D, V):
    # NaN and infinities of ignored tokens, and of their dloss, reach nothing but their own lse.
    dev = device()
    say("ignored", T, D, V)
    h, w, t, dl = _case(T, D, V, "bf16", 9, dev)
    t[0] = IGN if T > 1 else t[0].clamp_min(0)
    dead = t == IGN
    h2, dl2 = h.clone(), dl.clone()
    h2[dead] = float("nan")
    h2[dead, 0] = float("inf")
    dl2[dead] = float("nan")
    plan = fc.XentPlan(T, D, V, "bf16", ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    loss2, lse2 = plan.forward(h2, w, t)
    dh2, dw2 = plan.backward(h2, w, t, lse2, dl2)
    assert torch.equal(loss, loss2) and torch.equal(lse[~dead], lse2[~dead])
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2)
    assert (loss[dead] == 0).all() and (dh[dead] == 0).all()


@pytest.mark.parametrize("T,D,V", [(1, 33, 50), (20, 64, 300), (300, 64, 520)])
def test_all_tokens_ignored(T, D, V):
    dev = device()
    say("all ignored", T, D, V)
    h, w, t, dl = _case(T, D, V, "bf16", 9, dev)
    t.fill_(IGN)
    plan = fc.XentPlan(T, D, V, "bf16", ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    assert (loss == 0).all() and (dh == 0).all() and (dw == 0).all()


def test_ignore_index_may_be_a_class():
    dev = device()
    say("ignore class 3")
    h, w, t, dl = _case(50, 64, 10, "fp32", 9, dev)
    t = t.clamp_min(0)
    plan = fc.XentPlan(50, 64, 10, "fp32", ignore_index=3)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    rl, rlse, _ = ox.forward(_np(h), _np(w), t.cpu().numpy(), 3)
    rdh, rdw, _ = ox.backward(_np(h), _np(w), t.cpu().numpy(), rlse, _np(dl), 3)
    assert ((loss == 0) == (t == 3)).all()
    # fp32 sums of a few hundred terms of order one: 1e-4 is far above their error.
    assert np.abs(_np(loss) - rl).max() < 1e-4
    assert np.abs(_np(dh) - rdh).max() < 1e-4 and np.abs(_np(dw) - rdw).max() < 1e-4


def test_target_out_of_range_is_nan():
    dev = device()
    say("bad target")
    h, w, t, dl = _case(40, 64, 100, "bf16", 9, dev)
    t = t.clamp_min(0)
    t[5], t[6], t[7] = 100, -1, 1 << 40
    plan = fc.XentPlan(40, 64, 100, "bf16", ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    bad = torch.zeros(40, dtype=torch.bool, device=dev)
    bad[5:8] = True
    assert torch.equal(torch.isnan(loss), bad) and not torch.isnan(lse).any()
    dh, dw = plan.backward(h, w, t, lse, dl)
    assert torch.equal(torch.isnan(dh).any(1), bad) and torch.isnan(dw).all()


@pytest.mark.parametrize("T,V", [(4, 300), (300, 700)])
def test_infinite_and_nan_logits(T, V):
    dev = device()
    say("infinite logits", T, V)
    h, w, t, dl = _case(T, 64, V, "bf16", 9, dev)
    t = t.clamp_min(0)
    h[:, 0] = 1.0
    h[0, 0] = 0.0  # 0 * inf: NaN
    h[1, 0] = -1.0
    w[7, 0] = float("inf")
    t[2] = 7
    t[1] = 8
    t[3] = 9
    loss, lse = fc.XentPlan(T, 64, V, "bf16").forward(h, w, t)
    rl, rlse, _ = ox.forward(_np(h), _np(w), t.cpu().numpy())
    got = _np(lse)
    assert np.isnan(got[0]) and np.isfinite(got[1]) and (got[2:] == np.inf).all()
    assert abs(got[1] - rlse[1]) < 1e-4
    assert np.array_equal(np.isnan(_np(loss)), np.isnan(rl))
    assert np.array_equal(np.isinf(_np(loss)), np.isinf(rl))


def test_all_logits_minus_infinity():
    dev = device()
    say("minus infinity")
    h = torch.ones(3, 8, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(200, 8, dtype=torch.bfloat16, device=dev)
    w[:, 0] = float("-inf")
    _, lse = fc.XentPlan(3, 8, 200, "bf16").forward(h, w, torch.zeros(3, dtype=torch.int64, device=dev))
    assert (lse == float("-inf")).all()


def test_one_gradient_alone():
    dev = device()
    say("one gradient")
    h, w, t, dl = _case(90, 64, 300, "bf16", 9, dev)
    plan = fc.XentPlan(90, 64, 300, "bf16")
    _, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    dh1, none = plan.backward(h, w, t, lse, dl, need_dw=False)
    assert none is None and torch.equal(dh, dh1)
    none, dw1 = plan.backward(h, w, t, lse, dl, need_dh=False)
    assert none is None and torch.equal(dw, dw1)


@pytest.mark.parametrize("scale", [1e-30, 1e30, 0.0])
def test_scale_of_the_loss_gradient(scale):
    dev = device()
    say("dloss times", scale)
    h, w, t, dl = _case(70, 64, 300, "bf16", 9, dev)
    plan = fc.XentPlan(70, 64, 300, "bf16")
    _, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl * scale)
    if scale == 0.0:
        assert (dh == 0).all() and (dw == 0).all()
        return
    r = Ref(h, w, t, dl, "bf16")
    # The scaled dloss itself is rounded once more.
    assert (np.abs(_np(dh) / scale - r.dh) <= r.e_dh * 1.01).all()
    assert (np.abs(_np(dw) / scale - r.dw) <= r.e_dw * 1.01).all()


def test_no_tokens():
    dev = device()
    say("no tokens")
    plan = fc.XentPlan(0, 24, 50, "bf16")
    h = torch.empty(0, 24, dtype=torch.bfloat16, device=dev)
    w = torch.randn(50, 24, device=dev).bfloat16()
    t = torch.empty(0, dtype=torch.int64, device=dev)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, torch.empty(0, device=dev))
    assert loss.numel() == 0 and dh.shape == (0, 24) and (dw == 0).all()


def test_gradient_against_differences():
    # d/de of sum(dloss * loss) along a direction, from forward passes alone.
    dev = device()
    say("differences")
    T, D, V = 6, 12, 23
    h, w, t, dl = _case(T, D, V, "fp32", 5, dev)
    plan = fc.XentPlan(T, D, V, "fp32")
    _, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    g = torch.Generator().manual_seed(1)
    uh, uw = torch.randn(T, D, generator=g).to(dev), 0.3 * torch.randn(V, D, generator=g).to(dev)
    eps = 2.0 ** -6
    hd, ud, wd, vd = _np(h), _np(uh), _np(w), _np(uw)
    r = Ref(h, w, t, dl, "fp32")
    live = t.cpu().numpy() != IGN
    for sh, sw, got in ((1, 0, (dh.double() * uh).sum().item()), (0, 1, (dw.double() * uw).sum().item())):
        lp, _ = plan.forward(h + eps * sh * uh, w + eps * sw * uw, t)
        lm, _ = plan.forward(h - eps * sh * uh, w - eps * sw * uw, t)
        diff = ((lp.double() - lm.double()) * dl.double()).sum().item() / (2 * eps)
        # The logits move by at most a along the direction; the third derivative of lse is a third cumulant,
        # at most 2 a^3, and enters with eps^2 / 6.  The moved points' own roundings: one step of |h| and |w|.
        a = np.abs(sh * ud @ wd.T + sw * hd @ vd.T).max(1)
        move = 2 * U * (np.abs(hd) @ np.abs(wd).T).max(1)
        tol = (np.abs(_np(dl)) * (eps ** 2 / 6 * 2 * a ** 3 + (2 * r.e_loss + 2 * move) / (2 * eps)))[live].sum()
        tol += (r.e_dh * np.abs(ud)).sum() * sh + (r.e_dw * np.abs(vd)).sum() * sw
        assert abs(diff - got) <= 1.1 * tol, (diff, got, tol)


def test_many_pieces_and_counted_tokens():
    # Enough tokens that g is made in several pieces of the vocabulary and live tokens are counted apart.  64-bit products on
    # the GPU as the reference, in chunks.
    dev = device()
    T, D, V = 700001, 8, 1100
    say("pieces", T, D, V)
    h, w, t, dl = _case(T, D, V, "bf16", 2, dev)
    plan = fc.XentPlan(T, D, V, "bf16", ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    rdw = torch.zeros(V, D, dtype=torch.float64, device=dev)
    adw = torch.zeros(V, D, dtype=torch.float64, device=dev)
    wd = w.double()
    for i in range(0, T, 100000):
        s = slice(i, min(T, i + 100000))
        hd, keep = h[s].double(), t[s] != IGN
        z = torch.mm(hd, wd.t())
        l = torch.logsumexp(z, 1)
        assert ((lse[s].double() - l).abs() < 1e-5).all()
        at = torch.where(keep, t[s], 0).unsqueeze(1)
        rl = torch.where(keep, l - z.gather(1, at).squeeze(1), 0)
        assert ((loss[s].double() - rl).abs() < 1e-5).all()
        gr = (z - l.unsqueeze(1)).exp()
        gr.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
        gr *= torch.where(keep, dl[s].double(), 0).unsqueeze(1)
        rdh = torch.mm(gr, wd)
        # g off by 2^-8 of itself and a little, dh by another 2^-8.
        tol = 2.0 ** -8 * 1.02 * (torch.mm(gr.abs(), wd.abs()) + rdh.abs()) + 1e-6
        assert ((dh[s].double() - rdh).abs() <= tol).all()
        rdw += torch.mm(gr.t(), hd)
        adw += torch.mm(gr.abs().t(), hd.abs())
    assert ((dw.double() - rdw).abs() <= 2.0 ** -8 * 1.02 * (2 * adw + rdw.abs()) + 1e-3).all()


@pytest.mark.parametrize("T,D,V", [(1, 128, 600), (32, 512, 1000), (300, 256, 700)])
def test_same_bits_on_every_run_streams_and_graphs(T, D, V):
    dev = device()
    say("streams", T, D, V)
    h, w, t, dl = _case(T, D, V, "bf16", 2, dev)
    plan = fc.XentPlan(T, D, V, "bf16")
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        l1, s1 = plan.forward(h, w, t, stream=side)
        a1, b1 = plan.backward(h, w, t, s1, dl, stream=side)
        side.synchronize()
        assert torch.equal(l1, loss) and torch.equal(s1, lse) and torch.equal(a1, dh) and torch.equal(b1, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l2, s2 = plan.forward(h, w, t)
        a2, b2 = plan.backward(h, w, t, s2, dl)
    for _ in range(3):
        for x in (l2, s2, a2, b2):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(a2, dh) and torch.equal(b2, dw)
        plan.forward(h, w, t)


def _far(T, D, V, dtype, value, seed, dev):
    """Logits near the end of fp32's range: every row of w has `value` in
    column 0, times h's 1 there, but for V / 3 rows that have half of it; the
    other columns' products are lost beside it."""
    h, w, t, dl = _case(T, D, V, dtype, seed, dev)
    h[:, 0] = 1.0
    w[:, 0] = value
    w[: V // 3, 0] = value / 2
    return h, w, t, dl


@pytest.mark.parametrize("value", [3.0e38, -3.0e38])
@pytest.mark.parametrize("T,D,V", [(4, 40, 90), (100, 64, 300), (300, 128, 700)])
def test_logits_near_the_end_of_the_range(T, D, V, value):
    # All logits are one of two far values, exactly (fp32 loses the rest): the softmax is even over the larger ones.
    dev = device()
    for dtype in ("bf16", "fp32"):
        say("far logits", T, D, V, value, dtype)
        h, w, t, dl = _far(T, D, V, dtype, value, 3, dev)
        top = torch.arange(V, device=dev) >= V // 3
        if value < 0:
            top = ~top
        t = torch.where(t == IGN, t, torch.nonzero(top)[t % int(top.sum())].squeeze(1))
        plan = fc.XentPlan(T, D, V, dtype, ignore_index=IGN)
        loss, lse = plan.forward(h, w, t)
        big = w[top][0, 0].float()
        assert (lse == big).all()  # the logarithm of a count is far below a step
        assert (loss == 0).all()
        dh, dw = plan.backward(h, w, t, lse, dl)
        # exp(z - lse) is 1 for the larger logits, which fp32 cannot tell from lse, 0 for the others.
        live = t != IGN
        q = top.double().repeat(T, 1)
        q[live, t[live]] -= 1
        q *= torch.where(live, dl.double(), 0).unsqueeze(1)
        rdw = torch.mm(q.t(), h.double())
        adw = torch.mm(q.abs().t(), h.double().abs())
        r = 2.0 ** -8 if dtype == "bf16" else 4 * U
        assert ((dw.double() - rdw).abs() <= 1.01 * r * (adw + rdw.abs()) + 4 * U * T * adw).all()
        rdh = torch.mm(q[:, :], w.double())
        adh = torch.mm(q.abs(), w.double().abs())
        # Sums past fp32's range are infinities; the other columns are of order one.
        assert ((dh.double() - rdh).abs()[:, 1:] <= (1.01 * r * (adh + rdh.abs()) + 4 * U * V * adh)[:, 1:]).all()


def test_both_ways_through_a_call_agree():
    # Without a stream a call goes through csrc/call.cpp, with one or with given outputs through _dense.py.
    dev = device()
    say("ways")
    h, w, t, dl = _case(30, 64, 300, "bf16", 9, dev)
    plan = fc.XentPlan(30, 64, 300, "bf16")
    here = torch.cuda.current_stream()
    loss, lse = plan.forward(h, w, t)
    l2, s2 = plan.forward(h, w, t, stream=here)
    assert torch.equal(loss, l2) and torch.equal(lse, s2)
    dh, dw = plan.backward(h, w, t, lse, dl)
    a, b = plan.backward(h, w, t, lse, dl, dh=torch.empty_like(dh), dw=torch.empty_like(dw))
    assert torch.equal(dh, a) and torch.equal(dw, b)
    for bad, match in ((dict(h=h.float()), "dtype"), (dict(h=h[:29]), "shape"), (dict(w=w.cpu()), "GPU"),
                       (dict(target=t.int()), "dtype"), (dict(target=t[:7]), "elements")):
        with pytest.raises(ValueError, match=match):
            plan.forward(**dict(dict(h=h, w=w, target=t), **bad))
    with pytest.raises(ValueError, match="dtype"):
        plan.backward(h, w, t, lse, dl.double())
