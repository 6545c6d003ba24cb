"""The linear softmax cross entropy where tensors pass 2^31 elements: sampled
tokens and vocabulary rows against 64 bits on the GPU, with the tolerances of
test_gpu_xent_pieces.py."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from test_gpu_xent_pieces import IGN, TDT, U, case, sum_error

pytestmark = pytest.mark.gpu


def check_tokens(h, w, t, dl, loss, lse, dh, rows):
    """loss, lse and dh of some tokens."""
    D, V = h.shape[1], w.shape[0]
    hd = h[rows].double()
    z, ez = [], []
    step = max(1, (1 << 28) // D)
    for v in range(0, V, step):
        wd = w[v:v + step].double()
        z.append(torch.mm(hd, wd.t()))
        ez.append(sum_error(hd, wd.t(), D))
    z, ez = torch.cat(z, 1), torch.cat(ez, 1)
    l = torch.logsumexp(z, 1)
    p = (z - l.unsqueeze(1)).exp()
    el = (p * ez).sum(1) * 1.01 + (p * (2 * (z - z.amax(1, keepdim=True)).abs() + 4)).sum(1) * U \
        + (24 + V / 256) * U + 3 * U * l.abs()
    assert bool(((lse[rows].double() - l).abs() <= el).all())
    keep = t[rows] != IGN
    at = torch.where(keep, t[rows], 0).unsqueeze(1)
    rl = torch.where(keep, l - z.gather(1, at).squeeze(1), 0)
    assert bool(((loss[rows].double() - rl).abs() <= torch.where(keep, el + ez.gather(1, at).squeeze(1)
                                                                 + U * rl.abs(), 0)).all())
    ep = p * (ez + el.unsqueeze(1) + (2 * (z - l.unsqueeze(1)).abs() + 4) * U) + 2 * U * p
    q = p.scatter_add(1, at, torch.full_like(at, -1, dtype=torch.float64))
    d = torch.where(keep, dl[rows].double(), 0).unsqueeze(1)
    g, eg = q * d, (ep * 1.01 + (2.0 ** -8 + 2 * U) * q.abs()) * d.abs()
    rdh, edh, sdh = 0, 0, 0
    for v in range(0, V, step):
        wd, s = w[v:v + step].double(), slice(v, v + step)
        rdh = rdh + torch.mm(g[:, s], wd)
        edh = edh + torch.mm(eg[:, s], wd.abs())
        sdh = sdh + torch.mm(g[:, s] ** 2, wd ** 2)
    edh = 1.01 * edh + 4 * U * V * (sdh / V).sqrt() + 2.0 ** -8 * rdh.abs() + 1e-37
    assert bool(((dh[rows].double() - rdh).abs() <= edh).all())


def check_vocabulary(h, w, t, dl, lse, dw, rows):
    """dw of some rows, given that lse is right."""
    T, D = h.shape
    keep = t != IGN
    hd = torch.where(keep.unsqueeze(1), h.double(), 0)
    wd = w[rows].double()
    z = torch.mm(hd, wd.t())
    l = lse.double().unsqueeze(1)
    # lse is off by a mean of the logits' errors, at most the largest of many rows' here, and some steps more.
    ez = sum_error(hd, wd.t(), D)
    e = ez + ez.amax(1, keepdim=True) + (3 * l.abs() + 2 * (z - l).abs() + 64 + w.shape[0] / 256) * U
    p = (z - l).exp()
    q = p - (t.unsqueeze(1) == rows).double()
    d = torch.where(keep, dl.double(), 0).unsqueeze(1)
    g, eg = q * d, (1.01 * p * (e + 2 * U) + 2.0 ** -8 * q.abs()) * d.abs()
    ref = torch.mm(g.t(), hd)
    err = 1.01 * torch.mm((eg + 2.0 ** -8 * g.abs()).t(), hd.abs()) + sum_error(g.t(), hd, T) + 2.0 ** -8 * ref.abs()
    assert bool(((dw[rows].double() - ref).abs() <= err + 1e-37).all())


def _ends(n, k, dev):
    """The first and last of n, and some between."""
    g = torch.Generator(device=dev).manual_seed(5)
    return torch.cat([torch.arange(min(n, k), device=dev), torch.randint(0, n, (k,), generator=g, device=dev),
                      torch.arange(max(0, n - k), n, device=dev)]).unique()


@pytest.mark.parametrize("T,D,V", [(3, 8200, 262145), (200, 8192, 262147), (70, 2048, 1 << 20)])
def test_weights_past_2_31_elements(T, D, V):
    # Refused before, though only the zeros of a batch without tokens were made one element to a thread.
    dev = device()
    say("large weights", T, D, V)
    assert V * D >= 1 << 31
    h, w, t, dl = case(T, D, V, "bf16", dev)
    t[:2] = torch.tensor([V - 1, 0], device=dev)
    plan = fc.XentPlan(T, D, V, "bf16", ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    check_tokens(h, w, t, dl, loss, lse, dh, _ends(T, 4, dev))
    check_vocabulary(h, w, t, dl, lse, dw, torch.cat([_ends(V, 400, dev), t[t != IGN]]).unique())


def test_zeros_past_2_31_elements():
    dev = device()
    D, V = 8200, 262145
    say("no tokens, large weights", D, V)
    plan = fc.XentPlan(0, D, V, "bf16")
    none = torch.empty(0, device=dev)
    out = torch.full((V, D), 7.0, dtype=torch.bfloat16, device=dev)
    dh, dw = plan.backward(none.bfloat16().view(0, D), out, none.long(), none, none, dw=torch.full_like(out, 7.0))
    assert dh.shape == (0, D) and bool((dw == 0).all()) and bool((out == 7).all())


def test_logits_past_2_35():
    # 2^35 logits and more: 2^23 tiles of 64 x 64 were refused.
    dev = device()
    T, D, V = 131073, 8, 262145
    say("many logits", T, D, V)
    h, w, t, dl = case(T, D, V, "bf16", dev)
    plan = fc.XentPlan(T, D, V, "bf16", ignore_index=IGN)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    check_tokens(h, w, t, dl, loss, lse, dh, _ends(T, 30, dev))
    check_vocabulary(h, w, t, dl, lse, dw, _ends(V, 100, dev))
