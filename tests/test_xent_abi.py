"""Linear softmax cross entropy, no GPU: the oracle's pins, the C ABI's host
checks and the binding's refusals (failing runs return before anything is
enqueued, so the fake device addresses are never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi
from oracle import xent as ox

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = (
    _abi.FCONV_OK, _abi.FCONV_ERR_INVALID_ARG, _abi.FCONV_ERR_UNSUPPORTED, _abi.FCONV_ERR_WORKSPACE,
    _abi.FCONV_ERR_MISALIGNED)


# --- the oracle -----------------------------------------------------------

def test_oracle_agrees_with_autograd():
    rng = np.random.default_rng(0)
    T, D, V = 7, 5, 11
    h, w, dl = rng.normal(size=(T, D)), rng.normal(size=(V, D)), rng.normal(size=T)
    t = rng.integers(0, V, T)
    t[2] = -100
    ht, wt = torch.from_numpy(h).requires_grad_(), torch.from_numpy(w).requires_grad_()
    loss = torch.nn.functional.cross_entropy(ht @ wt.t(), torch.from_numpy(t), reduction="none")
    loss.backward(torch.from_numpy(dl))
    ol, lse, _ = ox.forward(h, w, t)
    dh, dw, _ = ox.backward(h, w, t, lse, dl)
    assert np.allclose(ol, loss.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dh, ht.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(1)
    T, D, V = 5, 6, 9
    h, w, dl = rng.normal(size=(T, D)), rng.normal(size=(V, D)), rng.normal(size=T)
    t = rng.integers(0, V, T)
    _, lse, _ = ox.forward(h, w, t)
    dh, dw, _ = ox.backward(h, w, t, lse, dl)
    uh, uw, e = rng.normal(size=h.shape), rng.normal(size=w.shape), 1e-5
    for a, b, got in ((uh, 0 * uw, (dh * uh).sum()), (0 * uh, uw, (dw * uw).sum())):
        lp, lm = ox.forward(h + e * a, w + e * b, t)[0], ox.forward(h - e * a, w - e * b, t)[0]
        assert abs(((lp - lm) * dl).sum() / (2 * e) - got) < 1e-7


def test_oracle_by_hand():
    # Two classes, equal logits: loss log 2, gradient +-1/2.
    h, w = np.array([[1.0]]), np.zeros((2, 1))
    loss, lse, _ = ox.forward(h, w, np.array([0]))
    assert loss[0] == lse[0] == np.log(2.0)
    _, dw, g = ox.backward(h, w, np.array([0]), lse, np.array([4.0]))
    assert np.allclose(g, [[-2, 2]], rtol=1e-15) and np.allclose(dw, [[-2], [2]], rtol=1e-15)
    assert ox.forward(h, w, np.array([-100]))[0][0] == 0
    assert np.isnan(ox.forward(h, w, np.array([2]))[0][0])


# --- the C ABI ------------------------------------------------------------

def test_header_and_exports_agree():
    text = open(os.path.join(ROOT, "include", "fconv_xent.h")).read()
    declared = set(re.findall(r"FCONV_API\s+[\w\s\*]+?\b(fconv_\w+)\s*\(", text))
    assert declared == set(_abi.XENT_EXPORTS)
    lib = ctypes.CDLL(_abi.lib_path())
    for name in declared:
        assert hasattr(lib, name), name


def _create(**kw):
    d = _abi.XentDesc()
    for k, v in dict(dict(T=4, D=64, V=100, dtype=1, ignore_index=-100, flags=0), **kw).items():
        setattr(d, k, v)
    h = ctypes.c_void_p()
    return _abi.xent_lib().fconv_xent_plan_create(ctypes.byref(d), ctypes.byref(h)), h


def _sizes(h):
    L, f, b = _abi.xent_lib(), ctypes.c_size_t(), ctypes.c_size_t()
    assert L.fconv_xent_plan_forward_workspace_size(h, ctypes.byref(f)) == OK
    assert L.fconv_xent_plan_backward_workspace_size(h, ctypes.byref(b)) == OK
    return f.value, b.value


def test_plan_refuses():
    L = _abi.xent_lib()
    for kw in (dict(T=-1), dict(D=0), dict(V=0)):
        assert _create(**kw)[0] == INVALID, kw
    for kw in (dict(dtype=0), dict(dtype=5), dict(flags=1), dict(D=(1 << 20) + 1), dict(T=(1 << 24) + 1),
               dict(V=(1 << 24) + 1), dict(T=1 << 24, V=1 << 24)):
        assert _create(**kw)[0] == UNSUPPORTED, kw
    assert L.fconv_xent_plan_create(None, None) == INVALID
    assert L.fconv_xent_plan_forward_workspace_size(None, None) == INVALID
    assert L.fconv_xent_plan_backward_workspace_size(None, None) == INVALID
    assert L.fconv_xent_plan_destroy(None) == OK


@pytest.mark.parametrize("T,D,V", [(1, 64, 500), (8192, 4096, 32768), (100000, 512, 100000)])
def test_workspace_stays_far_below_the_logits(T, D, V):
    st, h = _create(T=T, D=D, V=V)
    assert st == OK
    f, b = _sizes(h)
    _abi.xent_lib().fconv_xent_plan_destroy(h)
    assert f <= T * V // 4 + 4096 * T + (1 << 20)
    # A piece of g, the gathered h, and fp32 sums of dh or dw.
    if T * V > 1 << 28:
        assert b < T * V * 4 * 3 // 4


def _fill(a, base, kw):
    for k, v in dict(base, **kw).items():
        setattr(a, k, v)
    return a


def test_runs_refuse():
    L = _abi.xent_lib()
    st, h = _create(T=40, D=96, V=200)
    assert st == OK
    f, b = _sizes(h)
    base = dict(h=FAKE, ldh=96, w=2 * FAKE, ldw=96, target=3 * FAKE, loss=4 * FAKE, lse=5 * FAKE, dloss=6 * FAKE,
                dh=7 * FAKE, lddh=96, dw=8 * FAKE, lddw=96, workspace=16 * FAKE, workspace_bytes=max(f, b))

    def fwd(**kw):
        return L.fconv_xent_plan_forward(h, None, ctypes.byref(_fill(_abi.XentArgs(), base, kw)))

    def bwd(**kw):
        return L.fconv_xent_plan_backward(h, None, ctypes.byref(_fill(_abi.XentArgs(), base, kw)))
    both = (dict(h=None), dict(w=None), dict(target=None), dict(lse=None), dict(ldh=95), dict(ldw=95),
            dict(ldh=(1 << 21) + 1), dict(ldw=(1 << 21) + 1), dict(workspace=FAKE), dict(workspace=2 * FAKE),
            dict(workspace=3 * FAKE))
    for run, more in ((fwd, (dict(loss=None), dict(loss=FAKE), dict(lse=4 * FAKE), dict(loss=16 * FAKE))),
                      (bwd, (dict(dloss=None), dict(dh=None, dw=None), dict(lddh=95), dict(lddw=95),
                             dict(dh=FAKE), dict(dh=2 * FAKE), dict(dw=5 * FAKE), dict(dw=7 * FAKE),
                             dict(dh=16 * FAKE), dict(lddh=(1 << 21) + 1)))):
        for kw in both + more:
            assert run(**kw) == INVALID, kw
        for kw in (dict(h=FAKE + 1), dict(w=2 * FAKE + 1), dict(target=3 * FAKE + 4), dict(lse=5 * FAKE + 2),
                   dict(workspace=16 * FAKE + 8)):
            assert run(**kw) == MISALIGNED, kw
        assert run(workspace=None) == WORKSPACE
        assert run(workspace_bytes=(f if run is fwd else b) - 1) == WORKSPACE
    assert fwd(loss=4 * FAKE + 2) == MISALIGNED
    assert bwd(dh=7 * FAKE + 1) == MISALIGNED
    assert bwd(dw=8 * FAKE + 1) == MISALIGNED
    assert bwd(dloss=6 * FAKE + 2) == MISALIGNED
    assert L.fconv_xent_plan_forward(None, None, None) == INVALID
    assert L.fconv_xent_plan_backward(None, None, None) == INVALID
    assert L.fconv_xent_plan_destroy(h) == OK


def test_no_tokens_is_a_no_op():
    L = _abi.xent_lib()
    st, h = _create(T=0)
    assert st == OK
    a = _abi.XentArgs()
    assert L.fconv_xent_plan_forward(h, None, ctypes.byref(a)) == OK
    assert L.fconv_xent_plan_backward(h, None, ctypes.byref(a)) == INVALID  # no output
    a.dh, a.lddh = FAKE, 64  # dh of no tokens: nothing to write
    assert L.fconv_xent_plan_backward(h, None, ctypes.byref(a)) == OK
    L.fconv_xent_plan_destroy(h)


# --- the binding ----------------------------------------------------------

def test_binding_refuses():
    c = fc.XentPlan(4, 40, 9, "fp32")
    h, w, t = torch.zeros(4, 40), torch.zeros(9, 40), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="h: dtype"):
        c.forward(h.bfloat16(), w, t)
    with pytest.raises(ValueError, match="h: shape"):
        c.forward(torch.zeros(4, 41), w, t)
    with pytest.raises(ValueError, match="dense"):
        c.forward(torch.zeros(40, 4).t(), w, t)
    with pytest.raises(ValueError, match="GPU"):
        c.forward(h, w, t)
    with pytest.raises(ValueError, match="no gradient"):
        c.backward(h, w, t, h[:, 0], h[:, 0], need_dh=False, need_dw=False)
    with pytest.raises(ValueError, match="not needed"):
        c.backward(h, w, t, h[:, 0], h[:, 0], dh=h, need_dh=False)
    with pytest.raises(fc.FconvError):
        fc.XentPlan(4, 40, 9, "int8")
    with pytest.raises(fc.FconvError):
        fc.XentPlan(4, 0, 9)
