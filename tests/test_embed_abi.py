"""Embedding lookup, no GPU: the oracle's pins, the C ABI's host checks and the
binding's refusals (failing runs return before anything is enqueued, so the fake
device addresses are never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi
from oracle import embed as oe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = (
    _abi.FCONV_OK, _abi.FCONV_ERR_INVALID_ARG, _abi.FCONV_ERR_UNSUPPORTED, _abi.FCONV_ERR_WORKSPACE,
    _abi.FCONV_ERR_MISALIGNED)


def test_oracle_agrees_with_autograd():
    rng = np.random.default_rng(0)
    T, D, V = 30, 5, 7
    w, dy, token = rng.normal(size=(V, D)), rng.normal(size=(T, D)), rng.integers(0, V, T)
    wt = torch.from_numpy(w).requires_grad_()
    yt = 0.5 * torch.nn.functional.embedding(torch.from_numpy(token), wt)
    yt.backward(torch.from_numpy(dy))
    assert np.allclose(oe.forward(w, token, 0.5), yt.detach().numpy(), rtol=1e-15)
    assert np.allclose(oe.backward(token, dy, V, 0.5), wt.grad.numpy(), rtol=1e-13, atol=1e-13)


def test_oracle_by_hand():
    token = np.array([2, -100, 2, 9])
    y = oe.forward([[1.0], [2.0], [3.0]], token, 2.0)
    assert y[0, 0] == y[2, 0] == 6 and y[1, 0] == 0 and np.isnan(y[3, 0])
    assert np.array_equal(oe.backward(token, [[1.0], [8.0], [4.0], [16.0]], 3, 2.0), [[0.0], [0.0], [10.0]])


def test_header_and_exports_agree():
    text = open(os.path.join(ROOT, "include", "fconv_embed.h")).read()
    declared = set(re.findall(r"FCONV_API\s+[\w\s\*]+?\b(fconv_\w+)\s*\(", text))
    assert declared == set(_abi.EMBED_EXPORTS)
    lib = ctypes.CDLL(_abi.lib_path())
    for name in declared:
        assert hasattr(lib, name), name


def _create(**kw):
    d = _abi.EmbedDesc()
    for k, v in dict(dict(T=4, D=64, V=100, dtype=1, ignore_index=-100, scale=1.0, flags=0), **kw).items():
        setattr(d, k, v)
    h = ctypes.c_void_p()
    return _abi.embed_lib().fconv_embed_plan_create(ctypes.byref(d), ctypes.byref(h)), h


def test_plan_refuses():
    L = _abi.embed_lib()
    for kw in (dict(T=-1), dict(D=0), dict(V=0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _create(**kw)[0] == INVALID, kw
    for kw in (dict(dtype=0), dict(dtype=5), dict(flags=1), dict(D=(1 << 20) + 1), dict(T=4194241), dict(V=(1 << 24) + 1),
               dict(T=1 << 20, D=1 << 14), dict(V=1 << 20, D=1 << 14)):
        assert _create(**kw)[0] == UNSUPPORTED, kw
    assert L.fconv_embed_plan_create(None, None) == INVALID
    assert L.fconv_embed_plan_workspace_size(None, None) == INVALID
    assert L.fconv_embed_plan_forward(None, None, None) == INVALID
    assert L.fconv_embed_plan_backward(None, None, None) == INVALID
    assert L.fconv_embed_plan_destroy(None) == OK


@pytest.mark.parametrize("T", [40, 400, 5000])
def test_runs_refuse(T):
    L = _abi.embed_lib()
    st, h = _create(T=T, D=96, V=200)
    assert st == OK
    n = ctypes.c_size_t()
    assert L.fconv_embed_plan_workspace_size(h, ctypes.byref(n)) == OK
    base = dict(token=FAKE, w=4 * FAKE, ldw=96, y=8 * FAKE, ldy=96, dy=12 * FAKE, lddy=96, dw=16 * FAKE, lddw=96,
                workspace=32 * FAKE, workspace_bytes=n.value)

    def run(fn, **kw):
        a = _abi.EmbedArgs()
        for k, v in dict(base, **kw).items():
            setattr(a, k, v)
        return fn(h, None, ctypes.byref(a))
    fwd, bwd = L.fconv_embed_plan_forward, L.fconv_embed_plan_backward
    for kw in (dict(token=None), dict(w=None), dict(y=None), dict(ldw=95), dict(ldy=95), dict(ldw=(1 << 21) + 1), dict(y=FAKE),
               dict(y=4 * FAKE), dict(run_flags=1)):
        assert run(fwd, **kw) == INVALID, kw
    for kw in (dict(token=None), dict(dy=None), dict(dw=None), dict(lddy=95), dict(lddw=95), dict(lddw=(1 << 21) + 1),
               dict(dw=FAKE), dict(dw=12 * FAKE), dict(run_flags=2)):
        assert run(bwd, **kw) == INVALID, kw
    for kw in (dict(token=FAKE + 4), dict(w=4 * FAKE + 1), dict(y=8 * FAKE + 1)):
        assert run(fwd, **kw) == MISALIGNED, kw
    for kw in (dict(token=FAKE + 4), dict(dy=12 * FAKE + 1), dict(dw=16 * FAKE + 1), dict(workspace=32 * FAKE + 8)):
        assert run(bwd, **kw) == MISALIGNED, kw
    if n.value:
        assert run(bwd, workspace=None) == WORKSPACE and run(bwd, workspace_bytes=n.value - 1) == WORKSPACE
        for kw in (dict(workspace=FAKE), dict(workspace=12 * FAKE), dict(workspace=16 * FAKE)):
            assert run(bwd, **kw) == INVALID, kw
    else:
        assert T == 40  # sorted by each workgroup itself
    assert L.fconv_embed_plan_destroy(h) == OK


def test_no_tokens_is_a_no_op():
    L = _abi.embed_lib()
    st, h = _create(T=0)
    a = _abi.EmbedArgs()
    assert st == OK and L.fconv_embed_plan_forward(h, None, ctypes.byref(a)) == OK
    assert L.fconv_embed_plan_backward(h, None, ctypes.byref(a)) == INVALID  # no output
    a.dw, a.lddw, a.run_flags = FAKE, 64, _abi.FCONV_EMBED_ADD  # nothing to add
    assert L.fconv_embed_plan_backward(h, None, ctypes.byref(a)) == OK
    L.fconv_embed_plan_destroy(h)


@pytest.mark.parametrize("T,D,V", [(300, 64, 1000), (16384, 4096, 65536), (1000000, 1024, 1000), (4194240, 8, 1 << 24)])
def test_workspace_is_linear_in_the_tokens(T, D, V):
    # Keys twice, and two fp32 sums for each piece of at least sixteen of them.
    assert fc.EmbedPlan(T, D, V).workspace_bytes <= 16 * T + 512 + (T + 15) // 16 * 8 * (D + 8)


def test_binding_refuses():
    c = fc.EmbedPlan(4, 40, 9, "fp32", scale=0.1)
    assert c.scale == np.float32(0.1)
    w, t, dy = torch.zeros(9, 40), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 40)
    with pytest.raises(ValueError, match="w: dtype"):
        c.forward(w.bfloat16(), t)
    with pytest.raises(ValueError, match="token: dtype"):
        c.backward(t.int(), dy)
    with pytest.raises(ValueError, match="token: 3 elements"):
        c.backward(t[:3], dy)
    with pytest.raises(ValueError, match="w: shape"):
        c.forward(w[:8], t)
    with pytest.raises(ValueError, match="GPU"):
        c.forward(w, t)
    with pytest.raises(ValueError, match="accumulate"):
        c.backward(t, dy, accumulate=True)
    with pytest.raises(ValueError, match="dtype"):
        fc.EmbedPlan(4, 40, 9, "fp16")
    with pytest.raises(ValueError, match="32 bits"):
        fc.EmbedPlan(4, 40, (1 << 32) + 1)
    with pytest.raises(ValueError, match="64 bits"):
        fc.EmbedPlan(4, 40, 9, ignore_index=1 << 63)
    for scale in (float("nan"), float("inf"), 1e39):
        with pytest.raises(fc.FconvError):
            fc.EmbedPlan(4, 40, 9, scale=scale)
    with pytest.raises(fc.FconvError):
        fc.EmbedPlan(4, 40, 9, "int8")

