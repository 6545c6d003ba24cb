"""Gated feed-forward layer, no GPU: the oracle's pins, the C ABI's host checks
and the binding's refusals (failing runs return before anything is enqueued, so
the fake device addresses are never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi
from oracle import gated as og

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = (
    _abi.FCONV_OK, _abi.FCONV_ERR_INVALID_ARG, _abi.FCONV_ERR_UNSUPPORTED, _abi.FCONV_ERR_WORKSPACE,
    _abi.FCONV_ERR_MISALIGNED)

TORCH_ACT = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh"), "relu": torch.relu}


@pytest.mark.parametrize("name", _abi.ACTIVATIONS)
def test_oracle_agrees_with_autograd(name):
    rng = np.random.default_rng(0)
    T, D, F = 7, 5, 11
    x, w, dy = rng.normal(size=(T, D)), rng.normal(size=(2 * F, D)), rng.normal(size=(T, F))
    xt, wt = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    yt = TORCH_ACT[name](xt @ wt[:F].t()) * (xt @ wt[F:].t())
    yt.backward(torch.from_numpy(dy))
    y, g, u = og.forward(x, w, name)
    dx, dw, _ = og.backward(x, w, g, u, dy, name)
    for got, want in ((y, yt.detach()), (dx, xt.grad), (dw, wt.grad)):
        assert np.allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("name", _abi.ACTIVATIONS)
def test_oracle_gradient_against_differences(name):
    rng = np.random.default_rng(1)
    T, D, F, e = 5, 6, 4, 1e-5
    x, w, dy = rng.normal(size=(T, D)), rng.normal(size=(2 * F, D)), rng.normal(size=(T, F))
    _, g, u = og.forward(x, w, name)
    dx, dw, _ = og.backward(x, w, g, u, dy, name)
    ux, uw = rng.normal(size=x.shape), rng.normal(size=w.shape)
    for a, b, got in ((ux, 0 * uw, (dx * ux).sum()), (0 * ux, uw, (dw * uw).sum())):
        up, down = og.forward(x + e * a, w + e * b, name)[0], og.forward(x - e * a, w - e * b, name)[0]
        assert abs(((up - down) * dy).sum() / (2 * e) - got) < 1e-6


def test_oracle_by_hand():
    # One gate of 0: silu(0) = 0 with slope 1/2; one projection of 3.
    y, g, u = og.forward([[1.0]], [[0.0], [3.0]], "silu")
    assert y[0, 0] == 0 and g[0, 0] == 0 and u[0, 0] == 3
    dx, dw, dz = og.backward([[1.0]], [[0.0], [3.0]], g, u, [[2.0]], "silu")
    assert np.array_equal(dz, [[3.0, 0.0]]) and np.array_equal(dw, [[3.0], [0.0]]) and dx[0, 0] == 0


def test_header_and_exports_agree():
    text = open(os.path.join(ROOT, "include", "fconv_gated.h")).read()
    declared = set(re.findall(r"FCONV_API\s+[\w\s\*]+?\b(fconv_\w+)\s*\(", text))
    assert declared == set(_abi.GATED_EXPORTS)
    lib = ctypes.CDLL(_abi.lib_path())
    for name in declared:
        assert hasattr(lib, name), name


def _create(**kw):
    d = _abi.GatedDesc()
    for k, v in dict(dict(T=4, D=64, F=100, dtype=1, activation=0, flags=0), **kw).items():
        setattr(d, k, v)
    h = ctypes.c_void_p()
    return _abi.gated_lib().fconv_gated_plan_create(ctypes.byref(d), ctypes.byref(h)), h


def _size(h, what):
    n = ctypes.c_size_t()
    assert getattr(_abi.gated_lib(), "fconv_gated_plan_%s_size" % what)(h, ctypes.byref(n)) == OK
    return n.value


def test_plan_refuses():
    L = _abi.gated_lib()
    for kw in (dict(T=-1), dict(D=0), dict(F=0)):
        assert _create(**kw)[0] == INVALID, kw
    for kw in (dict(dtype=0), dict(dtype=5), dict(activation=4), dict(activation=-1), dict(flags=1), dict(D=(1 << 20) + 1),
               dict(F=(1 << 20) + 1), dict(T=4194241), dict(T=1 << 20, D=1 << 14), dict(T=1 << 20, F=1 << 13),
               dict(D=1 << 17, F=1 << 16)):
        assert _create(**kw)[0] == UNSUPPORTED, kw
    assert L.fconv_gated_plan_create(None, None) == INVALID
    for what in ("kept", "forward_workspace", "backward_workspace"):
        assert getattr(L, "fconv_gated_plan_%s_size" % what)(None, None) == INVALID
    assert L.fconv_gated_plan_forward(None, None, None) == INVALID
    assert L.fconv_gated_plan_backward(None, None, None) == INVALID
    assert L.fconv_gated_plan_kernel_name(None, 0) is None
    assert L.fconv_gated_plan_ranges(None, 0, None) == INVALID
    assert L.fconv_gated_plan_destroy(None) == OK


def _fill(base, kw):
    a = _abi.GatedArgs()
    for k, v in dict(base, **kw).items():
        setattr(a, k, v)
    return a


def test_runs_refuse():
    L = _abi.gated_lib()
    st, h = _create(T=40, D=96, F=200)
    assert st == OK
    b = _size(h, "backward_workspace")
    base = dict(x=FAKE, ldx=96, w=2 * FAKE, ldw=96, y=4 * FAKE, ldy=200, kept=6 * FAKE, dy=8 * FAKE, lddy=200,
                dx=10 * FAKE, lddx=96, dw=12 * FAKE, lddw=96, workspace=16 * FAKE, workspace_bytes=b)

    def fwd(**kw):
        return L.fconv_gated_plan_forward(h, None, ctypes.byref(_fill(base, kw)))

    def bwd(**kw):
        return L.fconv_gated_plan_backward(h, None, ctypes.byref(_fill(base, kw)))
    both = (dict(x=None), dict(w=None), dict(ldx=95), dict(ldw=95), dict(ldx=(1 << 21) + 1), dict(ldw=(1 << 21) + 1))
    for kw in both + (dict(y=None), dict(ldy=199), dict(ldy=(1 << 21) + 1), dict(y=FAKE), dict(y=2 * FAKE), dict(kept=FAKE),
                      dict(kept=4 * FAKE)):
        assert fwd(**kw) == INVALID, kw
    for kw in both + (dict(kept=None), dict(dy=None), dict(dx=None, dw=None), dict(lddy=199), dict(lddx=95), dict(lddw=95),
                      dict(dx=FAKE), dict(dw=2 * FAKE), dict(dx=8 * FAKE), dict(dw=6 * FAKE), dict(dx=12 * FAKE),
                      dict(dw=16 * FAKE), dict(workspace=FAKE), dict(workspace=8 * FAKE)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 1), dict(w=2 * FAKE + 1), dict(kept=6 * FAKE + 8)):
        assert fwd(**kw) == MISALIGNED and bwd(**kw) == MISALIGNED, kw
    assert fwd(y=4 * FAKE + 1) == MISALIGNED
    for kw in (dict(dy=8 * FAKE + 1), dict(dx=10 * FAKE + 1), dict(dw=12 * FAKE + 1), dict(workspace=16 * FAKE + 8)):
        assert bwd(**kw) == MISALIGNED, kw
    assert bwd(workspace=None) == WORKSPACE and bwd(workspace_bytes=b - 1) == WORKSPACE
    assert L.fconv_gated_plan_destroy(h) == OK


def test_no_tokens_is_a_no_op():
    L = _abi.gated_lib()
    st, h = _create(T=0)
    assert st == OK and _size(h, "kept") == 0
    a = _abi.GatedArgs()
    assert L.fconv_gated_plan_forward(h, None, ctypes.byref(a)) == OK
    assert L.fconv_gated_plan_backward(h, None, ctypes.byref(a)) == INVALID  # no output
    a.dx, a.lddx = FAKE, 64  # dx of no tokens: nothing to write
    assert L.fconv_gated_plan_backward(h, None, ctypes.byref(a)) == OK
    assert L.fconv_gated_plan_kernel_name(h, 0) is None
    L.fconv_gated_plan_destroy(h)


@pytest.mark.parametrize("T,D,F", [(1, 4096, 12288), (8192, 4096, 12288), (65536, 4096, 12288), (1999, 1000, 2731),
                                   (64, 1000, 200000), (100000, 1001, 77)])
@pytest.mark.parametrize("dtype,es", [("bf16", 2), ("fp32", 4)])
def test_memory_is_linear_in_the_operands(T, D, F, dtype, es):
    p = fc.GatedPlan(T, D, F, dtype)
    assert 8 * T * F <= p.kept_bytes <= 8 * T * (F + 7)
    pack = es * (2 * F + T) * (D + 8) if D % 8 else 0
    assert p.forward_workspace_bytes <= pack + 1024
    # [dg du], packed operands, the ranges' partial sums.
    x = es * T * (D + 8)
    assert p.backward_workspace_bytes <= es * T * (2 * F + 64) + pack + x + 2 * (512 << 20) + 8192


def test_kernels_by_size():
    def names(T, D, F, dtype="bf16"):
        p = fc.GatedPlan(T, D, F, dtype)
        return tuple(p.kernel_name(n) for n in ("forward", "dx", "dw"))
    assert names(1, 4096, 12288)[0] == "gated_few"
    assert names(8192, 4096, 8192) == ("gemm_tile_256",) * 3
    assert names(20, 64, 100) == ("gated_few", "gated_few_grads", "gemm_gen_64")
    assert names(2458, 623, 1344)[0] == "gemm_tile_128_packed"
    assert set(names(2048, 1024, 2816, "fp32")) == {"gemm_gen_64"}
    with pytest.raises(ValueError):
        fc.GatedPlan(4, 4, 4).kernel_name("dy")


def test_binding_refuses():
    c = fc.GatedPlan(4, 40, 9, "fp32")
    x, w, dy, kept = torch.zeros(4, 40), torch.zeros(18, 40), torch.zeros(4, 9), torch.zeros(c.kept_bytes // 4)
    with pytest.raises(ValueError, match="x: dtype"):
        c.forward(x.bfloat16(), w)
    with pytest.raises(ValueError, match="x: shape"):
        c.forward(x[:3], w)
    with pytest.raises(ValueError, match="dense"):
        c.forward(torch.zeros(40, 4).t(), w)
    with pytest.raises(ValueError, match="GPU"):
        c.forward(x, w)
    with pytest.raises(ValueError, match="no gradient"):
        c.backward(x, w, kept, dy, need_dx=False, need_dw=False)
    with pytest.raises(ValueError, match="not needed"):
        c.backward(x, w, kept, dy, dw=w, need_dw=False)
    with pytest.raises(ValueError, match="activation"):
        fc.GatedPlan(4, 40, 9, activation="tanh")
    with pytest.raises(ValueError, match="dtype"):
        fc.GatedPlan(4, 40, 9, "fp16")
    with pytest.raises(ValueError, match="32 bits"):
        fc.GatedPlan(4, 40, (1 << 32) + 1)
    with pytest.raises(fc.FconvError):
        fc.GatedPlan(4, 40, 9, "int8")
    with pytest.raises(fc.FconvError):
        fc.GatedPlan(4, 0, 9)
