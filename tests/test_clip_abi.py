"""Norm and clipping of many gradients, no GPU: the oracle's pins, the C ABI's
host checks and the binding's refusals (failing runs return before anything is
enqueued, so the fake device addresses are never dereferenced)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import _abi
from oracle import clip as oc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = (
    _abi.FCONV_OK, _abi.FCONV_ERR_INVALID_ARG, _abi.FCONV_ERR_UNSUPPORTED, _abi.FCONV_ERR_WORKSPACE,
    _abi.FCONV_ERR_MISALIGNED)


@pytest.mark.parametrize("limit", [0.0, 0.1, 3.0, 1e6, math.inf])
def test_oracle_agrees_with_torch(limit):
    rng = np.random.default_rng(0)
    grads = [rng.normal(size=n) for n in (5, 1, 40)]
    params = [torch.zeros(len(g), dtype=torch.float64, requires_grad=True) for g in grads]
    for p, g in zip(params, grads):
        p.grad = torch.from_numpy(g.copy())
    want = torch.nn.utils.clip_grad_norm_(params, limit)
    norm, out = oc.clip(grads, limit)
    assert abs(norm - float(want)) < 1e-12
    for o, p in zip(out, params):
        assert np.allclose(o, p.grad.numpy(), rtol=1e-12, atol=0)


def test_oracle_by_hand():
    norm, out = oc.clip([[3.0], [4.0]], 2.5, eps=0.0)
    assert norm == 5 and out[0][0] == 1.5 and out[1][0] == 2


def test_header_and_exports_agree():
    text = open(os.path.join(ROOT, "include", "fconv_clip.h")).read()
    declared = set(re.findall(r"FCONV_API\s+[\w\s\*]+?\b(fconv_\w+)\s*\(", text))
    assert declared == set(_abi.CLIP_EXPORTS)
    lib = ctypes.CDLL(_abi.lib_path())
    for name in declared:
        assert hasattr(lib, name), name


def _create(tensors, eps=1e-6, n=None):
    d = (_abi.ClipTensor * max(1, len(tensors)))()
    for x, (numel, dtype) in zip(d, tensors):
        x.numel, x.dtype = numel, dtype
    h = ctypes.c_void_p()
    return _abi.clip_lib().fconv_clip_plan_create(d, len(tensors) if n is None else n, eps, ctypes.byref(h)), h


def test_plan_refuses():
    L = _abi.clip_lib()
    for tensors, eps, n in (([(4, 1)], -1.0, None), ([(4, 1)], math.nan, None), ([(4, 1)], math.inf, None),
                            ([(-1, 1)], 0.0, None), ([(4, 1)], 0.0, -1)):
        assert _create(tensors, eps, n)[0] == INVALID
    for tensors in ([(4, 0)], [(4, 7)], [((1 << 40) + 1, 1)], [(1 << 40, 2)] * 9):
        assert _create(tensors)[0] == UNSUPPORTED
    assert _create([(4, 1)], n=(1 << 20) + 1)[0] == UNSUPPORTED
    assert L.fconv_clip_plan_create(None, 1, 0.0, None) == INVALID
    for fn in (L.fconv_clip_plan_norm, L.fconv_clip_plan_clip):
        assert fn(None, None, None) == INVALID
    assert L.fconv_clip_plan_workspace_size(None, None) == INVALID
    assert L.fconv_clip_plan_tensors(None, None, None) == INVALID
    assert L.fconv_clip_plan_destroy(None) == OK


def test_plan_keeps_its_tensors():
    L = _abi.clip_lib()
    st, h = _create([(4, 1), (0, 2), (1 << 33, 2)])
    assert st == OK
    t, n = ctypes.POINTER(_abi.ClipTensor)(), ctypes.c_int32()
    assert L.fconv_clip_plan_tensors(h, ctypes.byref(t), ctypes.byref(n)) == OK
    assert [(t[i].numel, t[i].dtype) for i in range(n.value)] == [(4, 1), (0, 2), (1 << 33, 2)]
    L.fconv_clip_plan_destroy(h)


@pytest.mark.parametrize("extra", [0, 400])
def test_runs_refuse(extra):
    # With 400 more tensors the ranges no longer fit what the call keeps on its stack.
    L = _abi.clip_lib()
    tensors = [(1000, 1), (0, 2), (2000, 2)] + [(8, 2)] * extra
    st, h = _create(tensors)
    assert st == OK
    size = ctypes.c_size_t()
    assert L.fconv_clip_plan_workspace_size(h, ctypes.byref(size)) == OK
    more = [64 * M + 1024 * i for i in range(extra)]

    def run(fn, first=M, second=3 * M, out=None, **kw):
        n = len(tensors)
        a = _abi.ClipArgs()
        a.in_ = (ctypes.c_void_p * n)(first, None, second, *more)
        a.out = (ctypes.c_void_p * n)(*((first, None, second) if out is None else out), *more)
        for k, v in dict(dict(max_norm=1.0, norm=40 * M, workspace=41 * M, workspace_bytes=size.value), **kw).items():
            setattr(a, k, v)
        return fn(h, None, ctypes.byref(a))
    norm, clip = L.fconv_clip_plan_norm, L.fconv_clip_plan_clip
    for fn in (norm, clip):
        for kw in (dict(first=None), dict(second=None), dict(norm=None), dict(in_=None), dict(norm=M + 4), dict(workspace=3 * M),
                   dict(norm=41 * M)):
            assert run(fn, **kw) == INVALID, kw
        for kw in (dict(first=M + 1), dict(second=3 * M + 2), dict(norm=40 * M + 2), dict(workspace=41 * M + 8)):
            assert run(fn, **kw) == MISALIGNED, kw
        assert run(fn, workspace=None) == WORKSPACE and run(fn, workspace_bytes=size.value - 1) == WORKSPACE
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(out=(M, None, None)), dict(out=(M + 2, None, 3 * M)),
               dict(out=(3 * M, None, 5 * M)), dict(out=(5 * M, None, 5 * M)), dict(out=(M, None, 3 * M + 8)),
               dict(out=(40 * M, None, 3 * M)), dict(out=None, second=M + 1000), dict(given_norm=M, norm=None),
               dict(given_norm=3 * M, norm=None)):
        assert run(clip, **kw) == INVALID, kw
    a = _abi.ClipArgs()
    a.in_ = (ctypes.c_void_p * len(tensors))(M, None, 3 * M, *more)
    a.max_norm, a.norm, a.workspace, a.workspace_bytes = 1.0, 40 * M, 41 * M, size.value
    assert clip(h, None, ctypes.byref(a)) == INVALID  # nowhere to write
    assert run(clip, given_norm=40 * M + 2) == MISALIGNED
    assert L.fconv_clip_plan_destroy(h) == OK


def test_the_same_tensor_twice_is_refused():
    # A tied parameter's gradient would be scaled twice.
    L = _abi.clip_lib()
    st, h = _create([(8, 2), (8, 2)])
    a = _abi.ClipArgs()
    a.in_ = a.out = (ctypes.c_void_p * 2)(M, M)
    a.max_norm, a.norm, a.workspace, a.workspace_bytes = 1.0, 40 * M, 41 * M, 1 << 16
    assert st == OK and L.fconv_clip_plan_clip(h, None, ctypes.byref(a)) == INVALID
    L.fconv_clip_plan_destroy(h)


def test_binding_refuses():
    c = fc.ClipPlan([(12, "fp32"), (5, "bf16")], eps=0.0)
    x, y = torch.zeros(3, 4), torch.zeros(5).bfloat16()
    with pytest.raises(ValueError, match=r"grads\[0\]: dtype"):
        c.norm([x.double(), y])
    with pytest.raises(ValueError, match=r"grads\[0\]: 6 elements"):
        c.norm([torch.zeros(6), y])
    with pytest.raises(ValueError, match="1 tensors, the plan needs 2"):
        c.clip([x], 1.0)
    with pytest.raises(ValueError, match="one after another"):
        c.clip([torch.zeros(3, 8)[:, ::2], y], 1.0)
    with pytest.raises(ValueError, match="one after another"):
        c.clip([torch.zeros(1).expand(12), y], 1.0)
    with pytest.raises(ValueError, match="GPU"):
        c.clip([x, y], 1.0)
    for bad in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            c.clip([x, y], bad)
    with pytest.raises(ValueError, match="no gradients"):
        fc.ClipPlan([])
    with pytest.raises(ValueError, match="dtype"):
        fc.ClipPlan([(4, "fp16")])
    with pytest.raises(fc.FconvError):
        fc.ClipPlan([(-1, "fp32")])
    with pytest.raises(fc.FconvError):
        fc.ClipPlan([(1, "int8")])
    with pytest.raises(fc.FconvError):
        fc.ClipPlan([(1, "fp32")], eps=-1.0)
