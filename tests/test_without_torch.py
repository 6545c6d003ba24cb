"""The convolution plans work where torch is not installed: the package is
imported, built and used with raw addresses in a child process whose imports
of torch fail."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NO_TORCH = "import sys; sys.path.insert(0, %r); sys.modules['torch'] = None\n" % ROOT


def _child(code, **env):
    r = subprocess.run([sys.executable, "-c", NO_TORCH + code], env=dict(os.environ, **env), capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    return r


def test_convolution_plans_are_created_and_run():
    # A stream of 0 and addresses as ints; the run's arguments are wrong, so nothing is enqueued.
    _child("""
import convolution_implicit_gemm_nhwc_amd as fc
from convolution_implicit_gemm_nhwc_amd import *
p = Plan(2, 6, 5, 16, 24, 3, 3, 1, "SAME", "int8", ops=("scale", "bias"))
a = p.make_args(1 << 20, 2 << 20, 3 << 20, None, bias=4 << 20, workspace_bytes=0)
a.y = None
assert p.run_args(a, stream=0) == fc._abi.FCONV_ERR_INVALID_ARG
g = WgradPlan(2, 6, 5, 16, 24, 3, 3, 1, "SAME", "bf16")
assert g.run_raw(1 << 20, 2 << 20, None, 3 << 20, stream=0) == fc._abi.FCONV_ERR_INVALID_ARG
""")


@pytest.mark.parametrize("name", ["MxTensor", "MxQuantPlan", "MxPlan", "XentPlan"])
def test_plans_of_torch_tensors_say_what_is_missing(name):
    _child("""
import convolution_implicit_gemm_nhwc_amd as fc
assert %r in dir(fc)
try:
    fc.%s
except ModuleNotFoundError as e:
    assert "torch" in str(e)
else:
    raise AssertionError("found without torch")
""" % (name, name))


def test_with_torch_all_names_are_there():
    code = """
import sys; sys.path.insert(0, %r)
import convolution_implicit_gemm_nhwc_amd as fc
assert "torch" not in sys.modules
from convolution_implicit_gemm_nhwc_amd import *
for name in ("Plan", "WgradPlan", "MxTensor", "MxQuantPlan", "MxPlan", "XentPlan"):
    assert globals()[name] is getattr(fc, name), name
try:
    fc.nothing
except AttributeError:
    pass
else:
    raise AssertionError
""" % ROOT
    subprocess.run([sys.executable, "-c", code], check=True, timeout=120)


def test_library_is_built(tmp_path):
    # A compiler that only leaves its output file stands for hipcc.
    cc = tmp_path / "cc"
    cc.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho built > "$2"\n')
    cc.chmod(0o755)
    (tmp_path / "_call.so").write_text("of other sources")
    _child("""
from convolution_implicit_gemm_nhwc_amd import build as b
b.CSRC, b.LIB, b.CALL = (%r + x for x in ("", "/libfconv.so", "/_call.so"))
b.build()
""" % str(tmp_path), HIPCC=str(cc))
    assert sorted(os.listdir(tmp_path)) == ["cc", "libfconv.so"]
