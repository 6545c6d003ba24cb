"""What the gated layer's calls launch (CPU only): the library is loaded by a
small program that defines the HIP runtime's entry points itself, so that every
launch is written down, with its kernel's name, grid and operands, and none is
made.  Addresses are numbers that nothing reads."""
import os
import re
import shutil
import subprocess

import pytest

import convolution_implicit_gemm_nhwc_amd as fc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "convolution_implicit_gemm_nhwc_amd", "libfconv.so")

PROGRAM = r"""
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>

#include "fconv_gated.h"

struct Dim { uint32_t x, y, z; };
static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static Dim grid_, block_;

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* h; return &h; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  names()[host] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim grid, Dim block, size_t, void*) { grid_ = grid; block_ = block; return 0; }
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* shared, void** stream) {
  *grid = grid_; *block = block_; *shared = 0; *stream = nullptr;
  return 0;
}
int hipGetLastError() { return 0; }
int hipLaunchKernel(const void* f, Dim grid, Dim block, void** args, size_t, void*) {
  const std::string& n = names()[f];
  printf("%s %u %u %u %u", n.c_str(), grid.x, grid.y, grid.z, block.x);
  // The first operand of each product: address and row distance.
  const bool pair = n.find("gemm_tile_pair") != std::string::npos || n.find("grads_kernel") != std::string::npos;
  if (n.find("gemm_") != std::string::npos || pair)
    for (int i = 0; i < (pair ? 2 : 1); ++i) {
      uint64_t a[2];
      memcpy(a, args[i], 16);
      printf(" %llx %llu", (unsigned long long)a[0], (unsigned long long)a[1]);
    }
  printf("\n");
  return 0;
}
}

template <typename F> static F sym(void* lib, const char* name) {
  void* p = dlsym(lib, name);
  if (!p) { fprintf(stderr, "%s\n", name); exit(2); }
  return reinterpret_cast<F>(p);
}
#define SYM(f) auto f##_ = sym<decltype(&f)>(lib, #f)

int main(int, char** argv) {
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (!lib) { fprintf(stderr, "%s\n", dlerror()); return 2; }
  SYM(fconv_gated_plan_create);
  SYM(fconv_gated_plan_backward_workspace_size);
  SYM(fconv_gated_plan_forward_workspace_size);
  SYM(fconv_gated_plan_forward);
  SYM(fconv_gated_plan_backward);
  SYM(fconv_gated_plan_destroy);
  // T D F dtype, row distances and offsets (elements) of x and w, which: 0 forward, 1 dx, 2 dw, 3 both
  fconv_gated_desc d = {};
  long long ldx, ldw, ox, ow;
  int which;
  while (scanf("%d %d %d %d %lld %lld %lld %lld %d", &d.T, &d.D, &d.F, &d.dtype, &ldx, &ldw, &ox, &ow, &which) == 9) {
    fconv_gated_plan p;
    if (fconv_gated_plan_create_(&d, &p) != FCONV_OK) return 3;
    const int es = d.dtype == FCONV_BF16 ? 2 : 4;
    auto at = [&](uint64_t tib, long long elements) { return reinterpret_cast<char*>((tib << 40) + elements * es); };
    fconv_gated_args a = {};
    a.x = at(1, ox);
    a.ldx = ldx;
    a.w = at(2, ow);
    a.ldw = ldw;
    a.kept = at(3, 0);
    a.dy = at(4, 0);
    a.lddy = d.F;
    a.workspace = at(5, 0);
    if (which) {
      if (which & 1) { a.dx = at(6, 0); a.lddx = d.D; }
      if (which & 2) { a.dw = at(7, 0); a.lddw = d.D; }
    } else {
      a.y = at(8, 0);
      a.ldy = d.F;
    }
    (which ? fconv_gated_plan_backward_workspace_size_ : fconv_gated_plan_forward_workspace_size_)(p, &a.workspace_bytes);
    const size_t bytes = a.workspace_bytes;
    const int st = (which ? fconv_gated_plan_backward_ : fconv_gated_plan_forward_)(p, nullptr, &a);
    printf("status %d %zu\n", st, bytes);
    fconv_gated_plan_destroy_(p);
  }
  return 0;
}
"""

TIB = 1 << 40
X, W, KEPT, DY, WS = (i * TIB for i in range(1, 6))


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """launches(cases): for each case (status, workspace bytes, [(kernel, grid, operands)])."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    at = tmp_path_factory.mktemp("launches")
    src, exe = at / "launches.cpp", at / "launches"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-rdynamic", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    "-ldl"], check=True, capture_output=True)

    def run(cases):
        r = subprocess.run([str(exe), LIB], input="\n".join(" ".join(map(str, c)) for c in cases) + "\n",
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr
        out, now = [], []
        for line in r.stdout.splitlines():
            part = line.split()
            if part[0] == "status":
                out.append((int(part[1]), int(part[2]), now))
                now = []
            else:
                numbers = part[5:]
                operands = [(int(numbers[i], 16), int(numbers[i + 1])) for i in range(0, len(numbers), 2)]
                now.append((part[0], tuple(map(int, part[1:5])), operands))
        assert len(out) == len(cases)
        return out
    return run


def _case(T, D, F, dtype, ldx=None, ldw=None, ox=0, ow=0, which=3):
    return (T, D, F, fc.DTYPES[dtype], ldx or D, ldw or D, ox, ow, which)


@pytest.mark.parametrize("which", [2, 3])
def test_rows_of_no_whole_pieces_are_not_copied_past_their_end(launches, which):
    # The tiles copy whole pieces of 16 bytes.  Of a D that is no multiple of 8 the last row's last piece is not all x,
    # also where x begins and its rows lie on 16 bytes: dw's x is the one in the workspace.
    sizes = [(171, 130, 15352), (1862, 76, 4346), (4332, 41, 9), (2458, 623, 1344), (7127, 130, 4211)]
    seen = 0
    for (T, D, F), (status, bytes, done) in zip(sizes, launches([
            _case(T, D, F, "bf16", ldx=-(-D // 8) * 8, which=which) for T, D, F in sizes])):
        assert status == 0
        tiles = [(name, operands[-1]) for name, _, operands in done if "gemm_tile" in name]
        if not tiles:
            continue
        name, (address, ld) = tiles[-1]  # dw comes last
        seen += 1
        assert WS <= address < WS + bytes and ld % 8 == 0, (T, D, F, name)
    assert seen >= 3


def test_tiles_begin_rows_on_16_bytes(launches):
    # Every operand of a tiled product, whatever the rows that the call is given.
    cases = [_case(T, D, F, "bf16", ldx=D + mx, ldw=D + mw, ox=ox, ow=ow, which=which)
             for T, D, F in ((2048, 1024, 2816), (1999, 1000, 731), (2458, 623, 1344), (171, 130, 15352), (700, 512, 640))
             for mx, mw, ox, ow in ((0, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 4), (8, 8, 8, 8), (3, 5, 1, 7))
             for which in range(4)]
    tiles = 0
    for case, (status, bytes, done) in zip(cases, launches(cases)):
        assert status == 0 and done
        for name, _, operands in done:
            if "gemm_tile" in name:
                tiles += 1
                assert all(address % 16 == 0 and ld % 8 == 0 for address, ld in operands), (case, name)
    assert tiles > 50


def test_few_token_kernel_has_a_workgroup_for_every_token_and_output(launches):
    sizes = [(T, D, F) for T in (1, 8, 9, 16, 17, 32, 33, 48, 64, 65, 128, 271, 1000) for D in (1, 7, 512, 3001, 8192)
             for F in (1, 16, 17, 300, 513, 9000)]
    for dtype in ("bf16", "fp32"):
        cases = [_case(T, D, F, dtype, which=0) for T, D, F in sizes]
        few = 0
        for (T, D, F), (status, _, done) in zip(sizes, launches(cases)):
            assert status == 0
            for name, grid, _ in done:
                m = re.search(r"gated_few_kernelI.*Lb([01])ELi(\d+)ELi(\d+)E", name)
                if not m:
                    continue
                few += 1
                odd, mt, waves = map(int, m.groups())
                assert grid == (-(-(-(-F // 16)) // 8) * 8 * -(-T // (16 * mt)), 1, 1, 64 * waves), (T, D, F, name)
                assert waves >= mt and not (odd and mt > 2)
                assert odd == (dtype == "bf16" and D % 2)
                if T <= 64 and odd == 0 and grid[0] == -(-(-(-F // 16)) // 8) * 8:
                    assert 16 * mt >= T
        assert few > 50
