"""The tiled kernels of the output layer's operators at tiles of 128 and of
256: odd and even numbers of slabs (at least three, so that copies made inside
the loop are used), ragged last tiles, more tiles than workgroups, ranges of the
sum, rows apart, packed rows.  Which kernel a size takes is asserted, and once
more without a GPU by test_tiled_selection.py.

References in 64 bits on the GPU.  Tolerances of the cross entropy: those of
test_gpu_xent_pieces.py.  The product's: 4 u K s with u = 2^-24 and s the root
mean square of an output's products (exact in fp32), the bias's addition, half
a step of bf16."""
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from test_gpu_xent_pieces import IGN, TDT, U, case, check, sum_error

pytestmark = pytest.mark.gpu

# T, D, V; kernel (without "xent_") and ranges > 1 of dh and dw; pieces of w that the forward pass packs.
XENT = [
    ((1025, 264, 8200), "tile_256", "tile_256", ("gen_64", True), ("gen_64", False), 1),     # 5 slabs of logits
    ((2000, 200, 5000), "tile_256", "tile_256", ("tile_128", True), ("tile_128", False), 1),  # 4 slabs
    ((4100, 328, 20011), "tile_256", "tile_256", ("tile_128", True), ("tile_128", False), 1),  # 6; 1343 tiles
    ((3000, 1024, 20000), "tile_256", "tile_256", ("tile_256", True), ("tile_256", False), 1),  # dw past the caches
    ((4097, 1544, 33000), "tile_256", "tile_256", ("tile_256", True), ("tile_256", False), 1),  # 903 tiles of dw
    ((7000, 1288, 5000), "tile_256", "tile_256", ("tile_256", False), ("tile_128", False), 1),  # dh written at once
    ((16000, 2056, 600), "tile_256", "tile_256", ("tile_256", False), ("tile_128", True), 1),
    ((600, 1024, 9000), "tile_128", "tile_128", ("tile_128", True), ("tile_256", False), 1),
    ((1025, 3080, 2100), "tile_128", "tile_128", ("tile_128", False), ("tile_128", False), 1),
    ((700, 1001, 9000), "tile_128_packed", "tile_128_packed", ("tile_128_packed", True), ("tile_256", False), 1),
    ((1999, 257, 9000), "tile_256_packed", "tile_256_packed", ("tile_128_packed", True), ("tile_128", False), 1),
    ((200, 4095, 33000), "tile_256_packed", "tile_256_packed", ("tile_128_packed", True), ("tile_256", False), 2),
    ((300, 4095, 40000), "tile_128_packed", "tile_128_packed", ("tile_256_packed", True), ("tile_256", False), 2),
]
# Sizes of test_gpu_xent_pieces.py: sums added to by every piece, partial sums of dw in tiles of 256.
PIECES = [
    ((20000, 264, 16500), "tile_256", "tile_256", ("tile_128", False), ("tile_128", True), 1),
    ((70001, 600, 9001), "tile_256", "tile_256", ("tile_256", False), ("tile_256", True), 1),
    ((2000, 513, 140001), "tile_256_packed", "tile_256_packed", ("tile_256_packed", True), ("tile_256", False), 1),
]
# M, N, K, kernel, ranges > 1.
MX = [
    ((4090, 4081, 1250), "mx_tile_256", False),   # 5 slabs, 256 tiles
    ((8200, 8200, 1800), "mx_tile_256", False),   # 8 slabs, the last of one k tile; 1089 tiles
    ((8090, 8137, 1700), "mx_tile_256", False),   # 7 slabs, 1024 tiles
    ((2049, 2049, 20000), "mx_tile_256", True),   # ranges of 27 slabs and fewer
    ((4100, 4100, 1300), "mx_tile_128", False),   # 6 slabs, 1089 tiles
    ((3001, 8003, 2300), "mx_tile_128", False),   # 9 slabs
    ((513, 1025, 40000), "mx_tile_128", True),
]


def xent_selection(size):
    plan = fc.XentPlan(*size, "bf16", ignore_index=IGN)
    k = {n: plan.kernel_name(n)[5:] for n in ("logits", "grad", "dh", "dw")}
    return plan, (size, k["logits"], k["grad"], (k["dh"], plan.division("dh")[1] > 1),
                  (k["dw"], plan.division("dw")[1] > 1), plan.division("logits")[0])


def mx_selection(size, dtype):
    M, N, K = size
    plan = fc.MxPlan(M, N, K, dtype)
    quantised = fc.MxQuantPlan(M, K, dtype).bytes
    return plan, (size, plan.kernel_name, plan.workspace_bytes >= quantised + 2 * 4 * M * N)


@pytest.mark.parametrize("row", XENT, ids=lambda r: "%dx%dx%d" % r[0])
def test_loss_and_gradient(row):
    dev = device()
    T, D, V = row[0]
    say("tiled", row)
    plan, got = xent_selection(row[0])
    assert got == row
    h, w, t, dl = case(T, D, V, "bf16", dev)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl)
    check(h, w, t, dl, loss, lse, dh, dw, "bf16", 4000)
    for _ in range(3):
        l2, s2 = plan.forward(h, w, t)
        a, b = plan.backward(h, w, t, s2, dl)
        assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(a, dh) and torch.equal(b, dw)


@pytest.mark.parametrize("T,D,V", [(2000, 200, 5000), (7000, 1288, 5000), (3000, 1024, 20000)])
def test_rows_apart(T, D, V):
    # Rows that stay on 16-byte boundaries: the tiled kernels; what lies between them is read and written by nobody.
    dev = device()
    say("rows apart", T, D, V)
    plan = fc.XentPlan(T, D, V, "bf16", ignore_index=IGN)
    h0, w0, t, dl = case(T, D, V, "bf16", dev)
    nan = float("nan")
    hb = torch.full((T, D + 24), nan, dtype=torch.bfloat16, device=dev)
    wb = torch.full((V, D + 40), nan, dtype=torch.bfloat16, device=dev)
    h, w = hb[:, 8:8 + D], wb[:, 16:16 + D]
    h.copy_(h0)
    w.copy_(w0)
    ob = torch.full((T, D + 16), 7.0, dtype=torch.bfloat16, device=dev)
    pb = torch.full((V, D + 8), 7.0, dtype=torch.bfloat16, device=dev)
    loss, lse = plan.forward(h, w, t)
    dh, dw = plan.backward(h, w, t, lse, dl, dh=ob[:, 8:8 + D], dw=pb[:, 8:8 + D])
    check(h, w, t, dl, loss, lse, dh, dw, "bf16", 4000)
    assert bool((ob[:, :8] == 7).all()) and bool((ob[:, 8 + D:] == 7).all()) and bool((pb[:, :8] == 7).all())
    l2, s2 = plan.forward(h0, w0, t)
    a, b = plan.backward(h0, w0, t, s2, dl)
    assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(a, dh) and torch.equal(b, dw)


def _values(rows, cols, dtype, seed, dev):
    """Values of many sizes, a power of two apart from block to block."""
    g = torch.Generator(device=dev).manual_seed(seed)
    e = torch.randint(-6, 7, (rows, -(-cols // 32)), generator=g, device=dev).float()
    return (torch.randn(rows, cols, generator=g, device=dev) * torch.exp2(e).repeat_interleave(32, 1)[:, :cols]).to(TDT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("row", MX, ids=lambda r: "%dx%dx%d" % r[0])
def test_product(row, dtype):
    dev = device()
    M, N, K = row[0]
    say("tiled product", row, dtype)
    plan, got = mx_selection(row[0], dtype)
    assert got == row
    x, bias = _values(M, K, dtype, 1, dev), torch.randn(N, device=dev)
    qw, qx = fc.MxQuantPlan(N, K, "fp32"), fc.MxQuantPlan(M, K, dtype)
    w4, x4 = qw(_values(N, K, "fp32", 2, dev)), qx(x)
    y, y2 = plan(x, w4, bias=bias), plan(x4, w4, bias=bias)
    xv = fc.MxQuantPlan(M, K, "fp32").dequantize(x4).double()  # exact, see test_gpu_mx.py
    wv = qw.dequantize(w4).double().t()
    ref = torch.mm(xv, wv) + bias.double()
    bound = sum_error(xv, wv, K) + U * ref.abs() + (2.0 ** -8 * ref.abs() if dtype == "bf16" else 0) + 1e-37
    assert bool(((y.double() - ref).abs() <= bound).all())
    assert torch.equal(y, y2)
    for _ in range(3):
        assert torch.equal(plan(x, w4, bias=bias), y)
