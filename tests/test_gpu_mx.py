"""MXFP4 on the GPU against plain numpy in 64 bits (oracle/mx.py).

Tolerances.  Quantisation and its inverse are exact.  The product sums K exact
products of fp32-representable values in fp32: with products of root mean
square s (per output), the partial sums grow like sqrt(k) s, each addition is
off by at most half a step (2^-24 relative), and the errors add up to about
2^-24 K s / 2.5; 4 * 2^-24 K s is ten of those.  A bf16 output adds half a
step, 2^-8 of its value, and the bias one fp32 addition."""
import numpy as np
import pytest
import torch

import convolution_implicit_gemm_nhwc_amd as fc
from gpu_helpers import device, say
from oracle import mx as omx

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _x(rows, cols, dtype, seed, dev):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, -(-cols // 32)), generator=g)
                                                          .float()).repeat_interleave(32, 1)[:, :cols]
    return x.to(TDT[dtype]).to(dev)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check_buffer(t, x):
    codes, scales, clean = omx.read_buffer(t.data.cpu().numpy(), t.rows, t.cols)
    rc, rs = omx.quantize(x)
    assert np.array_equal(scales, rs)
    live = np.where(codes == 8, 0, codes)  # the sign of a zero code is free
    assert np.array_equal(live, np.where(rc == 8, 0, rc))
    assert clean


SHAPES = [(1, 1), (1, 32), (3, 33), (16, 128), (17, 127), (31, 512), (5, 513), (33, 1000), (130, 640), (2, 4097)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_is_exact(rows, cols, dtype):
    dev = device()
    say("quantize", rows, cols, dtype)
    x = _x(rows, cols, dtype, rows * 7 + cols, dev)
    q = fc.MxQuantPlan(rows, cols, dtype)
    t = q(x)
    torch.cuda.synchronize()
    _check_buffer(t, _np(x))
    back = q.dequantize(t)
    assert np.array_equal(_np(back), omx.values(*omx.quantize(_np(x)), cols))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_strided_and_unaligned_rows(dtype):
    dev = device()
    say("strided", dtype)
    big = _x(37, 211, dtype, 5, dev)
    x = big[:, 3:203]
    t = fc.MxQuantPlan(37, 200, dtype)(x)
    torch.cuda.synchronize()
    _check_buffer(t, _np(x))
    nhwc = _x(2 * 3 * 5, 40, dtype, 6, dev).view(2, 3, 5, 40)
    t = fc.MxQuantPlan(30, 40, dtype)(nhwc)
    torch.cuda.synchronize()
    _check_buffer(t, _np(nhwc).reshape(30, 40))


def test_every_bf16_value_in_its_own_block():
    # 65536 blocks, each with one bf16 bit pattern among zeros: every scale, subnormals, infinities, NaNs.
    dev = device()
    say("every bf16")
    bits = np.arange(65536, dtype=np.uint16)
    x = np.zeros((65536, 32), np.uint16)
    x[np.arange(65536), np.arange(65536) % 32] = bits
    xt = torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16).view(4096, 512)
    q = fc.MxQuantPlan(4096, 512, "bf16")
    t = q(xt)
    torch.cuda.synchronize()
    _check_buffer(t, _np(xt))
    back = fc.MxQuantPlan(4096, 512, "fp32").dequantize(t)
    ref = omx.values(*omx.quantize(_np(xt)), 512)
    assert np.array_equal(_np(back), ref, equal_nan=True)


def test_every_rounding_border():
    # Next to and on every middle between two codes, at many scales, both signs.
    dev = device()
    say("borders")
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    rows = []
    for e in list(range(-126, 120, 7)) + [-148, -140]:
        with np.errstate(under="ignore"):
            blk = np.concatenate([v, -v[:6], [np.float32(4.0), np.float32(-7.99)]]).astype(np.float32)
            rows.append(np.ldexp(blk, e).astype(np.float32))
    x = torch.from_numpy(np.stack(rows)).to(dev)
    t = fc.MxQuantPlan(x.shape[0], 32, "fp32")(x)
    torch.cuda.synchronize()
    _check_buffer(t, _np(x))


def test_layout_from_row_major_codes():
    dev = device()
    rng = np.random.default_rng(3)
    for rows, cols in ((1, 5), (18, 100), (33, 1030), (16, 512)):
        say("layout", rows, cols)
        nb = -(-cols // 32)
        codes = rng.integers(0, 16, (rows, nb * 32), dtype=np.uint8)
        scales = rng.integers(100, 150, (rows, nb), dtype=np.uint8)
        t = fc.MxTensor.from_codes(torch.from_numpy(omx.pack(codes)).to(dev), torch.from_numpy(scales).to(dev), cols)
        torch.cuda.synchronize()
        got, gs, clean = omx.read_buffer(t.data.cpu().numpy(), rows, cols)
        codes[:, cols:] = 0
        assert np.array_equal(got, codes) and np.array_equal(gs, scales) and clean


def _bound(xv, wv, K, ref, dtype):
    s = np.sqrt((xv ** 2) @ (wv ** 2).T / K)
    b = 4 * 2.0 ** -24 * K * s + 2.0 ** -24 * np.abs(ref)
    return b + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0) + 1e-37


PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 1000, 512), (2, 33, 129), (5, 1000, 1000), (16, 64, 4096), (17, 300, 770),
            (33, 65, 640), (64, 128, 256), (100, 257, 1025), (300, 70, 384), (1000, 64, 256), (513, 260, 130),
            (4100, 1030, 300), (4097, 4100, 96)]
# Few rows (one kernel each for 1 to 16, 32 and 64, k cut into ranges or not, x quantised on the way or before),
# many rows of few outputs, and sums cut into ranges in the tiled kernels.
PRODUCTS += [(1, 32, 16385), (3, 40, 5000), (4, 16400, 520), (16, 16399, 1030), (15, 33, 16000), (31, 70, 9000),
             (33, 50, 9001), (40, 4000, 1500), (49, 33, 2049), (64, 64, 25088), (65, 100, 9000), (300, 200, 20000),
             (4096, 1, 33), (5000, 64, 256), (4099, 67, 700), (6000, 128, 1000), (4100, 17, 129), (20, 40, 40000), (2, 33, 70001),
             (4500, 100, 1500)]
# Small products by the rows kernel: rows and outputs that end inside a tile, one and several blocks of outputs.
PRODUCTS += [(17, 16, 31), (40, 100, 260), (65, 300, 127), (129, 513, 385), (500, 200, 512), (2000, 1001, 130)]
# Whole tiles one after another on a workgroup, whose stores overlap the next tile, and ragged ones between them.
PRODUCTS += [(2304, 9000, 512), (4096, 8192, 260), (2100, 8200, 1030)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, dtype):
    dev = device()
    x, w = _x(M, K, dtype, 1, dev), _x(N, K, "fp32", 2, dev)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(dev)
    wq = fc.MxQuantPlan(N, K, "fp32")(w)
    plan = fc.MxPlan(M, N, K, dtype, ops=("bias",))
    say("product", M, N, K, dtype, plan.kernel_name)
    y = plan(x, wq, bias=bias)
    xq = fc.MxQuantPlan(M, K, dtype)(x)
    y2 = plan(xq, wq, bias=bias)
    torch.cuda.synchronize()
    xv = omx.values(*omx.quantize(_np(x)), K)
    wv = omx.values(*omx.quantize(_np(w)), K)
    ref = xv @ wv.T + _np(bias)
    bound = _bound(xv, wv, K, ref, dtype)
    assert (np.abs(_np(y) - ref) <= bound).all()
    assert (np.abs(_np(y2) - ref) <= bound).all()


@pytest.mark.parametrize("ops,al,be", [((), 0, 0), (("relu",), 0, 0), (("bias", "leaky_relu"), 0.125, 0),
                                       (("clipped_relu",), 3.0, 0), (("bias", "clamp"), -2.0, 5.0)])
def test_product_epilogues(ops, al, be):
    dev = device()
    for M, N, K in ((3, 130, 96), (140, 70, 160)):
        say("epilogue", ops, M, N, K)
        x, w = _x(M, K, "fp32", 1, dev), _x(N, K, "fp32", 2, dev)
        bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(dev)
        y = fc.MxPlan(M, N, K, "fp32", ops=ops)(x, fc.MxQuantPlan(N, K, "fp32")(w),
                                              bias=bias if "bias" in ops else None, activ_alpha=al, activ_beta=be)
        xv = omx.values(*omx.quantize(_np(x)), K)
        wv = omx.values(*omx.quantize(_np(w)), K)
        t = xv @ wv.T + (_np(bias) if "bias" in ops else 0)
        ref = {"relu": lambda: np.maximum(t, 0), "leaky_relu": lambda: np.where(t > 0, t, al * t),
               "clipped_relu": lambda: np.clip(t, 0, al), "clamp": lambda: np.clip(t, al, be)
               }.get(ops[-1] if ops else "", lambda: t)()
        # The activations' slopes are at most 1, so t's own error bounds the result's.
        assert (np.abs(_np(y) - ref) <= _bound(xv, wv, K, t, "fp32")).all()


@pytest.mark.parametrize("M,N,K", [(3, 40, 300), (200, 150, 300)])
def test_product_strided_rows_and_output_guard(M, N, K):
    dev = device()
    say("strided product", M, N, K)
    xb, w = _x(M, K + 9, "bf16", 1, dev), _x(N, K, "fp32", 2, dev)
    x = xb[:, 5:5 + K]
    out = torch.full((M, N + 7), 7.0, dtype=torch.bfloat16, device=dev)
    fc.MxPlan(M, N, K, "bf16", ops=())(x, fc.MxQuantPlan(N, K, "fp32")(w), out=out[:, 3:3 + N])
    torch.cuda.synchronize()
    xv = omx.values(*omx.quantize(_np(x)), K)
    wv = omx.values(*omx.quantize(_np(w)), K)
    ref = xv @ wv.T
    assert (np.abs(_np(out[:, 3:3 + N]) - ref) <= _bound(xv, wv, K, ref, "bf16")).all()
    assert (out[:, :3] == 7).all() and (out[:, 3 + N:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(2, 40, 300), (150, 140, 300)])
def test_nan_and_infinity_reach_their_row_only(M, N, K):
    dev = device()
    say("nan", M, N, K)
    x, w = _x(M, K, "fp32", 1, dev), _x(N, K, "fp32", 2, dev)
    x[1, 40] = float("inf")
    w[7, 290] = float("nan")
    y = fc.MxPlan(M, N, K, "fp32", ops=("relu",))(x, fc.MxQuantPlan(N, K, "fp32")(w))
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[1, :] = True
    want[:, 7] = True
    assert np.array_equal(bad, want)


def test_extreme_scales_multiply_exactly():
    # Scales near both ends of e8m0: 2^-100 against 2^100, and products that leave fp32.
    dev = device()
    say("scales")
    M, N, K = 4, 32, 64
    x, w = torch.ones(M, K, device=dev), torch.ones(N, K, device=dev)
    for ex, ew in ((100, -100), (-120, 120), (-126, 60), (90, 30)):
        y = fc.MxPlan(M, N, K, "fp32", ops=())(x * 2.0 ** ex, fc.MxQuantPlan(N, K, "fp32")(w * 2.0 ** ew))
        assert (y.double() == K * 2.0 ** (ex + ew)).all()
    y = fc.MxPlan(M, N, K, "fp32", ops=())(x * 2.0 ** 100, fc.MxQuantPlan(N, K, "fp32")(w * 2.0 ** 60))
    assert torch.isinf(y).all()


def test_same_bits_on_every_run_streams_and_graphs():
    dev = device()
    for M, N, K in ((1, 500, 640), (20, 100, 5000), (300, 200, 256)):
        say("streams", M, N, K)
        x, w = _x(M, K, "bf16", 1, dev), _x(N, K, "fp32", 2, dev)
        wq = fc.MxQuantPlan(N, K, "fp32")(w)
        plan = fc.MxPlan(M, N, K, "bf16", ops=())
        y0 = plan(x, wq)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(3):
            y1 = plan(x, wq, stream=side)
            side.synchronize()
            assert torch.equal(y0, y1)
        y2 = torch.empty_like(y0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan(x, wq, out=y2)
        for _ in range(3):
            y2.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y0, y2)
            plan(x, wq)


def test_both_ways_through_a_call_agree():
    # Without a stream a call goes through csrc/call.cpp, with one through _dense.py; also what the first leaves to the second.
    dev = device()
    say("ways")
    x = _x(40, 100, "fp32", 1, dev)
    q = fc.MxQuantPlan(40, 100, "fp32")
    here = torch.cuda.current_stream()
    a, b = q(x), q(x, stream=here)
    # The gap between the last row's codes and whole tiles holds zeros in both.
    assert torch.equal(a.data, b.data)
    assert torch.equal(q.dequantize(a), q.dequantize(b, stream=here))
    w = fc.MxQuantPlan(24, 100, "fp32")(_x(24, 100, "fp32", 2, dev))
    p = fc.MxPlan(40, 24, 100, "fp32", ops=("bias", "clamp"))
    bias = torch.ones(24, device=dev)
    y = p(x, w, bias=bias)  # both bounds 0
    assert torch.equal(y, p(x, w, bias=bias, stream=here)) and (y == 0).all()
    y = p(x, w, bias=bias, activ_alpha=-1.0, activ_beta=1.0)
    assert torch.equal(y, p(x, w, bias=bias, activ_alpha=-1.0, activ_beta=1.0, stream=here)) and (y != 0).any()
    nhwc = x.view(2, 4, 5, 100)
    assert torch.equal(p(nhwc, w, bias=bias), p(x, w, bias=bias))
    param = torch.nn.Parameter(x)
    assert torch.equal(q(param).data, a.data)
    for bad, match in ((x.bfloat16(), "dtype"), (x[:39], "shape"), (x.cpu(), "GPU"), (x.t(), "shape")):
        with pytest.raises(ValueError, match=match):
            q(bad)
        with pytest.raises(ValueError, match=match):
            p(bad, w, bias=bias)
    with pytest.raises(ValueError, match="different devices|GPU"):
        p(x, w, bias=bias.cpu())
    with pytest.raises(ValueError, match="elements"):
        p(x, w, bias=bias[:23])
