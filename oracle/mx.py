"""MXFP4 in plain numpy: quantisation, values, and the matrix order of
include/fconv_mx.h.  Shares no code with the kernels."""
from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [rows, cols] (any float type) to codes [rows, nb*32] (one per byte,
    zeros past cols) and scale bytes [rows, nb].  Sign of a zero code: that of
    x.  Blocks with an infinity or NaN: scale 255, codes 0."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    m = np.abs(b).max(-1)
    # frexp: m = f 2^k, f in [0.5, 1).
    e = np.where(m > 0, np.clip(np.frexp(m)[1] - 3, -127, 127), -127)
    a = np.abs(b) * np.exp2(-e.astype(np.float64))[..., None]
    dist = np.abs(a[..., None] - VALUES)
    near = dist.min(-1, keepdims=True)
    even_first = np.where(dist == near, np.arange(8) + 8 * (np.arange(8) % 2), 99)
    code = even_first.argmin(-1).astype(np.uint8)
    code |= (np.signbit(b).astype(np.uint8) << 3)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    code[bad] = 0
    return code.reshape(rows, nb * 32), scale


def values(codes, scales, cols):
    """float64 values of codes [rows, nb*32] and scales [rows, nb]."""
    rows, nb = scales.shape
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(rows, nb, 32) * s[..., None]).reshape(rows, -1)[:, :cols]


def pack(codes):
    """Row-major pairs, low half first: [rows, nb*16]."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def read_buffer(buf, rows, cols):
    """Codes [rows, nb*32] and scales [rows, nb] of a laid-out buffer, and
    whether everything outside them is zero."""
    buf = np.asarray(buf, np.uint8).copy()
    kt, ks, nb = -(-cols // 128), -(-cols // 512), -(-cols // 32)
    base = -(-rows // 16) * kt * 1024
    assert buf.size == base + -(-rows // 16) * ks * 256
    r = np.arange(rows)[:, None]
    c = np.arange(nb * 32)[None, :]
    at = ((r // 16) * kt + c // 128) * 1024 + ((c % 128) // 32 * 16 + r % 16) * 16 + (c % 32) // 2
    codes = (buf[at] >> (4 * (c % 2))) & 15
    b = np.arange(nb)[None, :] * 32
    sat = base + ((r // 16) * ks + b // 512) * 256 + ((b % 128) // 32 * 16 + r % 16) * 4 + (b % 512) // 128
    scales = buf[sat]
    buf[at.ravel()] = 0
    buf[sat.ravel()] = 0
    return codes.astype(np.uint8), scales, not buf.any()
