"""8-bit blocks of activations and weights (TEST INFRASTRUCTURE ONLY).

Definition: a row is cut into blocks of 128 columns (a weight into blocks of
128 x 128). Each block has one power-of-two scale 2^e with e the least
integer >= -110 for which the largest finite magnitude of the block is at
most top 2^e (top = 448 for E4M3, 57344 for E5M2), kept as the byte e + 127;
each value is the code of x 2^-e rounded to nearest, ties to even. A NaN
becomes a NaN code (0x7F / 0xFF in E4M3, 0x7F / 0xFF or another NaN pattern
in E5M2); an infinity a NaN in E4M3 and an infinity in E5M2. Codes past the
last column and scale bytes past the last block are 0.

Gated activation: H = G s(G) U with s the logistic function, and
dG = dH U s(G) (1 + G (1 - s(G))), dU = dH G s(G), in float64.

Everything is exact or float64: x 2^-e is a power-of-two multiple of a bf16
value. Pinned by brute force over all codes, torch's float8 conversions, and
finite differences (tests/test_oracle_act8.py).
"""

import numpy as np

from . import fp8

BLOCK = 128
E_MIN = -110
FMT = (fp8.E4M3, fp8.E5M2)


def row_bytes(K):
    return -(-K // BLOCK) * BLOCK


def scale_row_bytes(K):
    return -(-(-(-K // BLOCK)) // 4) * 4


def exponent(amax, fmt):
    """Least e >= E_MIN with amax <= top 2^e (amax float64 array)."""
    top = fp8.max_finite(FMT[fmt])
    e = np.full(amax.shape, E_MIN, dtype=np.int64)
    for _ in range(260):  # counted up, one binade at a time
        more = amax > top * np.exp2(e.astype(np.float64))
        if not more.any():
            break
        e += more
    return e


def _encode(y, fmt):
    """Codes of float64 y, |y| <= top where finite."""
    finite = np.isfinite(y)
    # y is a bf16 value times a power of two; far below the smallest code it
    # may leave float32's range, where the code is a signed zero
    c = fp8.encode(np.where(finite, y, 0.0).astype(np.float32), FMT[fmt])
    sign = np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    c = np.where(finite, (c & 0x7F) | sign, c).astype(np.uint8)
    c = np.where(np.isnan(y) | (np.isinf(y) & (fmt == 0)), sign | 0x7F, c)
    return np.where(np.isinf(y) & (fmt == 1), sign | 0x7C, c).astype(np.uint8)


def quantize(x, fmt, rows=1):
    """(codes, scales) of a matrix; one scale per `rows` x 128 block."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    Rb, Cb = -(-R // rows), -(-C // BLOCK)
    codes = np.zeros((R, Cb * BLOCK), np.uint8)
    scales = np.zeros((Rb, scale_row_bytes(C)), np.uint8)
    p = np.zeros((Rb * rows, Cb * BLOCK))
    p[:R, :C] = x
    b = p.reshape(Rb, rows, Cb, BLOCK)
    e = exponent(np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=(1, 3)), fmt)
    y = (b * np.exp2(-e.astype(np.float64))[:, None, :, None]).reshape(Rb * rows, Cb * BLOCK)
    codes[:, :C] = _encode(y[:R, :C], fmt)
    scales[:, :Cb] = (e + 127).astype(np.uint8)
    return codes, scales


def dequantize(codes, scales, K, fmt, rows=1):
    """float64 values; NaN and infinity codes as such."""
    c = np.asarray(codes, np.uint8)
    v = fp8.decode(c, FMT[fmt]).astype(np.float64)
    m = c & 0x7F
    if fmt == 0:
        v = np.where(m == 0x7F, np.nan, v)
    else:
        v = np.where(m > 0x7C, np.nan, np.where(m == 0x7C, np.copysign(np.inf, v), v))
    s = np.exp2(np.asarray(scales, np.float64) - 127)
    s = np.repeat(np.repeat(s, rows, 0)[:c.shape[0]], BLOCK, 1)[:, :c.shape[1]]
    return (v * s)[:, :K]


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def swiglu_fwd(g, u):
    g, u = np.asarray(g, np.float64), np.asarray(u, np.float64)
    return g * sigmoid(g) * u


def swiglu_bwd(dh, g, u):
    dh, g, u = (np.asarray(t, np.float64) for t in (dh, g, u))
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * sigmoid(-g)), dh * g * s
