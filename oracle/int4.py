"""Weights in groups of 4-bit codes (TEST INFRASTRUCTURE ONLY).

w = s (q - z) for each group of G columns of a row (the last may be shorter).
Over a group's values, with float32 operations, each rounded once:
  asymmetric  lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15),
              z = the integer nearest to -lo / s, at most 15
  symmetric   s = bf16(max|w| / 7), z = 8
  q = the integer nearest to w / s, ties to even, plus z, cut to [0, 15];
a group with s = 0 has z = 0 (symmetric 8) and q = z. Column 2i of a row is in
the low nibble of byte i.

The integers are those nearest to the exact quotients: quotients of two 8-bit
significands are a tie or at least 2^-10 from one, far above float32's
rounding, so that float32, float64 and rational arithmetic agree
(tests/test_oracle_int4.py checks it with rationals).
"""

import numpy as np

from .bf16 import bf16_round


def groups(K, G):
    return -(-K // G)


def quantize(w, G, symmetric):
    """(codes [N, K / 2], scales float32 holding bf16 [N, groups], zeros uint8)."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    ng = groups(K, G)
    q = np.zeros((N, K), np.uint8)
    s = np.zeros((N, ng), np.float32)
    z = np.zeros((N, ng), np.uint8)
    for g in range(ng):
        part = w[:, g * G:(g + 1) * G]
        lo = np.minimum(part.min(axis=1), np.float32(0))
        hi = np.maximum(part.max(axis=1), np.float32(0))
        if symmetric:
            sg = bf16_round(np.maximum(-lo, hi) / np.float32(7))
            zg = np.full(N, 8, np.float32)
        else:
            sg = bf16_round((hi - lo) / np.float32(15))
            with np.errstate(all="ignore"):
                zg = np.where(sg > 0, np.minimum(np.rint(-lo / sg), 15), 0).astype(np.float32)
        with np.errstate(all="ignore"):
            r = np.where(sg[:, None] > 0, np.rint(part / sg[:, None]), 0)
        q[:, g * G:(g + 1) * G] = np.clip(r + zg[:, None], 0, 15)
        s[:, g], z[:, g] = sg, zg
    return q[:, 0::2] | (q[:, 1::2] << 4), s, z


def dequantize(codes, scales, zeros, G):
    """s (q - z) in float64 (exact)."""
    N, half = codes.shape
    q = np.empty((N, 2 * half), np.float64)
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    col = np.arange(2 * half) // G
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, np.float64)
    return np.asarray(scales, np.float64)[:, col] * (q - z[:, col])
