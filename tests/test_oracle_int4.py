"""Pins of the oracle's groups of 4-bit codes: rationals, brute force."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import int4
from oracle.bf16 import bf16_round


def _round_half_even(f):
    n = f.numerator // f.denominator
    rest = f - n
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2):
        n += 1
    return n


def _weights(N, K, seed):
    return bf16_round(np.random.default_rng(seed).normal(0, 0.02, (N, K)).astype(np.float32))


@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("G,K", [(32, 96), (64, 160), (128, 160)])
def test_codes_are_the_nearest_integers(G, K, sym):
    w = _weights(6, K, G)
    w[1, :K // 2] = 0
    w[2] = np.abs(w[2])
    w[3] = -np.abs(w[3])
    w[4] = np.round(w[4] * 64) / 64  # many ties
    codes, s, z = int4.quantize(w, G, sym)
    q = np.stack([codes & 15, codes >> 4], 2).reshape(6, K)
    for i in range(6):
        for k in range(K):
            sc, zz = Fraction(float(s[i, k // G])), 8 if sym else int(z[i, k // G])
            want = zz if sc == 0 else min(15, max(0, _round_half_even(Fraction(float(w[i, k])) / sc) + zz))
            assert q[i, k] == want
    if not sym:
        for i in range(6):
            for g in range(int4.groups(K, G)):
                lo = Fraction(float(min(0.0, w[i, g * G:(g + 1) * G].min())))
                sc = Fraction(float(s[i, g]))
                assert z[i, g] == (0 if sc == 0 else min(15, _round_half_even(-lo / sc)))


def test_error_is_half_a_step():
    """Away from the two ends no other code is nearer; the scale's own rounding
    (2^-8) moves an end by at most 15 2^-8 of a step more."""
    w = _weights(8, 256, 5)
    for sym in (False, True):
        codes, s, z = int4.quantize(w, 64, sym)
        d = int4.dequantize(codes, s, None if sym else z, 64)
        step = np.repeat(s, 64, axis=1)
        assert (np.abs(d - w) <= step * (0.5 + 16 * 2.0 ** -8) + 1e-12).all()


def test_layout_and_special_groups():
    w = np.zeros((1, 64), np.float32)
    w[0, :4] = [15.0, 0.0, 7.0, 3.0]
    codes, s, z = int4.quantize(w, 32, False)
    assert s.tolist() == [[1.0, 0.0]] and z.tolist() == [[0, 0]]
    assert codes[0, :2].tolist() == [0x0F, 0x37] and (codes[0, 2:] == 0).all()
    codes, s, z = int4.quantize(-w, 32, True)
    assert (codes[0, 16:] == 0x88).all() and s[0, 1] == 0
    assert (int4.dequantize(codes, s, None, 32)[0, 32:] == 0).all()
