"""The rules of the 8-bit blocks as a check of any (values, codes, scales),
and planted mistakes that it has to find (CPU only)."""

import numpy as np
import pytest

from oracle import act8
from oracle.bf16 import bf16_round


def _finite_codes(fmt):
    codes = np.arange(256, dtype=np.uint8)
    v = act8.dequantize(codes[None, :], np.full((1, 4), 127, np.uint8), 256, fmt)[0]
    ok = np.isfinite(v)
    return v[ok], codes[ok]


def check_blocks(x, codes, scales, fmt):
    """Raises where codes and scales of finite x [R x C] break a rule: the
    least exponent that covers the block, the nearest code, ties to the even
    one, the sign of zero, zeros past the last column."""
    vals, cs = _finite_codes(fmt)
    top = vals.max()
    R, C = x.shape
    for r in range(R):
        for b in range(-(-C // 128)):
            blk = x[r, b * 128:(b + 1) * 128]
            e = int(scales[r, b]) - 127
            assert e >= act8.E_MIN, "exponent below the least"
            assert np.abs(blk).max() <= top * 2.0 ** e, "scale too small"
            assert e == act8.E_MIN or np.abs(blk).max() > top * 2.0 ** (e - 1), "scale too large"
            d = np.abs(vals[None, :] * 2.0 ** e - blk[:, None])
            got = codes[r, b * 128:b * 128 + blk.size]
            for i in range(blk.size):
                near = cs[d[i] == d[i].min()]
                assert got[i] in near, "not the nearest code"
                assert (got[i] & 0x80 != 0) == np.signbit(blk[i]), "sign"
                if len(set(near & 0x7F)) > 1:  # a tie of two magnitudes
                    assert got[i] % 2 == 0, "tie to the odd code"
    assert not codes[:, C:].any() and not scales[:, -(-C // 128):].any(), "padding"


def _sample(seed=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((4, 300)) * 10.0 ** rng.uniform(-6, 6, (4, 1))
    x[2, 7], x[2, 9] = 0.0, -0.0
    x[3, :200] = np.arange(200) % 17 + 16.0  # integers whose codes tie
    return bf16_round(x.astype(np.float32)).astype(np.float64)


@pytest.mark.parametrize("fmt", [0, 1])
def test_the_oracle_keeps_the_rules(fmt):
    for seed in range(3):
        x = _sample(seed)
        check_blocks(x, *act8.quantize(x, fmt), fmt)


def _requantized(x, scales, fmt, r, b, by):
    """Codes and scales with one block's exponent moved by `by`, its codes the nearest ones there."""
    codes, scales = act8.quantize(x, fmt)[0].copy(), scales.copy()
    scales[r, b] = int(scales[r, b]) + by
    vals, cs = _finite_codes(fmt)
    blk = x[r, b * 128:(b + 1) * 128]
    d = np.abs(vals[None, :] * 2.0 ** (int(scales[r, b]) - 127) - blk[:, None])
    codes[r, b * 128:b * 128 + blk.size] = cs[d.argmin(axis=1)]
    return codes, scales


@pytest.mark.parametrize("fmt", [0, 1])
def test_planted_mistakes_are_found(fmt):
    x = _sample()
    codes, scales = act8.quantize(x, fmt)
    with pytest.raises(AssertionError, match="scale too large"):
        check_blocks(x, *_requantized(x, scales, fmt, 0, 1, 1), fmt)
    with pytest.raises(AssertionError, match="scale too small"):
        check_blocks(x, *_requantized(x, scales, fmt, 1, 2, -1), fmt)
    # one code moved to its neighbour, away from the block's largest
    for r, c in ((0, 3), (1, 299), (3, 130)):
        moved = codes.copy()
        moved[r, c] = codes[r, c] + 1 if codes[r, c] & 0x7F == 0 else codes[r, c] - 1
        with pytest.raises(AssertionError, match="nearest|tie|sign"):
            check_blocks(x, moved, scales, fmt)
    flipped = codes.copy()
    flipped[2, 9] = 0
    with pytest.raises(AssertionError, match="sign"):
        check_blocks(x, flipped, scales, fmt)
    late = codes.copy()
    late[0, 300] = 1
    with pytest.raises(AssertionError, match="padding"):
        check_blocks(x, late, scales, fmt)


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_tie_to_the_odd_code_is_found(fmt):
    step = 2.0 if fmt == 0 else 4.0  # spacing of the codes from 16 on
    x = np.zeros((1, 128))
    x[0, 0] = act8.fp8.max_finite(act8.FMT[fmt])  # the block's scale is 1
    x[0, 1], x[0, 2] = 16.0 + step / 2, 16.0 + 1.5 * step
    codes, scales = act8.quantize(x, fmt)
    assert scales[0, 0] == 127
    check_blocks(x, codes, scales, fmt)
    for c, by in ((1, 1), (2, -1)):
        moved = codes.copy()
        moved[0, c] = int(codes[0, c]) + by
        with pytest.raises(AssertionError, match="tie"):
            check_blocks(x, moved, scales, fmt)
