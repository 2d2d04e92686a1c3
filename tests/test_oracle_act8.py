"""Pins of the 8-bit block oracle (CPU only): brute force over every code and
every exponent, torch's float8 conversions, landmarks, and the gated
activation's gradient against finite differences."""

import numpy as np
import pytest
import torch

from oracle import act8, fp8
from oracle.bf16 import bf16_round


def _all_values(fmt):
    """(values, codes) of the finite codes."""
    codes = np.arange(256, dtype=np.uint8)
    v = act8.dequantize(codes[None, :], np.full((1, 4), 127, np.uint8), 256, fmt)[0]
    ok = np.isfinite(v)
    return v[ok], codes[ok]


@pytest.mark.parametrize("fmt", [0, 1])
def test_codes_are_nearest_by_brute_force(fmt):
    rng = np.random.default_rng(fmt)
    x = bf16_round((rng.standard_normal((6, 300)) * 10.0 ** rng.uniform(-6, 6, (6, 1)))
                   .astype(np.float32)).astype(np.float64)
    codes, scales = act8.quantize(x, fmt)
    vals, cs = _all_values(fmt)
    top = vals.max()
    for r in range(x.shape[0]):
        for b in range(3):
            blk = x[r, b * 128:(b + 1) * 128]
            e = int(scales[r, b]) - 127
            assert np.abs(blk).max() <= top * 2.0 ** e
            assert e == act8.E_MIN or np.abs(blk).max() > top * 2.0 ** (e - 1)
            d = np.abs(vals[None, :] * 2.0 ** e - blk[:, None])
            got = codes[r, b * 128:b * 128 + blk.size]
            for i in range(blk.size):
                near = cs[d[i] == d[i].min()]
                # equal distance: two codes (the even one), or +0 and -0
                even = [c for c in near if c % 2 == 0]
                assert got[i] in near and (len(near) == 1 or got[i] in even)
    assert not codes[:, 300:].any() and not scales[:, 3:].any()


@pytest.mark.parametrize("fmt,dt", [(0, torch.float8_e4m3fn), (1, torch.float8_e5m2)])
def test_codes_match_torch(fmt, dt):
    rng = np.random.default_rng(7)
    x = bf16_round(rng.standard_normal((5, 1024)).astype(np.float32)).astype(np.float64)
    codes, scales = act8.quantize(x, fmt)
    e = scales.astype(np.int64) - 127
    y = x * np.exp2(-np.repeat(e, 128, 1).astype(np.float64))
    want = torch.from_numpy(y.astype(np.float32)).to(dt).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)


def test_special_blocks():
    x = np.zeros((4, 128))
    x[1, 3], x[1, 5], x[1, 7] = np.nan, -np.inf, 2.0
    x[2, :] = 2.0 ** -133
    x[3, 0], x[3, 1] = -448.0 * 2.0 ** 100, -0.0
    for fmt in (0, 1):
        codes, scales = act8.quantize(x, fmt)
        assert not codes[0].any() and scales[0, 0] == 17
        v = act8.dequantize(codes, scales, 128, fmt)
        assert np.isnan(v[1, 3]) and v[1, 7] == 2.0
        assert np.isnan(v[1, 5]) if fmt == 0 else v[1, 5] == -np.inf
        assert scales[2, 0] == 17 and not codes[2].any()
        assert v[3, 0] == x[3, 0] and codes[3, 1] == 0x80
    assert scales[3, 0] == 127 + 100 - 7  # E5M2: 448 = 57344 / 128


def test_exponent_rule():
    for fmt in (0, 1):
        top = fp8.max_finite(act8.FMT[fmt])
        for k in (-110, -3, 0, 9, 100):
            a = np.array([top * 2.0 ** k, np.nextafter(top * 2.0 ** k, np.inf)])
            assert act8.exponent(a, fmt).tolist() == [k, k + 1]
        assert act8.exponent(np.array([0.0, 1e-40]), fmt).tolist() == [-110, -110]


def test_planted_wrong_scale_is_caught():
    """A scale one binade too large fails the least-exponent rule, and moves values."""
    rng = np.random.default_rng(1)
    x = bf16_round(rng.standard_normal((1, 128)).astype(np.float32)).astype(np.float64)
    codes, scales = act8.quantize(x, 0)
    fine = np.abs(act8.dequantize(codes, scales, 128, 0) - x).max()
    worse = act8._encode(x * 2.0 ** -(int(scales[0, 0]) - 126), 0)
    v = act8.dequantize(worse, scales + 1, 128, 0)
    assert np.abs(v - x).max() >= fine and (worse != codes).any()


def test_weight_blocks_are_order_free():
    """The codes of a 128 x 128 block do not depend on the order kept."""
    rng = np.random.default_rng(3)
    w = bf16_round((rng.standard_normal((200, 300)) * 0.02).astype(np.float32)).astype(np.float64)
    c, s = act8.quantize(w, 0, rows=128)
    ct, st = act8.quantize(w.T.copy(), 0, rows=128)
    assert np.array_equal(c[:, :300], ct[:, :200].T)
    assert np.array_equal(s[:2, :3], st[:3, :2].T)


def test_swiglu_gradient_by_differences():
    rng = np.random.default_rng(5)
    g, u, dh = rng.standard_normal(200) * 3, rng.standard_normal(200), rng.standard_normal(200)
    dg, du = act8.swiglu_bwd(dh, g, u)
    h = 1e-5
    ng = dh * (act8.swiglu_fwd(g + h, u) - act8.swiglu_fwd(g - h, u)) / (2 * h)
    nu = dh * (act8.swiglu_fwd(g, u + h) - act8.swiglu_fwd(g, u - h)) / (2 * h)
    # central differences: h^2/6 f''' (f''' < 1 here) plus 1e-16 / h of rounding
    assert np.abs(dg - ng).max() < 1e-9 and np.abs(du - nu).max() < 1e-9
