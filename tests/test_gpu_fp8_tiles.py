"""The linear calls on 8-bit inputs at sizes that take each tile of the
product: 64 x 64 and 128 x 64 tiles with one and with two sets of waves, the
low-rank term in one or more steps, the adapter's gradients beside the tiles
or in their own launch, each with the two code formats in all pairs of input
and upstream gradient, and on the NF4 base with and without dropout. Also
few tokens with ranks that several threads share. Bounds: those of
test_gpu_fp8_linear."""

import numpy as np
import pytest
import torch

import oracle
from oracle import act8
from tests.gpu_util import device
from tests.test_gpu_fp8_linear import (Case, _check, _dec, _f64, _fwd_check, _grad_check, _low, _norm,
                                       _steps, _steps8)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


# Tile of a product by its rows m, columns n and bytes of a row along the
# contraction: the library's rule, by which the sizes below were chosen.
def _tile(m, n, row_bytes):
    t64, t128 = -(-m // 64) * -(-n // 64), -(-m // 64) * -(-n // 128)
    if t128 > 256:
        return "128x64 alone" if t128 < 512 else "256x256"
    return ("64x64" if t64 <= 256 else "128x64") + (" two sets" if -(-row_bytes // 128) >= 16 else " one set")


# (M, N, K, r); the backward's product is M x K over N, the forward's M x N over K
BACKWARD = [(300, 2112, 3520, 8), (300, 2112, 3520, 24), (299, 2176, 3520, 64),
            (300, 512, 3520, 8), (300, 512, 3520, 24), (257, 512, 4032, 64),
            (300, 192, 3520, 200), (601, 512, 3520, 64), (600, 192, 3520, 8)]
FORWARD = [(300, 3520, 2112, 24), (299, 3520, 2176, 64), (300, 3520, 576, 16), (300, 3520, 320, 200),
           (601, 3520, 320, 24), (600, 3520, 2112, 100)]


def test_sizes_cover_the_tiles():
    names = [_tile(M, K, N) for M, N, K, _ in BACKWARD]
    for want in ("128x64 two sets", "128x64 one set", "128x64 alone"):
        assert want in names and want in [_tile(M, N, K) for M, N, K, _ in FORWARD]
    # the ranks of the three widths of the gradients' tiles beside 128 x 64 ones
    for sets in ("two", "one"):
        ranks = [s[3] for s, n in zip(BACKWARD, names) if n == f"128x64 {sets} set" + "s" * (sets == "two")]
        assert any(r <= 16 for r in ranks) and any(16 < r <= 32 for r in ranks) and any(r > 32 for r in ranks)
    # the bf16 product of the NF4 base, whose rows are twice as long
    bf = [_tile(M, K, 2 * N) for M, N, K, _ in BACKWARD]
    assert "128x64 two sets" in bf and "128x64 one set" in bf and "128x64 alone" in bf


@pytest.mark.parametrize("fmt,dfmt", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("M,N,K,r", BACKWARD + [(16, 256, 256, 8), (65, 128, 64, 64), (1100, 256, 4160, 64)])
def test_backward(q, M, N, K, r, fmt, dfmt):
    print(f"[case] fp8 backward M={M} N={N} K={K} r={r} fmt={fmt} dY fmt={dfmt}", flush=True)
    c = Case(q, M, N, K, r, fmt)
    W = q.qlora_fp8_weight_quantize(c.W)
    T = torch.from_numpy((c.X @ c.a).astype(np.float32)).to(device())
    dX, dA, dB = q.qlora_fp8_linear_bwd(c.dY, c.x8, T, W, c.A, c.B, c.s, fmt=dfmt)
    G, gabs = _grad_check(c, c.X, T, dA, dB, M, N, r)
    w = _dec(W.codes_t, W.scales_t, N, 0, 128)
    d = act8.dequantize(*act8.quantize(c.dy, dfmt), N, dfmt)
    low, ltol = _low(c, G, gabs, N, r)
    want = d @ w.T + low
    _check(_f64(dX), want, _steps8(N) * (np.abs(d) @ np.abs(w).T) + ltol
           + 2.0 ** -8 * 1.01 * np.abs(want), "dX")
    again = q.qlora_fp8_linear_bwd(c.dY, c.x8, T, W, c.A, c.B, c.s, fmt=dfmt)
    assert all(torch.equal(a, b) for a, b in zip(again, (dX, dA, dB)))


@pytest.mark.parametrize("drop", [0.0, 0.1])
@pytest.mark.parametrize("M,N,K,r", [s for s in BACKWARD if s[3] <= 192] + [(600, 64, 3520, 24)])
def test_nf4_backward(q, M, N, K, r, drop):
    print(f"[case] nf4 backward M={M} N={N} K={K} r={r} drop={drop}", flush=True)
    fmt = (M + r // 8) % 2
    c = Case(q, M, N, K, r, fmt)
    st = q.qlora_nf4_quantize(c.W)
    keep, kw, f, D = 1.0, {}, 1.0, c.X
    if drop:
        mask = q.qlora_dropout_mask(M, K, drop, seed=5, device=device())
        kw = dict(keep_mask=mask, p=drop)
        keep = oracle.unpack_keep(mask.cpu().numpy().view(np.uint32), K).astype(np.float64)
        f = oracle.keep_scale(drop)
        D = c.X * keep * f
    T = torch.from_numpy((D @ c.a).astype(np.float32)).to(device())
    dX, dA, dB = q.qlora_linear_bwd_act8(c.dY, c.x8, T, st, c.A, c.B, c.s, **kw)
    G, gabs = _grad_check(c, D, T, dA, dB, M, N, r)
    w = _f64(q.qlora_nf4_dequantize_bf16(st)).reshape(N, K)
    low, ltol = _low(c, G, gabs, N, r)
    want = c.dy @ w + low * keep * f
    _check(_f64(dX), want, _steps(N) * (np.abs(c.dy) @ np.abs(w)) + ltol * f
           + 2.0 ** -8 * 1.01 * np.abs(want), "dX")


def test_nf4_backward_wide_rank(q):
    """Four steps of the low-rank term in the bf16 product."""
    M, N, K, r = 300, 192, 3520, 200
    c = Case(q, M, N, K, r)
    st = q.qlora_nf4_quantize(c.W)
    T = torch.from_numpy((c.X @ c.a).astype(np.float32)).to(device())
    dX, dA, dB = q.qlora_linear_bwd_act8(c.dY, c.x8, T, st, c.A, c.B, c.s)
    G, gabs = _grad_check(c, c.X, T, dA, dB, M, N, r)
    w = _f64(q.qlora_nf4_dequantize_bf16(st)).reshape(N, K)
    low, ltol = _low(c, G, gabs, N, r)
    want = c.dy @ w + low
    _check(_f64(dX), want, _steps(N) * (np.abs(c.dy) @ np.abs(w)) + ltol
           + 2.0 ** -8 * 1.01 * np.abs(want), "dX")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K,r", FORWARD)
def test_forward(q, M, N, K, r, fmt):
    print(f"[case] fp8 forward M={M} N={N} K={K} r={r} fmt={fmt}", flush=True)
    c = Case(q, M, N, K, r, fmt)
    W = q.qlora_fp8_weight_quantize(c.W)
    Y, T = q.qlora_fp8_linear_fwd(c.x8, W, c.A, c.B, c.s)
    _fwd_check(c, W, Y, T, N, K, r)
    plain, none = q.qlora_fp8_linear_fwd(c.x8, W)
    w = _dec(W.codes, W.scales, K, 0, 128)
    want = c.X @ w.T
    _check(_f64(plain), want, _steps8(K) * (np.abs(c.X) @ np.abs(w).T) + 2.0 ** -8 * 1.01 * np.abs(want), "Y plain")
    _norm(_f64(plain), want, "Y plain")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,N,K,r", [(1, 1024, 320, 200), (1, 512, 640, 24), (2, 64, 64, 17), (3, 512, 640, 24),
                                     (5, 448, 2112, 100), (9, 128, 4160, 33), (13, 256, 1344, 100),
                                     (16, 512, 512, 48), (17, 192, 576, 24), (30, 1024, 192, 72)])
def test_few_tokens_share_ranks(q, M, N, K, r, fmt):
    """Ranks above 16 in the product for few tokens, split over threads in
    runs that a rank need not fill."""
    print(f"[case] few tokens M={M} N={N} K={K} r={r} fmt={fmt}", flush=True)
    assert -(-M // 16) * -(-N // 16) <= 512
    c = Case(q, M, N, K, r, fmt)
    W = q.qlora_fp8_weight_quantize(c.W)
    Y, T = q.qlora_fp8_linear_fwd(c.x8, W, c.A, c.B, c.s)
    _fwd_check(c, W, Y, T, N, K, r)
    g0 = q.qlora_fp8_linear_bwd(c.dY, c.x8, T, W, c.A, c.B, c.s, want_dX=False)
    g1 = q.qlora_fp8_linear_bwd(c.dY, c.x8, None, W, c.A, c.B, c.s, want_dX=False)
    assert torch.equal(g0[1], g1[1]) and torch.equal(g0[2], g1[2])
