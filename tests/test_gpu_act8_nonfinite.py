"""Infinities and NaN through the linear calls on 8-bit inputs: each reaches
what the formula says it reaches and nothing else, in every form of the
product, and finite factors at the top of float32's range stay finite."""

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import device, host_f32

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _f64(t):
    return host_f32(t).astype(np.float64)


class Positive:
    """Positive operands: a sum that an infinity enters is that infinity."""

    def __init__(self, M, N, K, r):
        dev = device()
        g = torch.Generator(device=dev)
        g.manual_seed(M + N + K + r)
        u = lambda lo, hi, *s: (lo + (hi - lo) * torch.rand(s, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
        self.x, self.W, self.dY = u(0.5, 2, M, K), u(0.5, 1, N, K), u(0.5, 2, M, N)
        self.A = u(0.01, 0.1, K, r) if r else None
        self.B = u(0.01, 0.1, r, N) if r else None


# few tokens with T formed there, with T beside, wide ranks; 64 x 64 and
# 128 x 64 tiles, shared ones, 256 x 256
@pytest.mark.parametrize("M,N,K,r", [(3, 256, 384, 0), (3, 256, 384, 16), (3, 256, 384, 24), (40, 192, 256, 100),
                                     (100, 1280, 576, 24), (100, 1280, 6400, 8), (300, 3520, 576, 16),
                                     (300, 3520, 2112, 0), (1030, 4224, 192, 8)])
def test_infinite_activation(q, M, N, K, r):
    print(f"[case] infinite x M={M} N={N} K={K} r={r}", flush=True)
    c = Positive(M, N, K, r)
    c.x[1, K - 3], c.x[M - 1, 5] = INF, -INF
    W = q.qlora_fp8_weight_quantize(c.W)
    Y, T = q.qlora_fp8_linear_fwd(q.qlora_act8_quantize(c.x, q.ACT8_E5M2), W, c.A, c.B)
    for out in (Y, T) if r else (Y,):
        y = _f64(out)
        assert (y[1] == INF).all() and (y[M - 1] == -INF).all()
        assert np.isfinite(np.delete(y, [1, M - 1], 0)).all()


def _grads(q, base, c, x8, T, drop):
    if base == "fp8":
        return q.qlora_fp8_linear_bwd(c.dY, x8, T, q.qlora_fp8_weight_quantize(c.W), c.A, c.B, 2.0, fmt=q.ACT8_E5M2)
    M, K = x8.shape
    kw = dict(keep_mask=q.qlora_dropout_mask(M, K, 0.2, seed=3, device=device()), p=0.2) if drop else {}
    return q.qlora_linear_bwd_act8(c.dY, x8, T, q.qlora_nf4_quantize(c.W), c.A, c.B, 2.0, **kw)


# dY B^T formed with the adapter's factors (N <= 1024, r <= 64; ranks that
# leave columns of a tile empty) and in a launch of its own
SHAPES = [(3, 256, 384, 8), (40, 192, 256, 16), (40, 1024, 256, 24), (40, 256, 192, 64), (40, 1088, 256, 8),
          (40, 256, 192, 100), (300, 512, 3520, 24), (1030, 192, 4160, 8)]


@pytest.mark.parametrize("base,drop", [("fp8", False), ("nf4", False), ("nf4", True)])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_infinite_upstream(q, M, N, K, r, base, drop):
    """dX's row is that infinity. The float32 gradients that it enters have
    no such value (their factors enter as three terms): not finite."""
    print(f"[case] infinite dY {base} drop={drop} M={M} N={N} K={K} r={r}", flush=True)
    c = Positive(M, N, K, r)
    c.dY[1, N - 2], c.dY[M - 1, 7] = INF, -INF
    x8 = q.qlora_act8_quantize(c.x)
    T = torch.ones(M, r, device=c.x.device)
    dX, dA, dB = (_f64(t) for t in _grads(q, base, c, x8, T, drop))
    assert (dX[1] == INF).all() and (dX[M - 1] == -INF).all()
    assert np.isfinite(np.delete(dX, [1, M - 1], 0)).all()
    assert not np.isfinite(dA).any()
    assert not np.isfinite(dB[:, [N - 2, 7]]).any()
    assert np.isfinite(np.delete(dB, [N - 2, 7], 1)).all()


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_nan_on_the_nf4_base(q, M, N, K, r, drop):
    print(f"[case] NaN, nf4 drop={drop} M={M} N={N} K={K} r={r}", flush=True)
    c = Positive(M, N, K, r)
    x8 = q.qlora_act8_quantize(c.x)
    c.dY[2, 9] = NAN
    dX, dA, dB = (_f64(t) for t in _grads(q, "nf4", c, x8, None, drop))
    assert np.isnan(dX[2]).all() and np.isfinite(np.delete(dX, 2, 0)).all()
    assert np.isnan(dA).all()
    assert np.isnan(dB[:, 9]).all() and np.isfinite(np.delete(dB, 9, 1)).all()


@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_dropped_elements_do_not_spread(q, M, N, K, r, value):
    """An element of x that the mask drops reaches no gradient, whatever it is."""
    print(f"[case] dropped {value} M={M} N={N} K={K} r={r}", flush=True)
    c = Positive(M, N, K, r)
    mask = q.qlora_dropout_mask(M, K, 0.2, seed=3, device=device())
    keep = torch.from_numpy(oracle.unpack_keep(mask.cpu().numpy().view(np.uint32), K).astype(bool)).to(c.x.device)
    st = q.qlora_nf4_quantize(c.W)
    got = []
    for v in (value, 0.5):  # 0.5 and not 0: no block's scale may change
        x = torch.where(keep, c.x, torch.full_like(c.x, v))
        x8 = q.qlora_act8_quantize(x, q.ACT8_E5M2)
        got.append(q.qlora_linear_bwd_act8(c.dY, x8, None, st, c.A, c.B, 2.0, keep_mask=mask, p=0.2))
    for a, b in zip(*got):
        assert torch.equal(a, b) and bool(torch.isfinite(a.float()).all())


# G = 1.998 2^127 is a float32 above the largest bf16 (1.992 2^127)
@pytest.mark.parametrize("base", ["fp8", "nf4"])
@pytest.mark.parametrize("N,r", [(128, 8), (128, 40), (1088, 8)])
def test_factors_above_the_largest_bf16(q, N, r, base):
    M, K = 35, 64
    dev = device()
    bf = dict(dtype=torch.bfloat16, device=dev)
    c = Positive(M, N, K, r)
    c.dY, c.B = torch.zeros(M, N, **bf), torch.zeros(r, N, **bf)
    c.dY[33, 0], c.dY[33, 1] = 1.9921875 * 2.0 ** 63, 1.5 * 2.0 ** 60
    c.B[:, 0], c.B[:, 1] = 2.0 ** 64, 2.0 ** 59
    G = (1.9921875 + 1.5 * 2.0 ** -8) * 2.0 ** 127
    assert G < torch.finfo(torch.float32).max and np.isinf(float(torch.tensor(G, **bf)))
    x = torch.full((M, K), 2.0 ** -10, **bf)
    x8 = q.qlora_act8_quantize(x)
    T = torch.zeros(M, r, device=dev)
    T[33, :] = -G
    c.dY[33, 2] = 2.0 ** -20
    if base == "fp8":
        w = q.qlora_fp8_weight_quantize(c.W)
        _, dA, dB = q.qlora_fp8_linear_bwd(c.dY, x8, T, w, c.A, c.B, 1.0, want_dX=False)
    else:
        _, dA, dB = q.qlora_linear_bwd_act8(c.dY, x8, T, q.qlora_nf4_quantize(c.W), c.A, c.B, 1.0, want_dX=False)
    # one product per element, of 24 bits: exact
    assert np.array_equal(_f64(dA), np.full((K, r), G * 2.0 ** -10))
    assert np.array_equal(_f64(dB)[:, 2], np.full(r, -G * 2.0 ** -20))
    assert np.array_equal(_f64(dB)[:, 3:], np.zeros((r, N - 3)))
