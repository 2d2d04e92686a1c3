"""Temperatures that float32 does not hold: 0.7 is off by 1.7e-8 of itself there. A
teacher's log q = t / 0.7 - lse is then off by 2.4e-8 of its logit, 4e-4 at one of
16384, as much again as 25 logits of a usual size are by 1e-6. Tolerances: those
of tests/test_gpu_logits.py."""

import numpy as np
import pytest
import torch

from oracle import logits as L
from tests.gpu_util import device
from tests.test_gpu_logits import BF, F32, U, _close, _np, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


@pytest.mark.parametrize("t", [0.7, 1.3, 2.1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,k", [(5, 300, 8), (3, 40000, 100), (1030, 1000, 20)])
def test_teachers_log_sum_exp(q, T, V, k, dtype, t):
    print(f"[case] temperature {t} {T} x {V} k={k} {dtype}", flush=True)
    Z, rng = _rows(T, V, dtype)
    full = Z.double() + torch.randn(T, V, generator=rng, device=Z.device) + 16384
    values, ids = torch.topk(full.float(), k, dim=1)
    lse = torch.logsumexp(full / t, 1).float()
    loss, stats = q.qlora_distill_fwd(Z, ids, values, lse, t)
    want, st = L.distill(_np(Z), t, _np(ids), _np(values), _np(lse))
    off = U * (600 + 6 * k)
    _close(loss, want, off * np.maximum(1.0, st[:, 2]) + 2 * U * np.abs(want), "loss")
    _close(stats[:, 5], st[:, 5], 2 * U * (1 + np.abs(st[:, 5])), "tl")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("t", [2.0 ** -40, 1e-3, 0.05, 30.0, 1e6, 2.0 ** 40])
@pytest.mark.parametrize("kind", ["plain", "lowest", "far"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,k", [(5, 300, 20), (3, 20000, 100)])
def test_distillation_at_extremes(q, T, V, k, dtype, kind, t, rest):
    """The smallest and largest temperatures, logits of the type's lowest value, and
    logits 1e4 apart: losses up to 1e17."""
    print(f"[case] distill {T} x {V} {dtype} {kind} t={t} rest={rest}", flush=True)
    Z, rng = _rows(T, V, dtype, spread=1e4 if kind == "far" else 1.0)
    Z = Z.clone()
    if kind == "lowest":
        Z[:, ::3] = torch.finfo(dtype).min
    ids = torch.stack([torch.randperm(V, generator=rng, device=Z.device)[:k] for _ in range(T)])
    values = torch.gather(Z, 1, ids).float().clamp(min=-1e30) + torch.randn(T, k, generator=rng, device=Z.device) * 0.1
    lse = torch.logsumexp(values.double() / t, 1).float() if rest else None
    loss, stats = q.qlora_distill_fwd(Z, ids, values, lse, t)
    want, st = L.distill(_np(Z), t, _np(ids), _np(values), _np(lse) if rest else None)
    with np.errstate(over="ignore"):
        want = np.where(np.abs(want) > 3.4e38, np.inf, want)
    off = U * (600 + 6 * k)
    # log q = t_i / t - lse: three roundings of 2^-53 of numbers up to |lse|
    fine = 2.0 ** -50 * (np.abs(_np(lse)) if rest else 0.0)
    _close(loss, want, (off + fine * (1 + np.where(np.isfinite(want), np.abs(want), 0))) * np.maximum(1.0, st[:, 2]) + 2 * U * np.abs(want), "loss")
    d = q.qlora_distill_bwd(Z, ids, values, stats, torch.ones(T, device=Z.device), t)
    assert torch.isfinite(d).all()
