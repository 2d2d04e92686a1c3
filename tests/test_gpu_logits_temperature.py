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
