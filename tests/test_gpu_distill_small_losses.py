"""Divergences near 0: a student close to its teacher, and rows that leave little
doubt. The loss is a difference of values near each other, so what it may be off by
is not what they are.

Tolerance. Of the student only the mass off the list, R, is a float32 sum, off by
fewer than 200 roundings and those of the exponents of entries |x| below the largest,
a = 2^-24 (200 + 8 |x|), |x| <= 60 for what counts; the list's masses and everything
after them are off by 1e-12. l = log(R + on) then moves by a p_r and log p_r by a (1 -
p_r), the loss by a |w p_r - q_r| (a p_r without the rest of the teacher's mass),
and its rounding to float32 by 2^-24 of it.
"""

import numpy as np
import pytest
import torch

from oracle import logits as L
from tests.gpu_util import device
from tests.test_gpu_logits import BF, F32, U, _close, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("t", [1.0, 0.7])
@pytest.mark.parametrize("noise", [0.01, 0.3])
@pytest.mark.parametrize("ahead", [0.0, 8.0, 18.0])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,k", [(40, 300, 1), (40, 300, 64), (6, 9001, 20), (3, 100003, 256), (1030, 1000, 32)])
def test_small_losses(q, T, V, k, dtype, ahead, noise, t, rest):
    print(f"[case] small losses {T} x {V} k={k} {dtype} ahead {ahead} noise {noise} t={t} rest={rest}", flush=True)
    g = torch.Generator(device=device())
    g.manual_seed(T + V + k)
    full = torch.randn(T, V, generator=g, device=device()) * 2.5
    full[:, V // 3] += ahead
    Z = full.to(dtype)
    full = Z.float() + torch.randn(T, V, generator=g, device=Z.device) * noise
    values, ids = torch.topk(full, k, dim=1)
    if T > 3 and k > 1:
        ids[1, k // 2:] = -1
        ids[2, k - 1] = ids[2, 0]  # an id twice
    lse = torch.logsumexp(full.double() / t, 1).float() if rest else None
    loss, _ = q.qlora_distill_fwd(Z, ids, values, lse, t)
    z, i, v = _np(Z), _np(ids), _np(values)
    e = _np(lse) if rest else None
    want, st = L.distill(z, t, i, v, e)
    logp, _, _ = L.log_softmax(z, t)
    p_r = np.where(L.listed(i, V), 0.0, np.exp(logp)).sum(axis=1)
    _, q_r, _, _ = L.teacher(i, v, e, t, V)
    a = U * (200 + 8 * 60)
    _close(loss, want, a * np.abs(st[:, 2] * p_r - q_r) + U * np.abs(want) + 1e-12, "loss")
