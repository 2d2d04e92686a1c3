"""Rows of logits whose parts have as many steps as a workgroup takes (16 of 8192),
rows longer than that, which are split however many there are, and a
teacher's logits of another type than the student's. Tolerances: those of
tests/test_gpu_logits.py, whose count of roundings holds for 16 steps to a part
and 32 parts to a row."""

import numpy as np
import pytest
import torch

from oracle import logits as L
from tests.gpu_util import device
from tests.test_gpu_logits import BF, F32, U, _close, _f32, _grad_tol, _np, _rows, _teacher

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


# one part of 16 steps, aligned; two of 9, three of 12 and 32 of 8, unaligned
LONG = [(1024, 131072), (1030, 140001), (1025, 280003), (2, 2097145)]


def _some(T):
    return sorted({0, min(1, T - 1), T // 2, T - 1})


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", LONG)
def test_logprobs(q, T, V, dtype):
    print(f"[case] long logprobs {T} x {V} {dtype}", flush=True)
    Z, g = _rows(T, V, dtype)
    y = torch.randint(0, V, (T,), generator=g, device=Z.device)
    rows = _some(T)
    logp, ent, ids, top, stats = (v[rows] for v in q.qlora_logprobs_fwd(Z, y, n_top=64))
    z = _np(Z[rows])
    ref, m, l = L.log_softmax(z, 1.0)
    H, order = L.entropy(ref), L.top(z, 64)
    assert np.array_equal(_np(ids), order)
    want = L.at_targets(ref, _np(y[rows]))
    bound = U * (200 + 4 * np.abs(l))
    _close(logp, want, bound + 4 * U * np.abs(want), "logp")
    best = np.take_along_axis(ref, order, 1)
    _close(top, best, bound[:, None] + 4 * U * np.abs(best), "top")
    tolH = bound + U * 250 * np.abs(H - l)
    _close(ent, H, tolH, "entropy")
    _close(stats, np.stack([m, l, H], 1), np.stack([0 * l + 1e-300, bound + 4 * U * np.abs(l), tolH], 1), "stats")


def _check_distill(q, Z, ids, values, lse, t, g, rows):
    """Forward and backward, the given rows against float64."""
    k, V = ids.shape[1], Z.shape[1]
    loss, stats = q.qlora_distill_fwd(Z, ids, values, lse, t)
    d = q.qlora_distill_bwd(Z, ids, values, stats, g, t)[rows]
    z, i, v, gr = _np(Z[rows]), _np(ids[rows]), _np(values[rows]), _np(g[rows])
    e = _np(lse[rows]) if lse is not None else None
    want, st = L.distill(z, t, i, v, e)
    logp, _, l = L.log_softmax(z, t)
    off = U * (600 + 6 * k)
    _close(loss[rows], want, off * np.maximum(1.0, st[:, 2]) + 2 * U * np.abs(want), "loss")
    ratio = np.abs(st[:, 2] - st[:, 3])
    tol = np.stack([0 * l + 1e-300, U * (200 + 6 * k + 4 * l), 2 * U * (1 + st[:, 2]),
                    (2 * off + 4 * U) * (1 + ratio + st[:, 2]), 0 * l + 1e-300, 2 * U * (1 + np.abs(st[:, 5]))], 1)
    _close(stats[rows], st, tol, "stats")
    ref = L.distill_grad(z, t, i, v, e, gr)
    qq, _, _, tl = L.teacher(i, v, e, t, V)
    spread = np.zeros_like(ref)
    r, c = np.nonzero(L.valid(i, V))
    np.add.at(spread, (r, i[r, c]), qq[r, c])
    gt = np.abs(gr)[:, None] / t
    tq = U * (30 + 4 * (np.abs(tl)[:, None] + 40)) * spread * gt
    coef = (np.abs(st[:, 2:3]) + np.abs(st[:, 3:4]) * (1 + 12 * (1 + k / 100))) * gt
    _close(d, ref, _grad_tol(ref, np.exp(logp), logp, l, coef, Z.dtype) + tq, "dz")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", LONG)
def test_distill(q, T, V, dtype, rest):
    print(f"[case] long distill {T} x {V} {dtype} rest={rest}", flush=True)
    Z, rng = _rows(T, V, dtype)
    k, t = 256, _f32(1.7)
    ids = torch.randint(0, V, (T, k), generator=rng, device=Z.device)
    ids[:, 0], ids[:, 1] = 0, V - 1  # the ends of the row
    values = torch.gather(Z, 1, ids).float() + torch.randn(T, k, generator=rng, device=Z.device)
    # the list has about a third of the teacher's mass
    lse = torch.logsumexp(values / t, 1) + 1.0 if rest else None
    g = torch.randn(T, generator=rng, device=Z.device)
    _check_distill(q, Z, ids, values, lse, t, g, _some(T))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype,values_dtype", [(F32, BF), (BF, F32), (F32, F32), (BF, BF)])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 7, 3), (3, 513, 65), (2, 8193, 256), (1030, 9001, 20), (2, 100003, 64)])
def test_types_of_a_teachers_logits(q, T, V, k, dtype, values_dtype, rest):
    print(f"[case] distill {T} x {V} k={k} {dtype}, values {values_dtype} rest={rest}", flush=True)
    t = _f32(0.9)
    Z, rng = _rows(T, V, dtype)
    ids, values, lse = _teacher(Z, rng, k, t, rest)
    if T > 1:
        ids[1, k // 2:] = -1
    g = torch.randn(T, generator=rng, device=Z.device)
    _check_distill(q, Z, ids, values.to(values_dtype), lse, t, g, _some(T))
