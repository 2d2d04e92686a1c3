"""Pins of the oracle's rows of logits: torch.autograd in float64, differences,
closed forms."""

import numpy as np
import pytest
import torch

from oracle import logits as L


def _rows(T, V, seed=0):
    r = np.random.default_rng(seed)
    return r.normal(0, 2.0, (T, V)), r


@pytest.mark.parametrize("t", [1.0, 0.7, 2.0])
def test_logprobs_against_torch(t):
    z, r = _rows(5, 23)
    target = np.array([3, -100, 22, 23, 0])
    g, h = r.normal(size=5), r.normal(size=5)
    Z = torch.tensor(z, requires_grad=True)
    logp = torch.log_softmax(Z / t, dim=1)
    H = -(logp.exp() * logp).sum(1)
    ok = L.valid(target, 23)
    chosen = logp[torch.arange(5), torch.tensor(np.where(ok, target, 0))] * torch.tensor(ok)
    ((chosen * torch.tensor(g)).sum() + (H * torch.tensor(h)).sum()).backward()
    got, m, l = L.log_softmax(z, t)
    assert np.allclose(got, logp.detach().numpy(), rtol=1e-13)
    assert np.allclose(L.entropy(got), H.detach().numpy(), rtol=1e-12)
    assert np.allclose(L.at_targets(got, target), chosen.detach().numpy(), rtol=1e-13)
    assert np.allclose(L.logprobs_grad(z, t, target, g, h), Z.grad.numpy(), rtol=1e-10, atol=1e-14)


def _loss_torch(Z, t, ids, values, lse):
    """One row's divergence, entry by entry."""
    V = Z.shape[0]
    logp = torch.log_softmax(Z / t, dim=0)
    ent = [(int(i), float(v)) for i, v in zip(ids, values) if 0 <= i < V]
    tv = torch.tensor([v / t for _, v in ent], dtype=torch.float64)
    logq = tv - (lse if lse is not None else torch.logsumexp(tv, 0))
    loss = sum((q.exp() * (q - logp[i]) for q, (i, _) in zip(logq, ent)), torch.zeros((), dtype=torch.float64))
    if lse is not None:
        qr = max(0.0, 1.0 - float(logq.exp().sum()))
        off = [j for j in range(V) if j not in {i for i, _ in ent}]
        if qr > 0 and off:
            loss = loss + qr * (np.log(qr) - torch.logsumexp(logp[off], 0))
    return loss


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("t", [1.0, 2.0])
def test_distill_against_torch(t, rest):
    z, r = _rows(6, 19, 1)
    full = z + r.normal(size=z.shape)
    ids = np.argsort(-full, axis=1)[:, :5]
    values = np.take_along_axis(full, ids, 1)
    ids[1, 3:] = -1          # a short list
    ids[2, 4] = ids[2, 0]    # an id twice
    ids[3] = 19              # no entry at all
    ids[4, 0] = 40
    lse = np.log(np.exp(full / t).sum(1)) if rest else None
    if rest:
        lse[5] -= 2.0        # sum q above 1: no rest
    g = r.normal(size=6)
    loss, stats = L.distill(z, t, ids, values, lse)
    grad = L.distill_grad(z, t, ids, values, lse, g)
    for i in range(6):
        Z = torch.tensor(z[i], requires_grad=True)
        want = _loss_torch(Z, t, ids[i], values[i], lse[i] if rest else None)
        assert np.isclose(loss[i], float(want.detach()), rtol=1e-11, atol=1e-13), i
        dz = torch.autograd.grad(want, Z)[0].numpy() if want.requires_grad else np.zeros(19)
        assert np.allclose(grad[i], g[i] * dz, rtol=1e-9, atol=1e-13), i
    assert loss[3] == 0.0 and (grad[3] == 0).all() or rest


def test_gradients_against_differences():
    z, r = _rows(3, 11, 2)
    ids = np.array([[0, 4, 7], [1, 2, -1], [10, 10, 3]])
    values = r.normal(size=(3, 3))
    lse = np.array([1.9, 2.5, 1.7])
    g, h, target = r.normal(size=3), r.normal(size=3), np.array([4, -1, 10])

    def f(z):
        logp, _, _ = L.log_softmax(z, 0.8)
        lp = (g * L.at_targets(logp, target) + h * L.entropy(logp)).sum()
        return lp, (g * L.distill(z, 0.8, ids, values, lse)[0]).sum(), \
            (g * L.distill(z, 0.8, ids, values)[0]).sum()

    want = [L.logprobs_grad(z, 0.8, target, g, h), L.distill_grad(z, 0.8, ids, values, lse, g),
            L.distill_grad(z, 0.8, ids, values, None, g)]
    e = 1e-5
    for i in range(3):
        for j in range(11):
            up, dn = z.copy(), z.copy()
            up[i, j] += e
            dn[i, j] -= e
            for a, b, w in zip(f(up), f(dn), want):
                assert abs((a - b) / (2 * e) - w[i, j]) < 1e-8


def test_special_rows():
    inf = np.inf
    z = np.array([[-inf] * 4, [0.0, -inf, -inf, -inf], [1.0, np.nan, 0, 0], [inf, 0, 0, 0], [2.0, 2, 2, 2]])
    logp, m, l = L.log_softmax(z, 1.0)
    assert (logp[0] == -inf).all() and L.entropy(logp)[0] == 0 and l[0] == 0
    assert logp[1, 0] == 0 and L.entropy(logp)[1] == 0
    assert np.isnan(logp[2]).all() and np.isnan(logp[3, 0])
    assert np.isclose(L.entropy(logp)[4], np.log(4))
    d = L.logprobs_grad(z, 1.0, np.zeros(5, int), np.ones(5), np.ones(5))
    assert (d[0] == 0).all() and np.isfinite(d[1]).all() and np.isnan(d[2]).all()
    # the list covers what the student has: the rest's term is left out
    ids = np.array([[0, 1], [0, 1], [0, 1], [0, 1], [0, 1]])
    loss, st = L.distill(z, 1.0, ids, np.zeros((5, 2)), np.full(5, 2.0))
    assert loss[0] == inf and loss[1] == inf and st[1, 2] == st[1, 3]
    assert L.distill(z[1:2], 1.0, ids[:1, :1], np.zeros((1, 1)))[0] == 0.0


def test_top_order():
    z = np.array([[1.0, 3, np.nan, 3, -np.inf, 0.0, -0.0]])
    assert L.top(z, 7).tolist() == [[1, 3, 0, 5, 6, 4, 2]]
