"""Rows of logits (TEST INFRASTRUCTURE ONLY).

Definition, in float64, for rows z [T x V] and a temperature t:
  x = z / t,  log p = x - log sum exp x,  H = -sum p log p (0 log 0 = 0);
  log p of a target inside [0, V), else 0;
  the n largest entries of a row, of equal ones the lowest index first, NaN last.
A row whose logits are all -inf: log p = -inf, H = 0, every gradient 0.

Distillation from k teacher logits t_i with ids (ids outside [0, V) are left
out): q_i = exp(t_i / t - L), q_r = max(0, 1 - sum q) the rest; without L the
softmax of the list and no rest. loss = sum q_i (log q_i - log p_i) + q_r (log
q_r - log p_r), p_r the mass off the list, whose term is left out if p_r = 0.

The gradients are those of the formulas: see each function. Pinned by
torch.autograd in float64 and by differences (tests/test_oracle_logits.py).
"""

import numpy as np


def log_softmax(z, t):
    """log p [T x V] and the log sum relative to the row maximum, (m, l)."""
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        m = np.where(np.isnan(z), -np.inf, z).max(axis=1)
        empty = (z == -np.inf).all(axis=1)
        x = (z - np.where(empty, 0.0, m)[:, None]) / t
        l = np.where(empty, 0.0, np.log(np.exp(x).sum(axis=1)))
        logp = np.where(empty[:, None], -np.inf, x - l[:, None])
    return logp, m, l


def entropy(logp):
    with np.errstate(all="ignore"):
        p = np.exp(logp)
        return -np.where(p == 0, 0.0, p * logp).sum(axis=1)


def valid(target, V):
    target = np.asarray(target)
    return (target >= 0) & (target < V)


def at_targets(logp, target):
    ok = valid(target, logp.shape[1])
    rows = np.arange(len(ok))
    return np.where(ok, logp[rows, np.where(ok, target, 0)], 0.0)


def top(z, n):
    """Indices of the n largest entries of each row."""
    z = np.asarray(z, np.float64) + 0.0
    order = np.empty((z.shape[0], n), np.int64)
    for i, row in enumerate(z):
        nan = np.isnan(row)
        rank = np.lexsort((np.arange(len(row)), -np.where(nan, 0.0, row), nan))
        order[i] = rank[:n]
    return order


def logprobs_grad(z, t, target, g, h):
    """(g ([j = target] - p_j) - h p_j (log p_j + H)) / t; g and h [T]."""
    logp, m, l = log_softmax(z, t)
    p = np.exp(logp)
    ok = valid(target, p.shape[1])
    g = np.where(ok, g, 0.0)
    H = entropy(logp)
    with np.errstate(all="ignore"):
        plogp = np.where(p == 0, 0.0, p * logp)
        d = -g[:, None] * p - h[:, None] * (plogp + p * H[:, None])
    d[np.arange(len(ok))[ok], np.asarray(target)[ok]] += g[ok]
    d[(m == -np.inf) & (l == 0)] = 0.0
    d[(g == 0) & (h == 0)] = 0.0
    return d / t


def teacher(ids, values, lse, t, V):
    """(q [T x k], q_r [T], tm, tl) with the entries left out at 0."""
    ok = valid(ids, V)
    v = np.where(ok, np.asarray(values, np.float64), -np.inf)
    tm = v.max(axis=1)
    tm = np.where(tm == -np.inf, 0.0, tm)
    with np.errstate(all="ignore"):
        e = np.exp((v - tm[:, None]) / t)
        if lse is None:
            s = e.sum(axis=1)
            tl = np.where(s > 0, np.log(s), 0.0)
        else:
            tl = np.asarray(lse, np.float64) - tm / t
        q = e * np.exp(-tl)[:, None]
    qr = np.maximum(0.0, 1.0 - q.sum(axis=1)) if lse is not None else np.zeros(len(tm))
    return q, qr, tm, tl


def listed(ids, V):
    mask = np.zeros((len(ids), V), bool)
    r, c = np.nonzero(valid(ids, V))
    mask[r, np.asarray(ids)[r, c]] = True
    return mask


def distill(z, t, ids, values, lse=None):
    """(loss [T], stats [T x 6] = m, l, w, w - q_r / p_r, tm, tl)."""
    logp, m, l = log_softmax(z, t)
    V = logp.shape[1]
    q, qr, tm, tl = teacher(ids, values, lse, t, V)
    ok = valid(ids, V)
    lp = np.where(ok, np.take_along_axis(logp, np.where(ok, ids, 0), axis=1), 0.0)
    with np.errstate(all="ignore"):
        term = np.where(q > 0, q * (np.log(np.where(q > 0, q, 1.0)) - lp), 0.0)
        loss = term.sum(axis=1)
        w = q.sum(axis=1)
        rest = np.where(listed(ids, V), -np.inf, logp)
        top_ = rest.max(axis=1)
        base = np.where(top_ == -np.inf, 0.0, top_)
        logr = np.log(np.exp(rest - base[:, None]).sum(axis=1)) + base
        there = (logr > -np.inf) & (qr > 0)
        ratio = np.where(there, np.exp(np.log(np.where(there, qr, 1.0)) - logr), 0.0)
        loss = loss + np.where(there, qr * (np.log(np.where(there, qr, 1.0)) - logr), 0.0)
    w = w + np.where(there, qr, 0.0)
    return loss, np.stack([m, l, w, w - ratio, tm, tl], axis=1)


def distill_grad(z, t, ids, values, lse, g):
    """g / t (w p_j - q_j) on the list, g / t (w - q_r / p_r) p_j off it."""
    logp, m, l = log_softmax(z, t)
    V = logp.shape[1]
    q, _, _, _ = teacher(ids, values, lse, t, V)
    _, stats = distill(z, t, ids, values, lse)
    mask = listed(ids, V)
    with np.errstate(all="ignore"):
        coef = np.where(mask, stats[:, 2:3], stats[:, 3:4])
        d = np.exp(logp) * coef
    r, c = np.nonzero(valid(ids, V))
    np.subtract.at(d, (r, np.asarray(ids)[r, c]), q[r, c])
    d[(m == -np.inf) & (l == 0)] = 0.0
    with np.errstate(all="ignore"):
        d = d * (np.asarray(g, np.float64) / t)[:, None]
    d[np.asarray(g) == 0] = 0.0
    return d
