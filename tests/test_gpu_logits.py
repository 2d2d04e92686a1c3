"""Rows of logits on the GPU against float64.

Tolerances. y = (z - m) c, c = log2(e) / t, has three roundings (the
difference, c, the product), exp2 one unit: 2^-23. A row's sum adds at most 8
products in one chain, 2 + 2 chains, one partial per step of 8192 (16 to a
part), rescaled (3 roundings) each time, then 6 + 4 + 5 joins: fewer than 200
roundings of 2^-24 in all, so |dl| <= 2^-24 (200 + 4 |l|) and with the target's
own three roundings |dlogp| <= 2^-24 (200 + 4 |l| + 4 |logp|). The entropy adds
u / s, both off by as much: 2^-24 (200 + 4 l + 250 (H - l)). A probability is off
by its exponent's error: 2^-24 (250 + 4 (|logp| + l)); bf16 outputs add 2^-8 of
the value. Below 2^-120 the hardware's exp2 gives 0.
"""

import numpy as np
import pytest
import torch

from oracle import logits as L
from tests.gpu_util import device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _np(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _f32(t):
    """A temperature as the library takes it: rounded to float32 (1.7 is off by
    2.8e-8 of itself there, ten of which are 2.8e-7 of a logit of 10)."""
    return float(np.float32(t))


def _rows(T, V, dtype, seed=0, ld=None, spread=3.0):
    g = torch.Generator(device=device())
    g.manual_seed(seed + T * 7919 + V)
    buf = torch.randn(T, ld or V, generator=g, device=device()) * spread
    return buf.to(dtype)[:, :V], g


def _close(got, want, tol, label):
    got, want = _np(got), np.asarray(want, np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(all="ignore"):
        far = np.where(same, 0.0, np.abs(got - want) / tol)
    far = np.where(np.isnan(far), np.inf, far)
    print(f"[parity] {label}: largest error / tolerance {far.max():.3f}", flush=True)
    assert far.max() <= 1.0, (label, np.unravel_index(far.argmax(), far.shape), got.flat[far.argmax()], want.flat[far.argmax()])


def _check_fwd(q, Z, target, t, n, ws=None):
    T, V = Z.shape
    logp, ent, ids, top, stats = q.qlora_logprobs_fwd(Z, target, t, n_top=n, ws=ws)
    z, t = _np(Z), _f32(t)
    ref, m, l = L.log_softmax(z, t)
    with np.errstate(all="ignore"):
        tol = lambda v: U * (200 + 4 * np.abs(l).reshape(-1, *[1] * (v.ndim - 1)) + 4 * np.where(np.isinf(v), 0, np.abs(v)))  # noqa: E731
        want = L.at_targets(ref, _np(target))
        _close(logp, want, tol(want), "logp")
        H = L.entropy(ref)
        tolH = U * (200 + 4 * np.abs(l) + 250 * np.abs(H - l))
        _close(ent, H, tolH, "entropy")
        _close(stats, np.stack([m, l, H], 1), np.stack([0 * l + 1e-300, tol(l), tolH], 1), "stats")
    if n:
        order = L.top(z, n)
        assert np.array_equal(_np(ids), order)
        want = np.take_along_axis(ref, order, 1)
        _close(top, want, tol(want), "top")
    return stats


SHAPES = [(1, 1), (3, 2), (2, 7), (2, 8), (5, 9), (2, 63), (3, 511), (3, 512), (2, 513), (4, 2047), (3, 2049), (2, 4097),
          (2, 8191), (1, 8192), (3, 8193), (7, 16389), (1100, 1000), (1030, 9001), (600, 24580), (2, 100003), (1, 131072),
          (3, 300001), (1, 2097152)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", SHAPES)
def test_logprobs(q, T, V, dtype):
    print(f"[case] logprobs {T} x {V} {dtype}", flush=True)
    Z, g = _rows(T, V, dtype)
    y = torch.randint(0, V, (T,), generator=g, device=Z.device)
    for i, v in enumerate((-100, V, 2 ** 40, -1)):
        if T > i + 1:
            y[i] = v
    for t, n in ((1.0, min(V, 5)), (0.7, min(V, 64)), (2.5, 0), (1.0, 1)):
        _check_fwd(q, Z, y, t, n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,off", [(100, 1), (1001, 3), (9000, 7)])
def test_strided_and_unaligned(q, V, off, dtype):
    print(f"[case] strided {V} {off} {dtype}", flush=True)
    buf, g = _rows(6, V + 50, dtype)
    y = torch.randint(0, V, (6,), generator=g, device=buf.device)
    Z = buf[:, off:off + V]
    _check_fwd(q, Z, y, 1.0, 20)
    _check_fwd(q, Z[1:2], y[1:2], 1.0, 20)


@pytest.mark.parametrize("kind", ["levels", "equal", "up", "down", "few", "lowest", "one", "zeros"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", [(3, 300), (2, 3000), (1025, 2500), (1, 50000), (1025, 9000)])
def test_ties_and_masks(q, T, V, dtype, kind):
    print(f"[case] ties {kind} {T} x {V} {dtype}", flush=True)
    Z, g = _rows(T, V, F32)
    if kind == "levels":
        Z = torch.round(Z / 4)
    elif kind == "equal":
        Z = torch.full_like(Z, 1.5)
    elif kind in ("up", "down"):  # neighbours, few or many of them equal in bf16
        Z = torch.arange(V, device=Z.device, dtype=F32).repeat(T, 1) * (1e-3 if kind == "up" else -1e-3)
    elif kind == "few":           # fewer tokens than alternatives
        Z[torch.rand(T, V, generator=g, device=Z.device) > 4.0 / V] = -INF
        Z[:, V // 2] = 1.0
    elif kind == "lowest":
        Z[:, ::3] = torch.finfo(dtype).min
    elif kind == "one":
        Z = torch.full_like(Z, torch.finfo(dtype).min)
        Z[:, 7] = 0.0
    else:
        Z = torch.where(Z > 0, 0.0, -0.0)
    y = torch.full((T,), 7, device=Z.device)
    _check_fwd(q, Z.to(dtype), y, 1.0, 64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 700, 40000])
def test_special_rows(q, V, dtype):
    """All masked, NaN here and there, all NaN, an infinity, all of the lowest value."""
    print(f"[case] special {V} {dtype}", flush=True)
    Z, _ = _rows(7, V, dtype)
    Z = Z.clone()
    Z[0] = -INF
    Z[1, V // 2] = NAN
    Z[2] = NAN
    Z[3, 1] = INF
    Z[4] = torch.finfo(dtype).min
    Z[5, :V // 2] = NAN
    y = torch.full((7,), 3, device=Z.device)
    stats = _check_fwd(q, Z, y, 1.0, 4)
    one = torch.ones(7, device=Z.device)
    d = _np(q.qlora_logprobs_bwd(Z, y, stats, one, one))
    assert (d[0] == 0).all() and np.isfinite(d[[4, 6]]).all() and np.isnan(d[[1, 2, 3, 5]]).all()
    zero = torch.zeros(7, device=Z.device)
    assert (_np(q.qlora_logprobs_bwd(Z, y, stats, zero, zero)) == 0).all()


def _grad_tol(ref, p, logp, l, coef, dtype, extra=0.0):
    rel = 2.0 ** -8 if dtype is BF else 2 * U
    lp = np.where(p > 0, np.abs(logp), 0.0)
    return rel * np.abs(ref) + U * (250 + 4 * (lp + l[:, None])) * p * coef + U * extra + 2.0 ** -120


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 7), (4, 513), (2, 8193), (1030, 9001), (2, 100003), (520, 24600)])
def test_logprobs_bwd(q, T, V, dtype):
    print(f"[case] logprobs_bwd {T} x {V} {dtype}", flush=True)
    Z, rng = _rows(T, V, dtype)
    Z = Z.clone()
    Z[0, : V // 3] = -INF
    y = torch.randint(V // 2, V, (T,), generator=rng, device=Z.device)
    if T > 2:
        y[1], y[2] = -100, V
    g, h = (torch.randn(T, generator=rng, device=Z.device) for _ in range(2))
    t = _f32(0.8)
    stats = q.qlora_logprobs_fwd(Z, y, t)[4]
    zero = torch.zeros_like(g)
    if T > 3:
        g[3], h[3] = 0.0, 0.0
    z = _np(Z)
    logp, _, l = L.log_softmax(z, t)
    p, H = np.exp(logp), L.entropy(logp)
    for gg, hh in ((g, None), (None, h), (g, h)):
        got = q.qlora_logprobs_bwd(Z, y, stats, gg, hh, t)
        a, b = _np(gg if gg is not None else zero), _np(hh if hh is not None else zero)
        ref = L.logprobs_grad(z, t, _np(y), a, b)
        with np.errstate(all="ignore"):
            coef = (np.abs(a)[:, None] + np.abs(b)[:, None] * (np.where(p > 0, np.abs(logp), 0) + 2 * H[:, None])) / t
            hot = np.zeros_like(p)
            ok = L.valid(_np(y), V)
            hot[np.arange(T)[ok], _np(y)[ok]] = 4 * np.abs(a)[ok] / t
            _close(got, ref, _grad_tol(ref, p, logp, l, coef, dtype, hot), "dz")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_entropy_gradients_leave_masked_logits_at_0(q, dtype):
    """A scaled loss at a low temperature: g / t = 2^40 times p log p is far from
    float32's range, and what is masked has no part of it."""
    Z, _ = _rows(4, 5000, dtype)
    Z = Z.clone()
    Z[:, 1000:] = -INF
    Z[2, 500:] = torch.finfo(dtype).min
    y = torch.full((4,), 3, device=Z.device)
    t = 2.0 ** -10
    stats = q.qlora_logprobs_fwd(Z, y, t)[4]
    h = torch.full((4,), 2.0 ** 30, device=Z.device)
    for g in (None, h):
        d = _np(q.qlora_logprobs_bwd(Z, y, stats, g, h, t))
        assert np.isfinite(d).all() and (d[:, 1000:] == 0).all() and (d[2, 500:] == 0).all()


def _teacher(Z, g, k, t, rest):
    full = Z.float() + torch.randn(Z.shape, generator=g, device=Z.device)
    full = torch.where(torch.isinf(full), torch.full_like(full, -30.0), full)
    values, ids = torch.topk(full, k, dim=1)
    perm = torch.randperm(k, generator=g, device=Z.device)
    lse = torch.logsumexp(full / t, 1).float() if rest else None
    return ids[:, perm].contiguous(), values[:, perm].contiguous(), lse


KD = [(1, 1, 1), (3, 7, 3), (3, 7, 7), (4, 100, 64), (3, 513, 65), (2, 8193, 256), (1030, 9001, 20), (600, 24580, 100),
      (2, 100003, 64), (1, 300001, 33)]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,k", KD)
def test_distill(q, T, V, k, dtype, rest):
    print(f"[case] distill {T} x {V} k={k} {dtype} rest={rest}", flush=True)
    t = _f32(1.7)
    Z, rng = _rows(T, V, dtype)
    ids, values, lse = _teacher(Z, rng, k, t, rest)
    if T > 2:
        ids[1, k // 2:] = -1
        ids[2, k - 1], values[2, 0] = ids[2, 0], -3.0  # an id twice (k > 1)
    if T > 3:
        ids[3] = V  # no entry
    if T > 5 and rest:
        lse[5] -= 1.0  # the list's mass above 1
    if dtype is BF:
        values = values.to(BF)
    z = _np(Z)
    lse64 = _np(lse) if rest else None
    want, st = L.distill(z, t, _np(ids), _np(values), lse64)
    loss, stats = q.qlora_distill_fwd(Z, ids, values, lse, t)
    logp, _, l = L.log_softmax(z, t)
    # q and the row's numbers are float64; the student's two sums join up to k
    # listed entries one by one (6 roundings each)
    off = U * (600 + 6 * k)
    _close(loss, want, off * np.maximum(1.0, st[:, 2]) + 2 * U * np.abs(want), "loss")
    ratio = np.abs(st[:, 2] - st[:, 3])
    tol = np.stack([0 * l + 1e-300, U * (200 + 6 * k + 4 * l), 2 * U * (1 + st[:, 2]), (2 * off + 4 * U) * (1 + ratio + st[:, 2]),
                    0 * l + 1e-300, 2 * U * (1 + np.abs(st[:, 5]))], 1)
    _close(stats, st, tol, "stats")
    g = torch.randn(T, generator=rng, device=Z.device)
    if T > 2:
        g[0] = 0.0
    got = q.qlora_distill_bwd(Z, ids, values, stats, g, t)
    ref = L.distill_grad(z, t, _np(ids), _np(values), lse64, _np(g))
    qq, _, _, tl = L.teacher(_np(ids), _np(values), lse64, t, V)
    spread = np.zeros_like(ref)
    r, c = np.nonzero(L.valid(_np(ids), V))
    np.add.at(spread, (r, _np(ids)[r, c]), qq[r, c])
    p = np.exp(logp)
    gt = np.abs(_np(g))[:, None] / t
    tq = U * (30 + 4 * (np.abs(tl)[:, None] + 40)) * spread * gt
    coef = (np.abs(st[:, 2:3]) + np.abs(st[:, 3:4]) * (1 + 12 * (1 + k / 100))) * gt
    _close(got, ref, _grad_tol(ref, p, logp, l, coef, dtype) + tq, "dz")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_distill_special_rows(q, dtype):
    V, k = 9000, 4
    Z, _ = _rows(6, V, dtype)
    Z = Z.clone()
    ids = torch.arange(k, device=Z.device).repeat(6, 1)
    Z[0] = -INF                # no distribution
    Z[1, k:] = -INF            # no mass off the list
    Z[2, 2] = -INF             # a listed token is masked
    Z[3, 100] = NAN
    Z[4, k:] -= 60             # a tiny mass off the list
    values = torch.tensor([1.0, 0.5, 0.0, -INF], device=Z.device).repeat(6, 1)
    lse = torch.full((6,), 2.2, device=Z.device)
    for le in (lse, None):
        loss, stats = q.qlora_distill_fwd(Z, ids, values, le)
        want, st = L.distill(_np(Z), 1.0, _np(ids), _np(values), _np(le) if le is not None else None)
        _close(loss, want, U * 700 * np.maximum(1, np.where(np.isfinite(want), np.abs(want), 1)), "loss")
        g = torch.ones(6, device=Z.device)
        d = _np(q.qlora_distill_bwd(Z, ids, values, stats, g))
        assert (d[0] == 0).all() and np.isnan(d[3]).all() and np.isfinite(d[[1, 2, 4, 5]]).all()
        assert (d[1, k:] == 0).all()
        ref = L.distill_grad(_np(Z), 1.0, _np(ids), _np(values), _np(le) if le is not None else None, np.ones(6))
        err = np.abs(d - ref) - (2.0 ** -8 if dtype is BF else 2.0 ** -14) * np.abs(ref)
        assert err[[1, 2, 4, 5]].max() <= 2.0 ** -20
        z = q.qlora_distill_bwd(Z, ids, values, stats, torch.zeros(6, device=Z.device))
        assert (_np(z) == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,ldd,off", [(1001, 1100, 0), (9001, 9001, 0), (9001, 9100, 3)])
def test_gradient_places(q, V, ldd, off, dtype):
    """dZ in rows of its own, strided, unaligned, and in Z's place; nothing beside it is written."""
    print(f"[case] places {V} {ldd} {off} {dtype}", flush=True)
    T, k = 5, 16
    Z, rng = _rows(T, V, dtype, ld=V + 13)
    y = torch.randint(0, V, (T,), generator=rng, device=Z.device)
    ids, values, lse = _teacher(Z, rng, k, 1.0, True)
    g = torch.randn(T, generator=rng, device=Z.device)
    s1 = q.qlora_logprobs_fwd(Z, y)[4]
    _, s2 = q.qlora_distill_fwd(Z, ids, values, lse)
    calls = [lambda z, d: q.qlora_logprobs_bwd(z, y, s1, g, g, dZ=d),
             lambda z, d: q.qlora_distill_bwd(z, ids, values, s2, g, dZ=d)]
    for f in calls:
        want = f(Z, None)
        buf = torch.full((T + 1, ldd + off), 77.0, dtype=dtype, device=Z.device)
        out = f(Z, buf[:T, off:off + V])
        assert torch.equal(out, want)
        rest = buf.clone()
        rest[:T, off:off + V] = 77.0
        assert (rest == 77.0).all()
        own = torch.empty(T, V + 13, dtype=dtype, device=Z.device)
        own.fill_(5.0)
        own[:, :V] = Z
        f(own[:, :V], own[:, :V])
        assert torch.equal(own[:, :V], want) and (own[:, V:] == 5.0).all()


def test_same_bits_every_time_and_on_other_streams(q):
    Z, rng = _rows(3, 120000, BF)
    y = torch.randint(0, 120000, (3,), generator=rng, device=Z.device)
    ids, values, lse = _teacher(Z, rng, 100, 1.0, True)
    ws = q.logits_workspace(3, 120000, 20, Z.device)
    first = None
    for i in range(6):
        ws.random_(0, 256)  # whatever it held before
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            a = q.qlora_logprobs_fwd(Z, y, n_top=20, ws=ws)
            b = q.qlora_distill_fwd(Z, ids, values, lse, ws=ws)
        torch.cuda.current_stream().wait_stream(s)
        got = [t.clone() for t in (*a, *b)]
        if first is None:
            first = got
        assert all(torch.equal(u, v) for u, v in zip(first, got))


def test_workspaces_side_by_side(q):
    """Two streams at once, each with its own workspace."""
    Z, rng = _rows(4, 90000, BF)
    want = q.qlora_logprobs_fwd(Z, n_top=8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(q.qlora_logprobs_fwd(Z, n_top=8))
    torch.cuda.synchronize()
    for a in got:
        assert all(torch.equal(u, v) for u, v in zip(a[1:], want[1:]))


def test_graphs_that_share_a_workspace(q):
    T, V, k = 2, 70000, 32
    Z, rng = _rows(T, V, BF)
    Z = Z.clone()
    y = torch.randint(0, V, (T,), generator=rng, device=Z.device)
    ids, values, lse = _teacher(Z, rng, k, 1.0, True)
    g = torch.randn(T, generator=rng, device=Z.device)
    ws = q.logits_workspace(T, V, 20, Z.device)

    def scores():
        return q.qlora_logprobs_fwd(Z, y, n_top=20, ws=ws)

    def step():
        loss, st = q.qlora_distill_fwd(Z, ids, values, lse, ws=ws)
        return loss, st, q.qlora_distill_bwd(Z, ids, values, st, g)

    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        scores(), step()
    torch.cuda.current_stream().wait_stream(side)
    for f in (scores, step):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = f()
        graphs.append((gr, out, f))
    for i in range(5):
        Z.copy_(torch.randn(T, V, generator=rng, device=Z.device) * (1 + i))
        for gr, out, f in graphs + graphs[::-1]:
            gr.replay()
            torch.cuda.synchronize()
            want = f()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_gradients_by_differences(q):
    """Steps of the GPU's own forward passes, float32 logits."""
    T, V, k, t = 2, 40, 6, 1.3
    Z, rng = _rows(T, V, F32, spread=1.0)
    Z = Z.contiguous()
    ids, values, lse = _teacher(Z, rng, k, t, True)
    y = torch.tensor([3, 17], device=Z.device)
    st = q.qlora_logprobs_fwd(Z, y, t)[4]
    _, sd = q.qlora_distill_fwd(Z, ids, values, lse, t)
    one = torch.ones(T, device=Z.device)
    d1, d2 = q.qlora_logprobs_bwd(Z, y, st, one, one, t), q.qlora_distill_bwd(Z, ids, values, sd, one, t)
    e = 2.0 ** -6
    for j in range(V):
        f = []
        for s in (e, -e):
            z = Z.clone()
            z[:, j] += s
            lp, H, *_ = q.qlora_logprobs_fwd(z, y, t)
            f.append((_np(lp) + _np(H), _np(q.qlora_distill_fwd(z, ids, values, lse, t)[0])))
        # e^2 / 6 of a third derivative (at most 4) and 2 x 2^-18 of a value over 2 e
        tol = e * e + 2.0 ** -18 / e
        for i, d in enumerate((d1, d2)):
            assert np.abs((f[0][i] - f[1][i]) / (2 * e) - _np(d)[:, j]).max() <= tol


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_that_outgrow_the_caches(q, dtype):
    """Above 128 MiB logits and gradients pass the caches: the same bits as in two
    halves that do not."""
    T, V, k = (2100, 40003, 40) if dtype is BF else (2050, 20003, 40)
    Z, rng = _rows(T, V, dtype)
    assert T * V * Z.element_size() > 128 << 20 > T // 2 * V * Z.element_size()
    y = torch.randint(-1, V, (T,), generator=rng, device=Z.device)
    ids = torch.randint(0, V, (T, k), generator=rng, device=Z.device)
    values = torch.randn(T, k, generator=rng, device=Z.device) * 3
    lse = torch.full((T,), 9.0, device=Z.device)
    g, h = (torch.randn(T, generator=rng, device=Z.device) for _ in range(2))

    def run(a, b):
        z = Z[a:b]
        s = q.qlora_logprobs_fwd(z, y[a:b], 0.9, n_top=9)
        d = q.qlora_distill_fwd(z, ids[a:b], values[a:b], lse[a:b], 0.9)
        e = q.qlora_distill_fwd(z, ids[a:b], values[a:b], None, 0.9)
        return [*s, *d, *e, q.qlora_logprobs_bwd(z, y[a:b], s[4], g[a:b], h[a:b], 0.9),
                q.qlora_distill_bwd(z, ids[a:b], values[a:b], d[1], g[a:b], 0.9)]

    whole, first, second = run(0, T), run(0, T // 2), run(T // 2, T)
    for w, a, b in zip(whole, first, second):
        assert torch.equal(w, torch.cat([a, b]))


def test_many_rows_past_32_bit_offsets(q):
    """Rows beyond 4 GiB of logits, checked by themselves."""
    T, V = 40000, 60000
    Z = torch.empty(T, V, dtype=BF, device=device())
    Z.normal_(0, 2)
    y = torch.full((T,), 11, device=Z.device)
    y[-1] = V - 1
    logp, ent, ids, top, stats = q.qlora_logprobs_fwd(Z, y, n_top=3)
    assert T * V > 2 ** 31
    for r in (0, T // 2, T - 1):
        one = q.qlora_logprobs_fwd(Z[r:r + 1], y[r:r + 1], n_top=3)
        for a, b in zip((logp, ent, top, stats), (one[0], one[1], one[3], one[4])):
            assert torch.allclose(a[r:r + 1], b, rtol=1e-5, atol=1e-5)
        assert torch.equal(ids[r:r + 1], one[2])
    g = torch.ones(T, device=Z.device)
    want = q.qlora_logprobs_bwd(Z[T - 1:], y[T - 1:], stats[T - 1:], g[T - 1:])
    q.qlora_logprobs_bwd(Z, y, stats, g, dZ=Z)
    assert torch.equal(Z[T - 1:], want)


def test_the_most_rows(q):
    """2^23 rows, a workgroup to each, of one and of five logits."""
    T = 1 << 23
    for V in (1, 5):
        print(f"[case] {T} x {V}", flush=True)
        Z, _ = _rows(1 << 13, V, BF)
        few = q.qlora_logprobs_fwd(Z, n_top=1)
        Z = Z.repeat(1 << 10, 1)
        many = q.qlora_logprobs_fwd(Z, n_top=1)
        for a, b in zip(few[1:], many[1:]):
            assert torch.equal(a.repeat(1 << 10, *[1] * (a.dim() - 1)), b)
        h = torch.ones(T, device=Z.device)
        d = q.qlora_logprobs_bwd(Z, None, many[4], None, h)
        assert torch.equal(d.view(1 << 10, 1 << 13, V), d[:1 << 13].expand(1 << 10, -1, -1))
        assert torch.equal(d[:1 << 13], q.qlora_logprobs_bwd(Z[:1 << 13], None, few[4], None, h[:1 << 13]))


def test_distillation_past_32_bit_offsets(q):
    """Rows beyond 4 GiB of logits and their gradients, checked by themselves."""
    T, V, k = 40000, 60000, 30
    Z = torch.empty(T, V, dtype=BF, device=device())
    Z.normal_(0, 2)
    ids = torch.randint(0, V, (T, k), device=Z.device)
    values = torch.randn(T, k, device=Z.device)
    lse = torch.full((T,), 12.0, device=Z.device)
    g = torch.ones(T, device=Z.device)
    loss, stats = q.qlora_distill_fwd(Z, ids, values, lse)
    for r in (0, T // 2, T - 1):
        one = slice(r, r + 1)
        a, b = q.qlora_distill_fwd(Z[one], ids[one], values[one], lse[one])
        # one row is split into parts: both within 2^-24 (600 + 6 k) of the exact loss, as above
        assert torch.allclose(loss[one], a, rtol=1e-4, atol=1e-4) and torch.allclose(stats[one], b, rtol=1e-4, atol=1e-4)
    last = slice(T - 1, T)
    want = q.qlora_distill_bwd(Z[last], ids[last], values[last], stats[last], g[last])
    q.qlora_distill_bwd(Z, ids, values, stats, g, dZ=Z)
    assert torch.equal(Z[last], want)


def test_calls_of_several_threads(q):
    """Host threads on streams of their own, each call with its own workspace."""
    import threading
    Z, rng = _rows(3, 70000, BF)
    ids, values, lse = _teacher(Z, rng, 16, 1.0, True)
    y = torch.tensor([5, 6, 7], device=Z.device)
    w = q.qlora_int4_quantize((torch.randn(9000, 512, generator=rng, device=Z.device) * 0.02).to(BF))
    x = torch.randn(60, 512, generator=rng, device=Z.device).to(BF)

    def calls():
        a = q.qlora_logprobs_fwd(Z, y, n_top=9)
        b = q.qlora_distill_fwd(Z, ids, values, lse)
        # all sizes of a workgroup's LDS
        c = [q.qlora_int4_linear_fwd(x[:m], w) for m in (1, 7, 16, 20, 48, 60)]
        return [*a, *b, *c]

    want = calls()
    torch.cuda.synchronize()
    bad = []

    def run():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = calls()
                    s.synchronize()
                    assert all(torch.equal(u, v) for u, v in zip(got, want))
        except BaseException as e:  # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=run) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
