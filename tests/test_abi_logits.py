"""Argument checks of the entry points on rows of logits (CPU only: every call
here is rejected before any HIP call)."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(1 << 20)       # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)  # misaligned
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_finetuning_quantize_amd._lib import LIB
    return LIB


def _lp(lib, Z=FAKE, dt=0, T=4, V=100, ld=100, y=FAKE, t=1.0, logp=FAKE, ent=FAKE, n=5, ids=FAKE, top=FAKE,
        stats=FAKE, ws=FAKE, wsb=1 << 40):
    return lib.qlora_logprobs_fwd(Z, dt, T, V, ld, y, t, logp, ent, n, ids, top, stats, ws, wsb, None)


def _lp_bwd(lib, Z=FAKE, dt=0, T=4, V=100, ld=100, y=FAKE, t=1.0, stats=FAKE, g=FAKE, h=FAKE, dZ=FAKE, ldd=100):
    return lib.qlora_logprobs_bwd(Z, dt, T, V, ld, y, t, stats, g, h, dZ, ldd, None)


def _kd(lib, Z=FAKE, dt=0, T=4, V=100, ld=100, ids=FAKE, val=FAKE, vt=1, k=8, lse=FAKE, t=1.0, loss=FAKE, stats=FAKE,
        ws=FAKE, wsb=1 << 40):
    return lib.qlora_distill_fwd(Z, dt, T, V, ld, ids, val, vt, k, lse, t, loss, stats, ws, wsb, None)


def _kd_bwd(lib, Z=FAKE, dt=0, T=4, V=100, ld=100, ids=FAKE, val=FAKE, vt=1, k=8, t=1.0, stats=FAKE, g=FAKE, dZ=FAKE,
            ldd=100):
    return lib.qlora_distill_bwd(Z, dt, T, V, ld, ids, val, vt, k, t, stats, g, dZ, ldd, None)


@pytest.mark.parametrize("f", [_lp, _lp_bwd, _kd, _kd_bwd])
def test_rows_rejected(lib, f):
    for kw in (dict(Z=None), dict(T=0), dict(T=-1), dict(V=0, n=0) if f is _lp else dict(V=0), dict(ld=99), dict(dt=2),
               dict(dt=-1), dict(t=0.0), dict(t=-1.0), dict(t=INF), dict(t=NAN)):
        assert f(lib, **kw) == INVALID, kw
    for kw in (dict(Z=ODD), dict(dt=1, Z=ctypes.c_void_p((1 << 20) + 2)), dict(T=(1 << 23) + 1),
               dict(V=(1 << 21) + 1, ld=1 << 22, **({"ldd": 1 << 22} if "bwd" in f.__name__ else {})),
               dict(ld=(1 << 32) + 1), dict(t=1e-13), dict(t=2e12)):
        assert f(lib, **kw) == UNSUPPORTED, kw


def test_logprobs_rejected(lib):
    for kw in (dict(y=None), dict(n=-1), dict(n=101), dict(ids=None), dict(top=None), dict(n=0),
               dict(n=0, ids=None), dict(n=0, ids=None, top=None, logp=None, ent=None, stats=None)):
        assert _lp(lib, **kw) == INVALID, kw
    for kw in (dict(n=65), dict(y=ODD), dict(ids=ctypes.c_void_p((1 << 20) + 4)), dict(top=ODD), dict(logp=ODD),
               dict(ent=ODD), dict(stats=ODD), dict(ws=ODD)):
        assert _lp(lib, **kw) == UNSUPPORTED, kw
    assert _lp(lib, ws=None) == WORKSPACE and _lp(lib, wsb=255) == WORKSPACE
    need = lib.qlora_logits_workspace_bytes(4, 100000, 5)
    assert _lp(lib, V=100000, ld=100000, wsb=need - 1) == WORKSPACE


def test_logprobs_bwd_rejected(lib):
    for kw in (dict(stats=None), dict(g=None, h=None), dict(y=None), dict(dZ=None), dict(ldd=99)):
        assert _lp_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(stats=ODD), dict(g=ODD), dict(h=ODD), dict(y=ODD), dict(dZ=ODD), dict(ldd=(1 << 32) + 1)):
        assert _lp_bwd(lib, **kw) == UNSUPPORTED, kw


def test_distill_rejected(lib):
    for kw in (dict(ids=None), dict(val=None), dict(vt=2), dict(k=0), dict(k=-1), dict(loss=None)):
        assert _kd(lib, **kw) == INVALID, kw
    for kw in (dict(k=257), dict(ids=ODD), dict(val=ODD), dict(val=ctypes.c_void_p((1 << 20) + 2)), dict(lse=ODD),
               dict(loss=ODD), dict(stats=ODD), dict(ws=ODD)):
        assert _kd(lib, **kw) == UNSUPPORTED, kw
    assert _kd(lib, ws=None) == WORKSPACE and _kd(lib, wsb=0) == WORKSPACE


def test_distill_bwd_rejected(lib):
    for kw in (dict(ids=None), dict(val=None), dict(vt=-1), dict(k=0), dict(stats=None), dict(g=None), dict(dZ=None),
               dict(ldd=99)):
        assert _kd_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(k=257), dict(ids=ODD), dict(val=ODD), dict(stats=ODD), dict(g=ODD), dict(dZ=ODD)):
        assert _kd_bwd(lib, **kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("f", [_lp_bwd, _kd_bwd])
def test_in_place_needs_the_same_rows(lib, f):
    assert f(lib, ldd=101) == INVALID and f(lib, ld=101) == INVALID


def test_workspace_query(lib):
    f = lib.qlora_logits_workspace_bytes
    for T, V, n in ((0, 10, 0), (1, 0, 0), (1, 10, 11), (1, 100, 65), (1, 10, -1), ((1 << 23) + 1, 10, 0),
                    (1, (1 << 21) + 1, 0)):
        assert f(T, V, n) == 0, (T, V, n)
    assert f(1, 1, 1) > 0 and f(1 << 23, 1 << 21, 64) > 0
    assert f(1, 131072, 20) > f(1, 131072, 0) > f(1, 8192, 0) > 0


def test_binding_rejects():
    import torch

    import bit_quantized_finetuning_quantize_amd as q
    Z = torch.zeros(2, 8)  # not on a GPU
    with pytest.raises(q.QloraError):
        q.qlora_logprobs_fwd(Z)
    with pytest.raises(q.QloraError):
        q.qlora_logprobs_bwd(Z, None, torch.zeros(2, 3), g_entropy=torch.zeros(2))
    ids = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(q.QloraError):
        q.qlora_distill_fwd(Z, ids, torch.zeros(2, 3))
    with pytest.raises(q.QloraError):
        q.qlora_distill_bwd(Z, ids, torch.zeros(2, 3), torch.zeros(2, 6), torch.zeros(2))
    with pytest.raises(q.QloraError):
        q.logits_workspace(1, 10, 11, "cpu")
