"""Argument checks of the 8-bit block entry points (CPU only: every call here
is rejected before any HIP call)."""

import ctypes

import pytest

from oracle import act8

FAKE = ctypes.c_void_p(1 << 20)       # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)  # misaligned
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_finetuning_quantize_amd._lib import LIB
    return LIB


@pytest.mark.parametrize("K", [0, 1, 127, 128, 129, 512, 513, 4096, 11008])
def test_sizes(lib, K):
    import bit_quantized_finetuning_quantize_amd as q
    assert lib.qlora_act8_row_bytes(K) == act8.row_bytes(K) == q.act8_row_bytes(K)
    assert lib.qlora_act8_scale_row_bytes(K) == act8.scale_row_bytes(K) == q.act8_scale_row_bytes(K)
    assert lib.qlora_act8_row_bytes(-1) == -1 and lib.qlora_act8_scale_row_bytes(-1) == -1


def _quant(lib, X=FAKE, M=4, K=128, ld=128, fmt=0, codes=FAKE, scales=FAKE):
    return lib.qlora_act8_quantize(X, M, K, ld, fmt, codes, scales, None)


def _dequant(lib, X=FAKE, M=4, K=128, ld=128, fmt=0, codes=FAKE, scales=FAKE):
    return lib.qlora_act8_dequantize(codes, scales, M, K, fmt, X, ld, None)


@pytest.mark.parametrize("f", [_quant, _dequant])
def test_quantize_rejects(lib, f):
    for kw in (dict(X=None), dict(codes=None), dict(scales=None), dict(M=0), dict(K=0), dict(M=-1),
               dict(ld=127), dict(fmt=2), dict(fmt=-1)):
        assert f(lib, **kw) == INVALID, kw
    for kw in (dict(X=ODD), dict(codes=ODD), dict(scales=ODD), dict(M=(1 << 30) + 1),
               dict(K=(1 << 21) + 1, ld=1 << 22), dict(M=1 << 30, K=129, ld=129)):
        assert f(lib, **kw) == UNSUPPORTED, kw


def _swiglu(lib, G=FAKE, U=FAKE, M=4, F=128, ldg=128, ldu=128, fmt=0, H=FAKE, ldh=128,
            h=(FAKE, FAKE), g=(FAKE, FAKE), u=(FAKE, FAKE)):
    return lib.qlora_swiglu_act8_fwd(G, ldg, U, ldu, M, F, fmt, H, ldh, *h, *g, *u, None)


def test_swiglu_fwd_rejects(lib):
    none = (None, None)
    for kw in (dict(G=None), dict(U=None), dict(M=0), dict(F=0), dict(ldg=1), dict(ldu=1), dict(ldh=1),
               dict(fmt=2), dict(h=(FAKE, None)), dict(g=(None, FAKE)), dict(u=(FAKE, None)),
               dict(H=None, h=none, g=none, u=none)):
        assert _swiglu(lib, **kw) == INVALID, kw
    for kw in (dict(G=ODD), dict(U=ODD), dict(H=ODD), dict(h=(ODD, FAKE)), dict(u=(FAKE, ODD))):
        assert _swiglu(lib, **kw) == UNSUPPORTED, kw


def test_swiglu_bwd_rejects(lib):
    def f(dH=FAKE, g=(FAKE, FAKE), u=(FAKE, FAKE), M=4, F=128, lddh=128, fmt=0, dG=FAKE, lddg=128,
          dU=FAKE, lddu=128):
        return lib.qlora_swiglu_act8_bwd(dH, lddh, *g, *u, M, F, fmt, dG, lddg, dU, lddu, None)
    for kw in (dict(dH=None), dict(dG=None), dict(dU=None), dict(g=(None, FAKE)), dict(u=(FAKE, None)),
               dict(M=0), dict(F=-3), dict(lddh=127), dict(lddg=127), dict(lddu=127), dict(fmt=7)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(dH=ODD), dict(dG=ODD), dict(dU=ODD), dict(g=(ODD, FAKE))):
        assert f(**kw) == UNSUPPORTED, kw


def test_weight_quantize_rejects(lib):
    f = lib.qlora_fp8_weight_quantize
    assert f(None, 4, 4, FAKE, FAKE, None, None, None) == INVALID
    assert f(FAKE, 0, 4, FAKE, FAKE, None, None, None) == INVALID
    assert f(FAKE, 4, 4, None, FAKE, None, None, None) == INVALID
    assert f(FAKE, 4, 4, FAKE, FAKE, FAKE, None, None) == INVALID
    assert f(FAKE, 4, 4, ODD, FAKE, None, None, None) == UNSUPPORTED
    assert f(FAKE, (1 << 21) + 1, 4, FAKE, FAKE, None, None, None) == UNSUPPORTED
    assert f(FAKE, 1 << 17, 1 << 15, FAKE, FAKE, None, None, None) == UNSUPPORTED


def _bwd(lib, dY=FAKE, x=(FAKE, FAKE), fmt=0, T=FAKE, codes=FAKE, s2=FAKE, A=FAKE, B=FAKE, M=32, N=128,
         K=128, r=8, mask=None, p=0.0, dX=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, wsb=1 << 32, st=0):
    return lib.qlora_linear_bwd_act8(dY, *x, fmt, T, codes, FAKE, s2, A, B, M, N, K, r, 1.0, mask, p, dX,
                                     dA, dB, ws, wsb, st, None)


def test_linear_bwd_act8_rejects(lib):
    for kw in (dict(dY=None), dict(x=(None, FAKE)), dict(x=(FAKE, None)), dict(fmt=2), dict(A=None),
               dict(B=None), dict(dA=None), dict(dB=None), dict(codes=None), dict(s2=None), dict(M=0),
               dict(st=4), dict(mask=FAKE, p=1.0), dict(mask=FAKE, p=-0.1)):
        assert _bwd(lib, **kw) == INVALID, kw
    for kw in (dict(K=100), dict(N=100), dict(r=0), dict(r=257), dict(r=-1), dict(dY=ODD), dict(B=ODD),
               dict(A=ODD), dict(T=ODD), dict(dX=ODD), dict(dA=ODD), dict(codes=ODD), dict(x=(ODD, FAKE)),
               dict(mask=ODD, p=0.1), dict(mask=FAKE, p=0.1, r=193),
               dict(M=1 << 20, N=1024), dict(M=1 << 24, N=64, K=64), dict(ws=ODD)):
        assert _bwd(lib, **kw) == UNSUPPORTED, kw
    assert _bwd(lib, ws=None) == WORKSPACE
    need = lib.qlora_act8_workspace_bytes(32, 128, 128, 8)
    assert need > 0 and _bwd(lib, wsb=need - 1) == WORKSPACE


def _fwd8(lib, x=(FAKE, FAKE), fmt=0, w=(FAKE, FAKE), A=FAKE, B=FAKE, M=32, N=128, K=128, r=8, Y=FAKE,
          T=FAKE, ws=FAKE, wsb=1 << 32):
    return lib.qlora_fp8_linear_fwd(*x, fmt, *w, A, B, M, N, K, r, 1.0, Y, T, ws, wsb, None)


def test_fp8_linear_fwd_rejects(lib):
    plain = dict(A=None, B=None, T=None, r=0)
    for kw in (dict(x=(None, FAKE)), dict(w=(FAKE, None)), dict(fmt=3), dict(A=None), dict(B=None),
               dict(Y=None), dict(r=0), dict(M=0), dict(N=0), dict(K=-5), dict(plain, A=FAKE),
               dict(plain, T=FAKE), dict(plain, K=0)):
        assert _fwd8(lib, **kw) == INVALID, kw
    for kw in (dict(K=100), dict(N=100), dict(r=257), dict(Y=ODD), dict(T=ODD), dict(B=ODD), dict(x=(ODD, FAKE)),
               dict(plain, N=(1 << 21) + 1), dict(plain, M=1 << 23, N=100),
               dict(plain, M=1, N=1 << 21, K=1 << 11), dict(ws=ODD)):
        assert _fwd8(lib, **kw) == UNSUPPORTED, kw
    assert _fwd8(lib, ws=None) == WORKSPACE and _fwd8(lib, wsb=8) == WORKSPACE


def _bwd8(lib, dY=FAKE, df=0, x=(FAKE, FAKE), fmt=0, T=FAKE, w=(FAKE, FAKE), A=FAKE, B=FAKE, M=32, N=128,
          K=128, r=8, dX=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, wsb=1 << 32):
    return lib.qlora_fp8_linear_bwd(dY, df, *x, fmt, T, *w, A, B, M, N, K, r, 1.0, dX, dA, dB, ws, wsb, None)


def test_fp8_linear_bwd_rejects(lib):
    plain = dict(A=None, B=None, T=None, dA=None, dB=None, r=0, x=(None, None))
    for kw in (dict(dY=None), dict(df=2), dict(fmt=2), dict(x=(None, FAKE)), dict(w=(None, FAKE)),
               dict(A=None), dict(dA=None), dict(dB=None), dict(plain, dX=None), dict(plain, dA=FAKE),
               dict(plain, T=FAKE), dict(M=0)):
        assert _bwd8(lib, **kw) == INVALID, kw
    for kw in (dict(N=100), dict(r=300), dict(dY=ODD), dict(dX=ODD), dict(dB=ODD), dict(w=(ODD, FAKE)),
               dict(plain, dY=ODD)):
        assert _bwd8(lib, **kw) == UNSUPPORTED, kw
    assert _bwd8(lib, wsb=0) == WORKSPACE


def test_workspace_query(lib):
    f = lib.qlora_act8_workspace_bytes
    assert f(16, 100, 100, 0) > 0 and f(16, 100, 100, 8) == 0 and f(0, 64, 64, 8) == 0
    assert f(1 << 24, 64, 64, 64) == 0  # M K = 2^30
    shapes = [(1, 64, 64, 1), (16, 256, 256, 8), (300, 320, 192, 64), (2048, 4096, 11008, 64),
              (4096, 22016, 8192, 128)]
    sizes = [f(*s) for s in shapes]
    assert sizes == sorted(sizes)
