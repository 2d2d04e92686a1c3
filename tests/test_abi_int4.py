"""Argument checks of the entry points on groups of 4-bit codes (CPU only: every
call here is rejected before any HIP call)."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)   # misaligned
EIGHT = ctypes.c_void_p((1 << 20) + 8)
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_finetuning_quantize_amd._lib import LIB
    return LIB


def _quant(lib, W=FAKE, N=4, K=128, ld=128, G=64, codes=FAKE, scales=FAKE, zeros=FAKE):
    return lib.qlora_int4_quantize(W, N, K, ld, G, codes, scales, zeros, None)


def _dequant(lib, W=FAKE, N=4, K=128, ld=128, G=64, codes=FAKE, scales=FAKE, zeros=FAKE):
    return lib.qlora_int4_dequantize(codes, scales, zeros, N, K, G, W, ld, None)


def _fwd(lib, X=FAKE, M=4, ldx=128, codes=FAKE, scales=FAKE, zeros=FAKE, N=4, K=128, G=64, Y=FAKE, dt=0, ldy=4):
    return lib.qlora_int4_linear_fwd(X, M, ldx, codes, scales, zeros, N, K, G, Y, dt, ldy, None)


@pytest.mark.parametrize("f", [_quant, _dequant])
def test_quantize_rejects(lib, f):
    for kw in (dict(W=None), dict(codes=None), dict(scales=None), dict(N=0), dict(K=0), dict(N=-4), dict(ld=127)):
        assert f(lib, **kw) == INVALID, kw
    for kw in (dict(W=ODD), dict(codes=EIGHT), dict(scales=ODD), dict(G=16), dict(G=0), dict(G=256), dict(K=100),
               dict(K=(1 << 21) + 32, ld=1 << 22), dict(N=(1 << 21) + 1), dict(N=1 << 16, K=1 << 16, ld=1 << 16),
               dict(ld=(1 << 32) + 1)):
        assert f(lib, **kw) == UNSUPPORTED, kw


def test_linear_rejects(lib):
    for kw in (dict(X=None), dict(Y=None), dict(codes=None), dict(scales=None), dict(M=0), dict(N=0), dict(K=0),
               dict(ldx=127), dict(ldy=3), dict(dt=2), dict(dt=-1)):
        assert _fwd(lib, **kw) == INVALID, kw
    for kw in (dict(X=EIGHT), dict(Y=ODD), dict(Y=ctypes.c_void_p((1 << 20) + 2), dt=1), dict(codes=EIGHT),
               dict(scales=ODD), dict(G=48), dict(K=48), dict(ldx=132), dict(M=(1 << 20) + 1), dict(ldx=1 << 30),
               dict(M=1 << 20, ldx=1024), dict(N=(1 << 21) + 1, ldy=1 << 22), dict(ldy=(1 << 32) + 1)):
        assert _fwd(lib, **kw) == UNSUPPORTED, kw


def test_binding_rejects():
    import torch

    import bit_quantized_finetuning_quantize_amd as q
    with pytest.raises(q.QloraError):
        q.qlora_int4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))  # not on a GPU
    w = q.Int4Weight(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16), None, (4, 64), 64)
    assert w.nbytes() == 4 * 32 + 8
    with pytest.raises(q.QloraError):
        q.qlora_int4_dequantize(w)
    with pytest.raises(q.QloraError):
        q.qlora_int4_linear_fwd(torch.zeros(1, 64, dtype=torch.bfloat16), w)
