"""Workspace sizes of the linear calls on 8-bit inputs (CPU only)."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
WORKSPACE = -3
SHAPES = [(1, 64, 64, 1), (1, 22016, 8192, 16), (16, 256, 256, 8), (300, 320, 192, 64), (2048, 4096, 11008, 64),
          (4096, 22016, 8192, 128)]


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_finetuning_quantize_amd._lib import LIB
    return LIB


@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_the_8_bit_weight_brings_no_copy_of_itself(lib, M, N, K, r):
    """Only what the call holds: padded factors, float32 factors and partials,
    and in the backward the 8-bit dY. A bf16 weight would be 2 N K bytes more."""
    up = lambda a, b: -(-a // b) * b  # noqa: E731
    r64, Mp = up(r, 64), up(M, 64)
    fwd = max(N, K) * r64 * 2 + Mp * r64 * (2 + 4 + 4) + max(256 * 4096, Mp * r64) * 4 + 1024
    bwd = fwd + M * up(N, 128) + M * up(up(N, 128) // 128, 4)
    for need, backward in ((fwd, 0), (bwd, 1)):
        got = lib.qlora_fp8_workspace_bytes(M, N, K, r, backward)
        assert need <= got <= need + 8 * 256  # each part rounded up to 256 bytes
    assert lib.qlora_act8_workspace_bytes(M, N, K, r) >= 2 * N * K


def test_order_and_rejected_shapes(lib):
    f, big = lib.qlora_fp8_workspace_bytes, lib.qlora_act8_workspace_bytes
    for s in SHAPES + [(16, 100, 100, 0), (1, 1, 1, 0)]:
        assert 0 < f(*s, 0) <= f(*s, 1) <= big(*s)
        assert f(*s, 0) % 256 == 0 and f(*s, 1) % 256 == 0
    for backward in (0, 1):
        sizes = [f(*s, backward) for s in sorted(SHAPES, key=lambda s: s[0] * s[1] * s[2])]
        assert sizes[0] == min(sizes) and sizes[-1] == max(sizes)
        assert f(16, 100, 100, 8, backward) == 0 and f(0, 64, 64, 8, backward) == 0
        assert f(16, 64, 64, 257, backward) == 0 and f(1 << 24, 64, 64, 64, backward) == 0


def test_a_byte_less_is_refused(lib):
    M, N, K, r = 32, 128, 192, 8
    f = lib.qlora_fp8_workspace_bytes

    def fwd(n):
        return lib.qlora_fp8_linear_fwd(FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, M, N, K, r, 1.0, FAKE, FAKE, FAKE, n,
                                        None)

    def bwd(n, dX=FAKE):
        return lib.qlora_fp8_linear_bwd(FAKE, 0, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, M, N, K, r, 1.0, dX,
                                        FAKE, FAKE, FAKE, n, None)

    def nf4(n, dX):
        return lib.qlora_linear_bwd_act8(FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, M, N, K, r, 1.0,
                                         None, 0.0, dX, FAKE, FAKE, FAKE, n, 0, None)

    small, large = f(M, N, K, r, 0), f(M, N, K, r, 1)
    assert fwd(small - 1) == WORKSPACE and bwd(large - 1) == WORKSPACE
    assert bwd(small - 1, None) == WORKSPACE and nf4(small - 1, None) == WORKSPACE
    assert nf4(large, FAKE) == WORKSPACE  # that one holds the bf16 weight

