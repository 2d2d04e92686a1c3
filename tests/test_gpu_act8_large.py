"""8-bit blocks and their products at sizes whose byte offsets pass 32 bits or
come near the calls' limits. Expected values come from smaller calls, which
other tests hold to the oracle, or from float64 sums."""

import pytest
import torch

from tests.gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _same_rows(big, small, times):
    """Every run of len(small) rows of `big` is `small`, bit for bit."""
    view = big.view(times, *small.shape)
    step = 100
    for i in range(0, times, step):
        part = view[i:i + step]
        assert torch.equal(part, small.expand_as(part)), f"runs {i} to {i + len(part)} differ"


def test_rows_past_32_bits(q):
    times, rows, K = 1100, 1000, 2048  # 2.25e9 codes, 4.5e9 bytes of bf16
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    base = torch.randn(rows, K, generator=g, device=dev).to(torch.bfloat16)
    big = base.repeat(times, 1)
    print(f"[case] act8 {big.shape}", flush=True)
    b8, s8 = q.qlora_act8_quantize(big, 1), q.qlora_act8_quantize(base, 1)
    _same_rows(b8.codes, s8.codes, times)
    _same_rows(b8.scales, s8.scales, times)
    _same_rows(q.qlora_act8_dequantize(b8), q.qlora_act8_dequantize(s8), times)
    print("[case] swiglu", flush=True)
    H, h8, g8, u8 = q.qlora_swiglu_act8_fwd(big, big, 1)
    h, hs, gs, us = q.qlora_swiglu_act8_fwd(base, base, 1)
    _same_rows(H, h, times)
    for a, b in ((h8, hs), (g8, gs), (u8, us)):
        _same_rows(a.codes, b.codes, times)
    # in place: dG over dH
    dG, dU = q.qlora_swiglu_act8_bwd(H, g8, u8, dG=H)
    dg, du = q.qlora_swiglu_act8_bwd(h, gs, us)
    _same_rows(dG, dg, times)
    _same_rows(dU, du, times)


def test_product_with_many_rows(q):
    M, N, K = 200_000, 5120, 128  # 2 GiB of output
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    print(f"[case] fp8 product M={M} N={N} K={K}", flush=True)
    x = torch.randn(M, K, generator=g, device=dev).to(torch.bfloat16)
    W = q.qlora_fp8_weight_quantize((torch.randn(N, K, generator=g, device=dev) * 0.1).to(torch.bfloat16))
    Y, _ = q.qlora_fp8_linear_fwd(q.qlora_act8_quantize(x), W)
    for at in (0, 104_857, M - 300):  # around the middle row of the output's bytes too
        part, _ = q.qlora_fp8_linear_fwd(q.qlora_act8_quantize(x[at:at + 300].contiguous()), W)
        # two float32 sums of the same 128 products, rounded to bf16: one place apart at most
        torch.testing.assert_close(Y[at:at + 300].float(), part.float(), rtol=2.0 ** -7, atol=1e-5)


@pytest.mark.parametrize("base", ["fp8", "nf4"])
def test_gradients_over_many_rows(q, base):
    """Positive data, so that a lost run of rows shows. A wave's sum is M / 8 / 32
    instructions for each of three terms, of 32 products each: at most that many
    roundings of 2^-24."""
    M, N, K, r = 524_287, 2048, 64, 8  # dY just below 2^30 elements
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    print(f"[case] gradients M={M} N={N} K={K} r={r} {base}", flush=True)
    dY = torch.rand(M, N, generator=g, device=dev, dtype=torch.bfloat16)
    x8 = q.qlora_act8_quantize(torch.rand(M, K, generator=g, device=dev, dtype=torch.bfloat16))
    A = torch.rand(K, r, generator=g, device=dev, dtype=torch.bfloat16)
    B = torch.rand(r, N, generator=g, device=dev, dtype=torch.bfloat16)
    W = torch.rand(N, K, generator=g, device=dev, dtype=torch.bfloat16) * 0.1
    if base == "fp8":
        w = q.qlora_fp8_weight_quantize(W)
        dX, dA, dB = q.qlora_fp8_linear_bwd(dY, x8, None, w, A, B, 0.5)
    else:
        w = q.qlora_nf4_quantize(W)
        dX, dA, dB = q.qlora_linear_bwd_act8(dY, x8, None, w, A, B, 0.5)
    X = q.qlora_act8_dequantize(x8)
    wA = torch.zeros(K, r, dtype=torch.float64, device=dev)
    wB = torch.zeros(r, N, dtype=torch.float64, device=dev)
    for i in range(0, M, 65536):
        d, x = dY[i:i + 65536].double(), X[i:i + 65536].double()
        wA += 0.5 * x.T @ (d @ B.double().T)
        wB += 0.5 * (x @ A.double()).T @ d
    tol = (M / 8 / 32 + 1) * 3 * 32 * 2.0 ** -24
    for got, want, name in ((dA, wA, "dA"), (dB, wB, "dB")):
        e = ((got.double() - want).abs() / want).max().item()
        print(f"[parity] {name}: {e:.2e} of {tol:.2e}", flush=True)
        assert e <= tol, name
    # dX of the last rows from a call of their own
    tail = slice(M - 256, M)
    t8 = q.qlora_act8_quantize(X[tail].contiguous())
    bwd = q.qlora_fp8_linear_bwd if base == "fp8" else q.qlora_linear_bwd_act8
    part = bwd(dY[tail].contiguous(), t8, None, w, A, B, 0.5)[0]
    torch.testing.assert_close(dX[tail].float(), part.float(), rtol=2.0 ** -6, atol=1e-5)
