"""Gradients over many rows, one region of them at a time: every other row is
zero, so that the region is the whole sum and a lost row shows."""

import pytest
import torch

from tests.gpu_util import device

pytestmark = pytest.mark.gpu

M, N, K, R = 524_287, 2048, 64, 8  # dY just below 2^30 elements and 2 GiB
REGIONS = {
    "first rows": (0, 8),
    "around 2^30 bytes of dY": (262_140, 262_148),
    "a wave's last turn": (M // 32 // 8 * 8 * 32, M // 32 // 8 * 8 * 32 + 16),
    "last whole block": (M - 31 - 32, M - 31 - 28),
    "odd last block": (M - 31, M - 23),
    "last row": (M - 1, M),
}


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


@pytest.mark.parametrize("base", ["fp8", "nf4"])
def test_each_region_counts(q, base):
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    rand = lambda *s: torch.rand(s, generator=g, device=dev) + 0.5  # noqa: E731
    A, B = rand(K, R).to(torch.bfloat16), rand(R, N).to(torch.bfloat16)
    W = (rand(N, K) * 0.1).to(torch.bfloat16)
    w = q.qlora_fp8_weight_quantize(W) if base == "fp8" else q.qlora_nf4_quantize(W)
    bwd = q.qlora_fp8_linear_bwd if base == "fp8" else q.qlora_linear_bwd_act8
    dY = torch.zeros(M, N, dtype=torch.bfloat16, device=dev)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    ws = q.act8_workspace(M, N, K, R, dev)
    for name, (lo, hi) in REGIONS.items():
        print(f"[case] {base}: {name}, rows {lo} to {hi}", flush=True)
        dY[lo:hi] = rand(hi - lo, N).to(torch.bfloat16)
        x[lo:hi] = rand(hi - lo, K).to(torch.bfloat16)
        x8 = q.qlora_act8_quantize(x)
        X, d = q.qlora_act8_dequantize(x8)[lo:hi].double(), dY[lo:hi].double()
        T = torch.zeros(M, R, device=dev)
        T[lo:hi] = (X @ A.double()).float()
        _, dA, dB = bwd(dY, x8, T, w, A, B, 0.5, want_dX=False, ws=ws)
        wA = 0.5 * (X.T @ (d @ B.double().T))
        wB = 0.5 * (T[lo:hi].double().T @ d)
        # float32 sums of positive terms, zeros adding nothing: G's of 2048 in
        # pieces of 64, then 16 rows at most and the waves' and terms' 24
        tol = (N / 64 + 64 + 16 + 24) * 2.0 ** -24
        for got, want, what in ((dA, wA, "dA"), (dB, wB, "dB")):
            e = ((got.double() - want).abs() / want).max().item()
            print(f"[parity] {what}: {e:.2e} of {tol:.2e}", flush=True)
            assert e <= tol, f"{what}: {name}"
        dY[lo:hi], x[lo:hi] = 0, 0
