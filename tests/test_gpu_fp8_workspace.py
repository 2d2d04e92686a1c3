"""The linear calls on 8-bit inputs in workspaces of exactly their size: the
results of a larger one, and no byte behind it written."""

import pytest
import torch

from tests.gpu_util import device

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _in_place_of(n, call, label):
    """The call's results with a workspace of n bytes, and the bytes behind it."""
    buf = torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device=device())
    out = call(buf[:n])
    assert bool((buf[n:] == 0xA5).all()), f"{label}: written behind the workspace"
    return out


def _same(a, b, label):
    for x, y in zip(a, b):
        assert (x is None) == (y is None) and (x is None or torch.equal(x, y)), label


# few tokens, small tiles, shared ones, column products beside tiles and alone, large tiles
@pytest.mark.parametrize("M,N,K,r", [(1, 64, 64, 1), (1, 512, 4096, 16), (3, 512, 640, 24), (16, 256, 256, 8),
                                     (100, 1280, 6400, 64), (300, 512, 3520, 24), (65, 1344, 128, 200),
                                     (600, 512, 3520, 64), (1100, 256, 4160, 64)])
def test_exact_workspaces(q, M, N, K, r):
    print(f"[case] workspace M={M} N={N} K={K} r={r}", flush=True)
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(M + N + K)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    W, A, B, dY = rnd(N, K), rnd(K, r), rnd(r, N), rnd(M, N)
    x8 = q.qlora_act8_quantize(rnd(M, K))
    w, st = q.qlora_fp8_weight_quantize(W), q.qlora_nf4_quantize(W)
    big = q.act8_workspace(M, N, K, r, dev)
    small, large = (q.qlora_fp8_workspace_bytes(M, N, K, r, b) for b in (False, True))
    ref = q.qlora_fp8_linear_fwd(x8, w, A, B, 0.1, ws=big)
    T = ref[1]
    _same(ref, _in_place_of(small, lambda ws: q.qlora_fp8_linear_fwd(x8, w, A, B, 0.1, ws=ws), "fwd"), "fwd")
    for t in (T, None):
        for want_dX in (True, False):
            kw = dict(want_dX=want_dX)
            ref = q.qlora_fp8_linear_bwd(dY, x8, t, w, A, B, 0.1, ws=big, **kw)
            got = _in_place_of(large if want_dX else small,
                               lambda ws: q.qlora_fp8_linear_bwd(dY, x8, t, w, A, B, 0.1, ws=ws, **kw), "bwd")
            _same(ref, got, f"bwd {want_dX}")
            _same(ref, q.qlora_fp8_linear_bwd(dY, x8, t, w, A, B, 0.1, **kw), "bwd, its own workspace")
            ref = q.qlora_linear_bwd_act8(dY, x8, t, st, A, B, 0.1, ws=big, **kw)
            got = _in_place_of(big.numel() if want_dX else small,
                               lambda ws: q.qlora_linear_bwd_act8(dY, x8, t, st, A, B, 0.1, ws=ws, **kw), "nf4")
            _same(ref, got, f"nf4 {want_dX}")
            _same(ref, q.qlora_linear_bwd_act8(dY, x8, t, st, A, B, 0.1, **kw), "nf4, its own workspace")


@pytest.mark.parametrize("M,N,K", [(1, 100, 129), (333, 1001, 1544), (2040, 2041, 130)])
def test_exact_workspaces_without_adapter(q, M, N, K):
    dev = device()
    w = q.qlora_fp8_weight_quantize(torch.randn(N, K, device=dev).to(torch.bfloat16))
    x8 = q.qlora_act8_quantize(torch.randn(M, K, device=dev).to(torch.bfloat16))
    dY = torch.randn(M, N, device=dev).to(torch.bfloat16)
    small, large = (q.qlora_fp8_workspace_bytes(M, N, K, 0, b) for b in (False, True))
    _same(q.qlora_fp8_linear_fwd(x8, w), _in_place_of(small, lambda ws: q.qlora_fp8_linear_fwd(x8, w, ws=ws), "fwd"), "fwd")
    _same(q.qlora_fp8_linear_bwd(dY, None, None, w),
          _in_place_of(large, lambda ws: q.qlora_fp8_linear_bwd(dY, None, None, w, ws=ws), "bwd"), "bwd")


def test_default_workspace_holds_no_weight(q):
    """One token through a wide 8-bit weight allocates far less than the weight's own bytes."""
    M, N, K, r = 1, 8192, 4096, 16
    dev = device()
    w = q.qlora_fp8_weight_quantize(torch.randn(N, K, device=dev).to(torch.bfloat16))
    x8 = q.qlora_act8_quantize(torch.randn(M, K, device=dev).to(torch.bfloat16))
    A = torch.randn(K, r, device=dev).to(torch.bfloat16)
    B = torch.randn(r, N, device=dev).to(torch.bfloat16)
    dY = torch.randn(M, N, device=dev).to(torch.bfloat16)
    for call in (lambda: q.qlora_fp8_linear_fwd(x8, w, A, B, 0.1),
                 lambda: q.qlora_fp8_linear_bwd(dY, x8, None, w, A, B, 0.1)):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call()
        took = torch.cuda.max_memory_allocated() - before
        print(f"[case] {took} bytes beside a weight of {N * K}", flush=True)
        assert took < N * K // 4
