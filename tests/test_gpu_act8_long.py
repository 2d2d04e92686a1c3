"""Products along contractions of several hundred thousand elements, in each
tile. The operands are integers up to 8, which the codes hold exactly, and
every partial sum stays below 2^24: the float32 result is the exact one."""

import pytest
import torch

from tests.gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _ints(g, *shape):
    return torch.randint(-8, 9, shape, generator=g, device=g.device, dtype=torch.int8).to(torch.bfloat16)


def _exact(a, b):
    """a [M x K] b [N x K]^T: integer sums below 2^24, in any order."""
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for k in range(0, a.shape[1], 65536):
        out += (a[:, k:k + 65536].float() @ b[:, k:k + 65536].float().t()).double()
    return out


# one token and a few, 64 x 64, 128 x 64, and 256 x 256 tiles with parts of the
# last round; K near the longest row too
@pytest.mark.parametrize("M,N,K", [(1, 100, 2_097_152), (40, 96, 2_097_000), (300, 500, 700_001),
                                   (300, 3600, 1_100_000), (2560, 1664, 400_000)])
def test_long_product(q, M, N, K):
    print(f"[case] long product M={M} N={N} K={K}", flush=True)
    g = torch.Generator(device=device())
    g.manual_seed(K)
    x, w = _ints(g, M, K), _ints(g, N, K)
    W = q.qlora_fp8_weight_quantize(w, transposed=False)
    Y, _ = q.qlora_fp8_linear_fwd(q.qlora_act8_quantize(x), W)
    assert torch.equal(Y, _exact(x, w).to(torch.bfloat16))


def test_long_product_with_adapter(q):
    M, N, K, r = 2560, 1664, 400_000, 24
    print(f"[case] long product M={M} N={N} K={K} r={r}", flush=True)
    g = torch.Generator(device=device())
    g.manual_seed(5)
    x, w = _ints(g, M, K), _ints(g, N, K)
    A, B = _ints(g, K, r), torch.zeros(r, N, dtype=torch.bfloat16, device=x.device)
    B[0, :] = 1.0
    A[:, 0] = 0
    A[:64, 0] = 1.0  # T[:, 0] a sum of 64 integers, whose bf16 rounding is exact below 2^8
    x[:, 32:64] = -x[:, :32]  # and here 0 but for the first column
    x[:, 0] += 1
    W = q.qlora_fp8_weight_quantize(w, transposed=False)
    Y, T = q.qlora_fp8_linear_fwd(q.qlora_act8_quantize(x), W, A, B, 1.0)
    want = _exact(x, A.t().contiguous())
    assert torch.equal(T.double(), want) and bool((want[:, 0] == 1).all())
    assert torch.equal(Y, (_exact(x, w) + want[:, :1]).to(torch.bfloat16))


def test_long_backward(q):
    """The bf16 product of the NF4 base and the row products, along N."""
    M, N, K, r = 2560, 200_000, 1664, 24
    print(f"[case] long backward M={M} N={N} K={K} r={r}", flush=True)
    g = torch.Generator(device=device())
    g.manual_seed(6)
    dY = _ints(g, M, N)
    w = _ints(g, N, K) / 64
    st = q.qlora_nf4_quantize(w)
    x = _ints(g, M, K)
    A, B = torch.zeros(K, r, dtype=torch.bfloat16, device=x.device), _ints(g, r, N)
    dX, dA, _ = q.qlora_linear_bwd_act8(dY, q.qlora_act8_quantize(x), None, st, A, B, 1.0)
    G = _exact(dY, B)
    want = x.double().t() @ G
    # 2560 terms of 24 bits: float32 sums over waves, blocks and three terms each
    tol = (M / 64 + 64) * 2.0 ** -24 * (x.double().abs().t() @ G.abs())
    assert bool(((dA.double() - want).abs() <= tol).all())
    v = q.qlora_nf4_dequantize_bf16(st).view(N, K)
    want = torch.zeros(M, K, dtype=torch.float64, device=x.device)
    mags = torch.zeros_like(want)
    for n in range(0, N, 25_000):
        d, b = dY[:, n:n + 25_000].double(), v[n:n + 25_000].double()
        want += d @ b
        mags += d.abs() @ b.abs()
    tol = (N / 64 + 64) * 2.0 ** -24 * mags + 2.0 ** -8 * 1.01 * want.abs()
    assert bool(((dX.double() - want).abs() <= tol).all())
    # the same contraction on the 8-bit base, where W and dY are exact
    W = q.qlora_fp8_weight_quantize(w)
    dX = q.qlora_fp8_linear_bwd(dY, None, None, W)[0]
    assert torch.equal(dX, (_exact(dY, (w * 64).t().contiguous()) / 64).to(torch.bfloat16))
