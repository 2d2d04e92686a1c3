"""Groups of 4-bit codes on the GPU: codes, scales, zero points and decoded values
against the oracle bit for bit, products against float64.

Products: with whole numbers for tokens and powers of two for scales every
product and sum is exact in float32 (below 2^24 of the smallest unit), so the
outputs are the exact sums, rounded once to bf16. With other values, the 2 G
products x (16 + q) and -x (16 + z) of a group are exact and their sum has at
most 2 G roundings of at most 2^-23 of its running magnitude, below 62 sum|x|;
scaling and adding K / G groups and eight waves round 2^-24 each of a sum below
15 sum s|x|.
"""

import numpy as np
import pytest
import torch

from oracle import int4
from oracle.bf16 import bf16_round
from tests.gpu_util import device, host_f32

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _gen(*seed):
    g = torch.Generator(device=device())
    g.manual_seed(sum(s * 7919 ** i for i, s in enumerate(seed)) % (1 << 31))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=device())


QUANT = [(1, 32), (3, 64), (5, 96), (7, 160), (17, 1504), (64, 4096), (200, 11008)]


@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,K", QUANT)
def test_quantize(q, N, K, G, sym):
    print(f"[case] quantize {N} x {K} G={G} sym={sym}", flush=True)
    g = _gen(N, K, G)
    w = _randn(g, N, K) * 0.02
    if N > 6:
        w[1] = 0
        w[2] = w[2].abs()
        w[3] = -w[3].abs()
        w[4] = torch.round(w[4] * 128) / 128  # ties
        w[5] = w[5] * 2.0 ** -120             # scales without full precision
        w[6] = w[6] * 2.0 ** 125            # (2^130 is no float32: it made infinities, which are unsupported)
        w[1, 5] = 1e-39                       # a scale that rounds to little or nothing
    w = w.to(BF)
    st = q.qlora_int4_quantize(w, G, sym)
    codes, s, z = int4.quantize(host_f32(w), G, sym)
    assert np.array_equal(host_f32(st.scales), s)
    if sym:
        assert st.zeros is None
    else:
        assert np.array_equal(st.zeros.cpu().numpy(), z)
    assert np.array_equal(st.codes.cpu().numpy(), codes)
    d = q.qlora_int4_dequantize(st)
    want = int4.dequantize(codes, s, None if sym else z, G)
    assert np.array_equal(host_f32(d), bf16_round(want.astype(np.float32)))
    # strided, unaligned rows; nothing beside them written
    wide = torch.full((N, K + 21), 9.0, dtype=BF, device=w.device)
    wide[:, 3:3 + K] = w
    again = q.qlora_int4_quantize(wide[:, 3:3 + K], G, sym)
    assert torch.equal(again.codes, st.codes) and torch.equal(again.scales, st.scales)
    out = torch.full((N, K + 21), 9.0, dtype=BF, device=w.device)
    q.qlora_int4_dequantize(st, out=out[:, 3:3 + K])
    assert torch.equal(out[:, 3:3 + K], d) and (out[:, :3] == 9.0).all() and (out[:, 3 + K:] == 9.0).all()


def _weight(q, g, N, K, G, sym, exact):
    ng = -(-K // G)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=device(), dtype=torch.uint8)
    if exact:
        scales = torch.exp2(torch.randint(-1, 2, (N, ng), generator=g, device=device()).float())
    else:
        scales = (0.5 + torch.rand(N, ng, generator=g, device=device())) * 0.005
    zeros = None if sym else torch.randint(0, 16, (N, ng), generator=g, device=device(), dtype=torch.uint8)
    return q.Int4Weight(codes, scales.to(BF), zeros, (N, K), G)


def _dense(w):
    return int4.dequantize(w.codes.cpu().numpy(), host_f32(w.scales), None if w.zeros is None else w.zeros.cpu().numpy(),
                           w.group)


LINEAR = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 100, 128), (5, 1001, 1504), (16, 33, 160), (17, 64, 4096),
          (1, 4096, 4096), (33, 130, 1056), (48, 300, 2048), (64, 65, 8224), (65, 40, 256), (130, 70, 416),
          (1, 24, 11008), (300, 17, 64),
          # 32 and 48 rows to a workgroup
          (9, 4100, 96), (20, 8191, 160), (33, 8300, 128), (50, 8200, 96), (70, 5000, 64), (4, 9000, 224),
          # two runs to a step, the rows' end in the first or the second
          (5, 40, 4096), (8, 100, 4320), (9, 30, 4224), (16, 70, 8352),
          # 64 tokens and 32 rows
          (49, 8000, 96), (130, 4100, 160)]


@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_exact(q, M, N, K, G, sym):
    print(f"[case] linear {M} x {N} x {K} G={G} sym={sym}", flush=True)
    g = _gen(M, N, K, G)
    w = _weight(q, g, N, K, G, sym, True)
    x = torch.randint(-8, 9, (M, K), generator=g, device=device()).to(BF)
    want = host_f32(x).astype(np.float64) @ _dense(w).T
    assert np.abs(want).max() < 2 ** 22
    y = q.qlora_int4_linear_fwd(x, w, F32)
    assert np.array_equal(host_f32(y), want)
    assert torch.equal(q.qlora_int4_linear_fwd(x, w), y.to(BF))
    # strided rows in and out; nothing beside them written
    xs = torch.full((M, K + 24), 3.0, dtype=BF, device=x.device)
    xs[:, 8:8 + K] = x
    for dt in (BF, F32):
        ys = torch.full((M, N + 5), 9.0, dtype=dt, device=x.device)
        q.qlora_int4_linear_fwd(xs[:, 8:8 + K], w, Y=ys[:, 2:2 + N])
        assert torch.equal(ys[:, 2:2 + N], y.to(dt)) and (ys[:, :2] == 9.0).all() and (ys[:, 2 + N:] == 9.0).all()


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (5, 1001, 1504), (48, 320, 4096), (64, 100, 11008)])
def test_linear(q, M, N, K, G):
    print(f"[case] linear, real values {M} x {N} x {K} G={G}", flush=True)
    g = _gen(M, N, K, G, 1)
    w = _weight(q, g, N, K, G, False, False)
    x = _randn(g, M, K).to(BF)
    xd, wd = host_f32(x).astype(np.float64), _dense(w)
    want = xd @ wd.T
    scale = np.repeat(host_f32(w.scales).astype(np.float64), G, axis=1)[:, :K]
    size = np.abs(xd) @ scale.T
    tol = size * (2 * G * 2.0 ** -23 * 62 + (K / G + 10) * 2.0 ** -24 * 15)
    y = host_f32(q.qlora_int4_linear_fwd(x, w, F32)).astype(np.float64)
    far = (np.abs(y - want) / tol).max()
    print(f"[parity] error / tolerance {far:.4f}, of the largest output {np.abs(y - want).max() / np.abs(want).max():.2e}",
          flush=True)
    assert far <= 1.0
    yb = host_f32(q.qlora_int4_linear_fwd(x, w)).astype(np.float64)
    assert (np.abs(yb - want) <= tol + 2.0 ** -8 * np.abs(want)).all()


def test_quantized_product_is_the_dequantized_ones(q):
    """The product of a quantized weight against that of its decoded values, which
    bf16 rounds by 2^-9 of a value at most."""
    g = _gen(3)
    w = (_randn(g, 256, 512) * 0.02).to(BF)
    st = q.qlora_int4_quantize(w)
    x = _randn(g, 4, 512).to(BF)
    y = q.qlora_int4_linear_fwd(x, st, F32)
    d = q.qlora_int4_dequantize(st).double()
    bound = (x.double().abs() @ d.abs().T.contiguous()) * 2.0 ** -8 + 1e-6
    assert ((y.double() - x.double() @ d.T.contiguous()).abs() <= bound).all()


@pytest.mark.parametrize("G", [32, 64, 128])
def test_upper_bits_of_zero_points_are_not_read(q, G):
    g = _gen(7, G)
    w = _weight(q, g, 70, 416, G, False, True)
    x = torch.randint(-8, 9, (5, 416), generator=g, device=device()).to(BF)
    y, d = q.qlora_int4_linear_fwd(x, w, F32), q.qlora_int4_dequantize(w)
    w.zeros |= torch.randint(0, 16, w.zeros.shape, generator=g, device=device(), dtype=torch.uint8) << 4
    assert (w.zeros > 15).any()
    assert torch.equal(q.qlora_int4_linear_fwd(x, w, F32), y) and torch.equal(q.qlora_int4_dequantize(w), d)


def test_not_finite_tokens_stay_in_their_rows(q):
    g = _gen(4)
    w = _weight(q, g, 100, 256, 64, False, True)
    x = torch.randint(-8, 9, (20, 256), generator=g, device=device()).to(BF)
    clean = q.qlora_int4_linear_fwd(x, w, F32)
    bad = x.clone()
    bad[3, 7], bad[17, 200] = float("nan"), float("inf")
    y = q.qlora_int4_linear_fwd(bad, w, F32)
    keep = [i for i in range(20) if i not in (3, 17)]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[[3, 17]]).all()


def test_graph_and_streams(q):
    g = _gen(5)
    w = _weight(q, g, 1000, 2048, 128, False, True)
    x = torch.randint(-8, 9, (3, 2048), generator=g, device=device()).to(BF)
    q.qlora_int4_linear_fwd(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.qlora_int4_linear_fwd(x, w)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = q.qlora_int4_linear_fwd(x, w, F32)
    for _ in range(4):
        x.copy_(torch.randint(-8, 9, (3, 2048), generator=g, device=device()))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, q.qlora_int4_linear_fwd(x, w, F32))


def test_largest_weight(q):
    """Codes up to the last byte below 2^31: rows at both ends of it."""
    K = 16384
    N = (1 << 32) // K - 1
    g = _gen(6)
    w = _weight(q, g, N, K, 128, False, True)
    x = torch.randint(-8, 9, (2, K), generator=g, device=device()).to(BF)
    y = q.qlora_int4_linear_fwd(x, w, F32)
    rows = [0, 1, N // 2, N - 2, N - 1]
    part = q.Int4Weight(w.codes[rows], w.scales[rows], w.zeros[rows], (len(rows), K), 128)
    want = host_f32(x).astype(np.float64) @ _dense(part).T
    assert np.array_equal(host_f32(y[:, rows]), want)


def test_largest_quantization(q):
    """Nearly 2^32 values: groups at both ends as they come by themselves."""
    K = 16384
    N = (1 << 32) // K - 1
    w = torch.empty(N, K, dtype=BF, device=device())
    w.normal_(0, 0.02)
    st = q.qlora_int4_quantize(w, 32)
    d = q.qlora_int4_dequantize(st)
    for rows in (slice(0, 2), slice(N // 2, N // 2 + 2), slice(N - 2, N)):
        few = q.qlora_int4_quantize(w[rows], 32)
        assert torch.equal(few.codes, st.codes[rows]) and torch.equal(few.scales, st.scales[rows])
        assert torch.equal(few.zeros, st.zeros[rows]) and torch.equal(q.qlora_int4_dequantize(few), d[rows])
