"""Rows that leave (nearly) no doubt: no log-probability is above 0, no entropy and
no divergence below it, whatever the sums round to. One token far ahead of the
others has p = 1 to float32's last bit."""

import pytest
import torch

from tests.gpu_util import device

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


@pytest.mark.parametrize("t", [1.0, 0.7, 3.3])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", [(3000, 1), (3000, 2), (2000, 100), (1500, 5000), (100, 40000)])
def test_nothing_above_a_probability_of_1(q, T, V, dtype, t):
    print(f"[case] certain {T} x {V} {dtype} t={t}", flush=True)
    g = torch.Generator(device=device())
    g.manual_seed(T + V)
    Z = torch.randn(T, V, generator=g, device=device()) * 3
    y = torch.randint(0, V, (T,), generator=g, device=Z.device)
    # 420 - 20 ahead or more, at t = 3.3 121: the others' share is below 2^-100
    ahead = torch.randn(T, 1, generator=g, device=Z.device).clamp(-4, 4) * 20 + 500
    Z = Z.scatter(1, y[:, None], ahead).to(dtype)
    logp, entropy, ids, top, stats = q.qlora_logprobs_fwd(Z, y, t, n_top=1)
    assert torch.equal(ids[:, 0], y)
    assert (logp <= 0).all() and (top <= 0).all() and (entropy >= 0).all() and (stats[:, 1:] >= 0).all()
    assert (logp >= -2.0 ** -22).all() and (entropy <= 2.0 ** -22).all()
    one = torch.ones(T, device=Z.device)
    assert q.qlora_logprobs_bwd(Z, y, stats, one, one, t).abs().max() <= 2.0 ** -21 / t
    # a teacher as certain, by its list alone and with the rest of its mass
    ids, values = y[:, None].contiguous(), ahead.to(dtype).contiguous()
    for lse in (None, values[:, 0].float() / t):
        loss, stats = q.qlora_distill_fwd(Z, ids, values, lse, t)
        assert (stats[:, 1] >= 0).all()
        if lse is None:
            assert (loss >= 0).all() and (loss <= 2.0 ** -22).all()
