"""The order of a row's largest entries where few of its logits are numbers:
numbers first, then the NaNs, each by lowest id."""

import numpy as np
import pytest
import torch

from oracle import logits as L
from tests.gpu_util import device

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def q():
    device()
    import bit_quantized_finetuning_quantize_amd as q
    return q


def _special(V, dtype):
    """Rows of NaN with a few numbers: one, some in a vector, some far apart, some
    beside masked logits, and as many as n_top needs but one."""
    g = torch.Generator(device=device())
    g.manual_seed(V)
    rows = [[900 % V], [900 % V, 901 % V, 903 % V], [0, V - 1], [V - 1], [V // 2, V // 2 + 1, V - 2],
            list(range(5, V, max(1, V // 63)))[:63], list(range(7, V, max(1, V // 63)))[:3]]
    Z = torch.full((len(rows) + 2, V), NAN, device=device())
    for i, ids in enumerate(rows):
        Z[i, ids] = torch.randn(len(ids), generator=g, device=Z.device)
    Z[len(rows)] = -INF             # two numbers, masked logits, then NaNs
    Z[len(rows), V // 4:] = NAN
    Z[len(rows), 3:V // 4] = NAN
    Z[len(rows), 1] = 2.0
    Z[len(rows) + 1, V - 3] = -INF  # one masked logit and NaNs
    return Z.to(dtype)


@pytest.mark.parametrize("n", [1, 4, 20, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [9, 1030])
@pytest.mark.parametrize("V", [300, 1000, 8191, 8192, 9000, 16384, 40000])
def test_nan_last_lowest_id_first(q, V, T, dtype, n):
    print(f"[case] NaN order {T} x {V} {dtype} n={n}", flush=True)
    few = _special(V, dtype)
    Z = torch.zeros(T, V, dtype=dtype, device=few.device)
    Z[:len(few)] = few
    got = q.qlora_logprobs_fwd(Z, n_top=n)[2][:len(few)].cpu().numpy()
    assert np.array_equal(got, L.top(few.double().cpu().numpy(), n))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [1, 5])
def test_nan_last_in_unaligned_rows(q, off, dtype):
    few = _special(24000, dtype)
    wide = torch.zeros(len(few), 24000 + 11, dtype=dtype, device=few.device)
    wide[:, off:off + 24000] = few
    got = q.qlora_logprobs_fwd(wide[:, off:off + 24000], n_top=30)[2].cpu().numpy()
    assert np.array_equal(got, L.top(few.double().cpu().numpy(), 30))
