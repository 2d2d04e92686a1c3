"""A forward pass over split rows leaves none of its flags set: a full set left in a
kept workspace would join a row early in a later call that had the same tag.
The flags are the workspace's first words, one to a row and part."""

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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,parts", [(1, 131072, 16), (3, 120000, 15), (5, 16384, 2), (600, 24576, 2), (1024, 131080, 2)])
def test_flags_are_0_after_a_call(q, T, V, parts, dtype):
    print(f"[case] flags {T} x {V} {dtype}", flush=True)
    g = torch.Generator(device=device())
    g.manual_seed(V + T)
    Z = torch.randn(T, V, generator=g, device=device()).to(dtype)
    ids = torch.randint(0, V, (T, 16), generator=g, device=Z.device)
    values = torch.randn(T, 16, generator=g, device=Z.device)
    lse = torch.full((T,), 12.0, device=Z.device)
    ws = q.logits_workspace(T, V, 20, Z.device)
    calls = [lambda: q.qlora_logprobs_fwd(Z, ws=ws), lambda: q.qlora_logprobs_fwd(Z, n_top=20, ws=ws),
             lambda: q.qlora_distill_fwd(Z, ids, values, ws=ws), lambda: q.qlora_distill_fwd(Z, ids, values, lse, ws=ws)]
    for f in calls:
        outputs = []
        for before in (0, 255):
            ws.fill_(before)
            outputs.append(f())
            assert (ws[:T * parts * 8].view(torch.int64) == 0).all()
        for a, b in zip(*outputs):
            assert a is None and b is None or torch.equal(a, b)
