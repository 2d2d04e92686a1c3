"""The 8-bit checkpoint MLP example on both bases: the loss falls, the
gradients are those of the float64 layer at the decoded operands, and the
whole step replays from a HIP graph."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import act8
from tests.gpu_util import device, host_f32

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    device()
    spec = importlib.util.spec_from_file_location(
        "mlp_8bit_checkpoints", os.path.join(ROOT, "examples", "mlp_8bit_checkpoints.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("base", ["nf4", "fp8"])
def test_training_reduces_the_loss(ex, base):
    losses, size = ex.train(base, tokens=200, width=256, hidden=704, rank=8, steps=60, report=None)
    print(f"[case] mlp {base}: loss {losses[0]:.4f} -> {losses[-1]:.4f}, kept {size} bytes", flush=True)
    assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]
    # the 8-bit blocks and T's, against the four bf16 activations
    assert size < 0.6 * 2 * 200 * (256 + 3 * 704)


@pytest.mark.parametrize("base", ["nf4", "fp8"])
def test_gradients_against_float64(ex, base):
    """dA and dB of gate, up and down, and dX, against the chain rule in
    float64 at the kept 8-bit values and the GPU's own dH, dG and dU."""
    dev = device()
    q = ex.q
    mlp = ex.Mlp(192, 320, 8, base, seed=3, device=dev)
    for lin in (mlp.gate, mlp.up, mlp.down):  # an adapter that is not zero
        lin.B.normal_(0, 0.05)
    x = torch.randn(70, 192, device=dev).to(torch.bfloat16)
    dY = (torch.randn(70, 192, device=dev) * 1e-2).to(torch.bfloat16)
    _, kept = mlp.forward(x)
    x8, tg, tu, g8, u8, h8, td = kept
    dH, *_ = mlp.down.backward(dY, h8, td)
    dG, dU = q.qlora_swiglu_act8_bwd(dH, g8, u8)
    dX, grads = mlp.backward(dY, kept)
    f = lambda t: host_f32(t).astype(np.float64)  # noqa: E731
    dec = lambda a: act8.dequantize(a.codes.cpu().numpy(), a.scales.cpu().numpy(), a.shape[1], a.fmt)  # noqa: E731
    want_g, want_u = act8.swiglu_bwd(f(dH), dec(g8), dec(u8))
    for got, want in ((dG, want_g), (dU, want_u)):
        # bf16 rounding: 2^-8 / sqrt(3) of the norm at most
        assert np.linalg.norm(f(got) - want) <= 2.5e-3 * np.linalg.norm(want)
    for lin, inp, T, up, (dA, dB) in ((mlp.gate, x8, tg, dG, grads[0]), (mlp.up, x8, tu, dU, grads[1]),
                                      (mlp.down, h8, td, dY, grads[2])):
        G = f(up) @ f(lin.B).T
        wa, wb = lin.scale * (dec(inp).T @ G), lin.scale * (f(T).T @ f(up))
        # float32 sums of 70 and 320 terms: (70 / 64 + 320 / 64 + 128) 2^-24 of the magnitudes
        tol = 140 * 2.0 ** -24
        assert (np.abs(f(dA) - wa) <= tol * lin.scale * (np.abs(dec(inp)).T @ (np.abs(f(up)) @ np.abs(f(lin.B)).T))).all()
        assert (np.abs(f(dB) - wb) <= tol * lin.scale * (np.abs(f(T)).T @ np.abs(f(up)))).all()
    assert np.isfinite(f(dX)).all()


@pytest.mark.parametrize("base", ["nf4", "fp8"])
def test_step_replays_from_a_graph(ex, base):
    """Forward and backward captured once; every replay, with eager work and
    synchronizations between, gives the eager results bit for bit on new inputs."""
    dev = device()
    mlp = ex.Mlp(256, 704, 8, base, seed=5, device=dev)
    for lin in (mlp.gate, mlp.up, mlp.down):
        lin.B.normal_(0, 0.05)
    x = torch.randn(130, 256, device=dev).to(torch.bfloat16)
    dY = (torch.randn(130, 256, device=dev) * 1e-2).to(torch.bfloat16)

    def run():
        y, kept = mlp.forward(x)
        dX, grads = mlp.backward(dY, kept)
        return [y, dX] + [g for pair in grads for g in pair]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        x.copy_(torch.randn(130, 256, device=dev).to(torch.bfloat16))
        dY.copy_((torch.randn(130, 256, device=dev) * 1e-2).to(torch.bfloat16))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), f"replay {i}, output {k}"
