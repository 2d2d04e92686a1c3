"""The 8-bit checkpoint MLP example's backward on both bases: dH and the
whole input gradient against float64 products of the decoded operands."""

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


def _f64(t):
    return host_f32(t).astype(np.float64)


def _input_grad(q, lin, dY, base):
    """(dX, bound on the norm of the call's error) of one linear."""
    dy, a, b = _f64(dY), _f64(lin.A), _f64(lin.B)
    if base == "nf4":
        w, d = _f64(q.qlora_nf4_dequantize_bf16(lin.W)).reshape(lin.N, lin.K), dy
    else:
        w = act8.dequantize(lin.W.codes.cpu().numpy(), lin.W.scales.cpu().numpy(), lin.K, 0, 128)
        d = act8.dequantize(*act8.quantize(dy, 0), lin.N, 0)
    low = lin.scale * (dy @ b.T)
    want = d @ w + low @ a.T
    # a rounding to bf16 is 2^-8 / sqrt(3) of a norm at most: the result's, and
    # bf16(s G)'s through A; 1e-4 of the result covers float32 and 8-bit sums
    n = np.linalg.norm
    return want, 2.0 ** -8 / 3 ** 0.5 * (n(want) + n(low) * n(a, 2)) + 1e-4 * n(want)


@pytest.mark.parametrize("base", ["nf4", "fp8"])
def test_input_gradient(ex, base):
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
    want, tol = _input_grad(q, mlp.down, dY, base)
    err = np.linalg.norm(_f64(dH) - want)
    print(f"[parity] dH {base}: {err / tol:.3f} of the bound", flush=True)
    assert err <= tol
    dG, dU = q.qlora_swiglu_act8_bwd(dH, g8, u8)
    wg, tolg = _input_grad(q, mlp.gate, dG, base)
    wu, tolu = _input_grad(q, mlp.up, dU, base)
    dX, _ = mlp.backward(dY, kept)
    tol = tolg + tolu + 2.0 ** -8 / 3 ** 0.5 * np.linalg.norm(wg + wu)  # the sum's own rounding
    err = np.linalg.norm(_f64(dX) - (wg + wu))
    print(f"[parity] dX {base}: {err / tol:.3f} of the bound", flush=True)
    assert err <= tol
    # either path or adapter term left out, or the wrong upstream gradient, is far outside
    n = np.linalg.norm
    for wrong in (wg, wu, _input_grad(q, mlp.gate, dU, base)[0] + wu,
                  wg + wu - mlp.up.scale * _f64(dU) @ _f64(mlp.up.B).T @ _f64(mlp.up.A).T):
        assert n(wrong - (wg + wu)) > 10 * tol
