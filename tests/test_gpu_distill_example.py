"""The distillation example: its gradients against float64, its captured step, the
chain from the merged weight to the served log-probabilities, and that it runs."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import int4
from oracle import logits as L
from tests.gpu_util import TOL, assert_close, device, host_f32

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    device()
    spec = importlib.util.spec_from_file_location("distill_and_serve", os.path.join(ROOT, "examples", "distill_and_serve.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _setup(ex, T, K, V, r, top, temperature):
    gen = torch.Generator(device=device())
    gen.manual_seed(T + K + V)
    rnd = lambda *s: torch.randn(s, generator=gen, device=device())  # noqa: E731
    W = (rnd(V, K) * (3.0 / K ** 0.5)).to(torch.bfloat16)
    X = rnd(T, K).to(torch.bfloat16)
    s = ex.Student(W, r)
    s.B.copy_(rnd(r, V) * 0.05)  # so that dA is not 0
    return s, W, X, ex.teacher_rows(X, W, top, temperature)


def _f64(t):
    return host_f32(t).astype(np.float64)


@pytest.mark.parametrize("T,K,V,r,top", [(7, 128, 192, 8, 5), (40, 256, 1024, 16, 32), (300, 192, 8256, 8, 64)])
def test_gradients(ex, T, K, V, r, top):
    """Each step in float64 from the one before: the logits from the stored weight's
    values, then loss, dA and dB by the chain rule from the bf16 logits. (From
    exact logits there is no useful bound: a rounding of 2^-9 of a logit of 16
    changes p by 3 % of itself, and p - q is a small part of p.)"""
    t = 2.0
    s, W, X, teacher = _setup(ex, T, K, V, r, top, t)
    loss, dA, dB = s.gradients(X, teacher, t)
    x, a, b = _f64(X), _f64(s.A), _f64(s.B)
    wp = oracle.bf16_round(_f64(ex.q.qlora_nf4_dequantize(s.W)).astype(np.float32)).astype(np.float64).reshape(V, K)
    Z = s.logits(X)[0]
    assert_close(host_f32(Z), x @ wp.T + s.scale * (x @ a) @ b, "Z")
    ids, values, lse = (v.cpu().numpy() for v in teacher)
    values, lse = values.astype(np.float64), lse.astype(np.float64)
    want, st = L.distill(_f64(Z), t, ids, values, lse)
    assert (np.abs(_f64(loss) - want) <= 2.0 ** -24 * (600 + 6 * top) * np.maximum(1, st[:, 2])).all()
    dz = L.distill_grad(_f64(Z), t, ids, values, lse, np.full(T, t * t / T))
    # the products take dz in bf16: 2^-9 of each, well inside the products' own bound
    assert_close(host_f32(dA), s.scale * x.T @ (dz @ b.T), "dA", TOL)
    assert_close(host_f32(dB), s.scale * (x @ a).T @ dz, "dB", TOL)


def test_captured_step(ex):
    t = 1.5
    s, W, X, teacher = _setup(ex, 64, 256, 2048, 8, 16, t)
    s.gradients(X, teacher, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.gradients(X, teacher, t)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = s.gradients(X, teacher, t)
    for i in range(4):
        X.copy_(torch.randn_like(X, dtype=torch.float32) * (1 + i))
        gr.replay()
        torch.cuda.synchronize()
        want = s.gradients(X, teacher, t)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("M", [1, 5, 40])
def test_served(ex, M):
    """Merged weight, its codes, the products and the log-probabilities, each step
    against float64 from the one before."""
    s, W, X, _ = _setup(ex, 64, 256, 2048, 8, 16, 1.0)
    merged = ex.q.qlora_nf4_merge(s.W, s.A, s.B, s.scale)
    w = s.served(64)
    codes, scales, zeros = int4.quantize(host_f32(merged), 64, False)
    assert np.array_equal(w.codes.cpu().numpy(), codes) and np.array_equal(w.zeros.cpu().numpy(), zeros)
    dense = int4.dequantize(codes, scales, zeros, 64)
    x = _f64(X[:M])
    z = x @ dense.T
    Z = ex.q.qlora_int4_linear_fwd(X[:M], w, torch.float32)
    # per group of 64: 128 roundings of 2^-23 of sums below 62 s |x|; then 4 groups
    size = np.abs(x) @ np.repeat(scales.astype(np.float64), 64, axis=1).T
    tol = size * (2 * 64 * 62 * 2.0 ** -23 + 14 * 15 * 2.0 ** -24)
    assert (np.abs(_f64(Z) - z) <= tol).all()
    ids, logp, entropy = ex.answer(w, X[:M], 7)
    assert np.array_equal(ids.cpu().numpy(), L.top(_f64(Z), 7))
    ref, _, l = L.log_softmax(_f64(Z), 1.0)
    want = np.take_along_axis(ref, ids.cpu().numpy(), 1)
    assert (np.abs(_f64(logp) - want) <= 2.0 ** -24 * (200 + 4 * l[:, None] + 4 * np.abs(want))).all()
    H = L.entropy(ref)
    assert (np.abs(_f64(entropy) - H) <= 2.0 ** -24 * (200 + 4 * l + 250 * np.abs(H - l))).all()


def test_runs(ex):
    losses, student, W, X = ex.train(tokens=64, width=128, vocabulary=640, rank=8, top=16, steps=3, report=None)
    assert len(losses) == 3 and np.isfinite(losses).all()
    ids, logp, entropy = ex.answer(student.served(32), X[:2], 3)
    assert ids.shape == (2, 3) and bool((logp <= 0).all()) and bool((entropy >= 0).all())
