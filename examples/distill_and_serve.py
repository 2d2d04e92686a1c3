#!/usr/bin/env python3
"""A 4-bit output layer distilled from its 16-bit original, merged, requantized
and served.

The student is the original's NF4 store with a LoRA adapter. Of the teacher
only the largest logits of each token and their log sum exp are kept. A step is
the student's logits, their divergence from the teacher's, the gradient of
the logits (in the logits' place), and the adapter's. The adapter is then merged
into a bf16 weight, which is held in 4 bits with a scale and a zero point to a
group and answers single tokens with their most likely continuations.

    python examples/distill_and_serve.py [--tokens 512] [--width 1024]
        [--vocabulary 8192] [--rank 16] [--top 32] [--steps 30]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_finetuning_quantize_amd as q  # noqa: E402


class Student:
    """The output layer [V x K] in NF4 with a trainable adapter A [K x r], B [r x V]."""

    def __init__(self, W, r, alpha=16, seed=0):
        self.V, self.K = W.shape
        self.r, self.scale = r, alpha / r
        self.W = q.qlora_nf4_quantize(W)
        gen = torch.Generator(device=W.device)
        gen.manual_seed(seed)
        # float32 parameters with a bf16 copy; A random, B zero
        self.params = [torch.randn(self.K, r, generator=gen, device=W.device) / self.K ** 0.5,
                       torch.zeros(r, self.V, device=W.device)]
        self.A, self.B = (p.to(torch.bfloat16) for p in self.params)
        self.state = [q.adamw_state(p.numel(), W.device) for p in self.params]

    def logits(self, X):
        """(bf16 logits [T x V], T = X A)."""
        return q.qlora_linear_fwd(X, self.W, self.A, self.B, self.scale)

    def gradients(self, X, teacher, temperature):
        """(loss of each token, dA, dB) of the mean divergence."""
        ids, values, lse = teacher
        Z, T = self.logits(X)
        loss, stats = q.qlora_distill_fwd(Z, ids, values, lse, temperature)
        g = torch.full_like(loss, temperature ** 2 / loss.numel())
        dZ = q.qlora_distill_bwd(Z, ids, values, stats, g, temperature, dZ=Z)  # in Z's place
        _, dA, dB = q.qlora_linear_bwd(dZ, X, T, self.W, self.A, self.B, self.scale, want_dX=False)
        return loss, dA, dB

    def update(self, grads, lr, step):
        for p, (m, v), g, copy in zip(self.params, self.state, grads, (self.A, self.B)):
            q.qlora_adamw_step(p, m, v, g, lr, step=step, p_bf16=copy)

    def served(self, group=128):
        """The merged weight in groups of 4 bits."""
        return q.qlora_int4_quantize(q.qlora_nf4_merge(self.W, self.A, self.B, self.scale), group)


def teacher_rows(X, W, top, temperature):
    """(ids, logits, log sum exp at the temperature) of the 16-bit layer."""
    Z = (X @ W.t()).float()
    values, ids = torch.topk(Z, top, dim=1)
    return ids, values, torch.logsumexp(Z / temperature, dim=1)


def answer(weight, x, n_top):
    """(ids, log-probabilities) of the likeliest continuations of tokens x [M x K], and
    the entropy of their distributions."""
    Z = q.qlora_int4_linear_fwd(x, weight, torch.float32)
    _, entropy, ids, logp, _ = q.qlora_logprobs_fwd(Z, n_top=n_top, want_stats=False)
    return ids, logp, entropy


def train(tokens=512, width=1024, vocabulary=8192, rank=16, top=32, steps=30, lr=1e-3, temperature=2.0, seed=0,
          report=print):
    """Distils; returns (mean losses, student, the 16-bit weight, the tokens)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    W = (torch.randn(vocabulary, width, generator=gen, device=dev) * (3.0 / width ** 0.5)).to(torch.bfloat16)
    X = torch.randn(tokens, width, generator=gen, device=dev).to(torch.bfloat16)
    student = Student(W, rank, seed=seed)
    teacher = teacher_rows(X, W, top, temperature)
    losses = []
    for step in range(1, steps + 1):
        loss, *grads = student.gradients(X, teacher, temperature)
        student.update(grads, lr, step)
        losses.append(float(loss.mean()))
        if report and (step == 1 or step % 10 == 0):
            report(f"step {step:3d}  divergence {losses[-1]:.6f}")
    return losses, student, W, X


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 1024), ("vocabulary", 8192), ("rank", 16), ("top", 32),
                          ("steps", 30)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    losses, student, W, X = train(a.tokens, a.width, a.vocabulary, a.rank, a.top, a.steps)
    print(f"divergence {losses[0]:.6f} -> {losses[-1]:.6f}")
    weight = student.served()
    print(f"weight: {2 * W.numel() / 1e6:.1f} MB in bf16, {student.W.nbytes() / 1e6:.1f} in NF4, "
          f"{weight.nbytes() / 1e6:.1f} in groups of 4 bits")
    ids, logp, entropy = answer(weight, X[:4], 5)
    for i in range(ids.shape[0]):
        print(f"token {i}: entropy {float(entropy[i]):.3f}, " +
              ", ".join(f"{int(k)} ({float(p):.2f})" for k, p in zip(ids[i], logp[i])))


if __name__ == "__main__":
    main()
