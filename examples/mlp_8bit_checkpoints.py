#!/usr/bin/env python3
"""A gated MLP (gate, up, down) finetuned with LoRA on a frozen base, its
activation checkpoints in 8 bits.

The base is held in NF4 or in 8-bit blocks. A step keeps, for the backward
pass, the 8-bit blocks of the MLP's input, of gate's and up's outputs and of
down's input, half the bytes of the bf16 tensors they stand for. With the
8-bit base the kept blocks are the forward products'
operands too.

    python examples/mlp_8bit_checkpoints.py [--base nf4|fp8] [--tokens 512]
        [--width 1024] [--hidden 2816] [--rank 16] [--steps 40]

prints the loss every few steps and the bytes kept per step.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_finetuning_quantize_amd as q  # noqa: E402


class Linear:
    """A frozen weight [N x K] with a trainable adapter A [K x r], B [r x N]."""

    def __init__(self, W, r, alpha, base, gen):
        self.N, self.K = W.shape
        self.r, self.scale, self.base = r, alpha / r, base
        self.W = q.qlora_nf4_quantize(W) if base == "nf4" else q.qlora_fp8_weight_quantize(W)
        dev = W.device
        # the usual start: A random, B zero; float32 parameters with a bf16 copy
        a = torch.randn(self.K, r, generator=gen, device=dev) / self.K ** 0.5
        self.params = [a, torch.zeros(r, self.N, device=dev)]
        self.A, self.B = (p.to(torch.bfloat16) for p in self.params)
        self.state = [q.adamw_state(p.numel(), dev) for p in self.params]

    def forward(self, x, x8):
        """(Y, T) from the bf16 input (NF4 base) or its 8-bit blocks."""
        if self.base == "nf4":
            return q.qlora_linear_fwd(x, self.W, self.A, self.B, self.scale)
        return q.qlora_fp8_linear_fwd(x8, self.W, self.A, self.B, self.scale)

    def backward(self, dY, x8, T):
        """(dX, dA, dB) from the 8-bit input."""
        if self.base == "nf4":
            return q.qlora_linear_bwd_act8(dY, x8, T, self.W, self.A, self.B, self.scale)
        return q.qlora_fp8_linear_bwd(dY, x8, T, self.W, self.A, self.B, self.scale)

    def update(self, grads, lr, step):
        for p, (m, v), g, copy in zip(self.params, self.state, grads, (self.A, self.B)):
            q.qlora_adamw_step(p, m, v, g, lr, step=step, p_bf16=copy)


class Mlp:
    def __init__(self, width, hidden, r, base, seed=0, alpha=16, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=gen, device=device) / k ** 0.5).to(torch.bfloat16)

        self.gate = Linear(weight(hidden, width), r, alpha, base, gen)
        self.up = Linear(weight(hidden, width), r, alpha, base, gen)
        self.down = Linear(weight(width, hidden), r, alpha, base, gen)
        self.base = base

    def forward(self, x):
        """(Y, what the backward needs)."""
        x8 = q.qlora_act8_quantize(x)
        g, tg = self.gate.forward(x, x8)
        u, tu = self.up.forward(x, x8)
        # the bf16 h feeds the NF4 product; the 8-bit product takes h8 itself
        h, h8, g8, u8 = q.qlora_swiglu_act8_fwd(g, u, want_h=self.base == "nf4")
        y, td = self.down.forward(h, h8)
        return y, (x8, tg, tu, g8, u8, h8, td)

    def backward(self, dY, kept):
        """Gradient of the input, and [(dA, dB)] of gate, up and down."""
        x8, tg, tu, g8, u8, h8, td = kept
        dH, *down = self.down.backward(dY, h8, td)
        dG, dU = q.qlora_swiglu_act8_bwd(dH, g8, u8, dG=dH)  # dG takes dH's place
        dXg, *gate = self.gate.backward(dG, x8, tg)
        dXu, *up = self.up.backward(dU, x8, tu)
        return dXg + dXu, [gate, up, down]

    def update(self, grads, lr, step):
        for lin, g in zip((self.gate, self.up, self.down), grads):
            lin.update(g, lr, step)


def kept_bytes(kept):
    return sum(k.nbytes() if isinstance(k, q.Act8) else k.numel() * k.element_size() for k in kept)


def train(base="nf4", tokens=512, width=1024, hidden=2816, rank=16, steps=40, lr=2e-3, seed=0,
          report=print):
    """Fits the adapters to a target that differs from the base's output;
    returns the losses and the bytes kept in a step."""
    dev = torch.device("cuda", torch.cuda.current_device())
    mlp = Mlp(width, hidden, rank, base, seed, device=dev)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed + 1)
    x = torch.randn(tokens, width, generator=gen, device=dev).to(torch.bfloat16)
    y0, kept = mlp.forward(x)
    shift = torch.randn(width, 4, generator=gen, device=dev) @ torch.randn(4, width, generator=gen, device=dev)
    target = y0.float() + 0.3 * (x.float() @ shift) / (2 * width ** 0.5)
    losses, size = [], kept_bytes(kept)
    for step in range(1, steps + 1):
        y, kept = mlp.forward(x)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        dY = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        _, grads = mlp.backward(dY, kept)
        mlp.update(grads, lr, step)
        if report and (step == 1 or step % 10 == 0):
            report(f"step {step:3d}  loss {losses[-1]:.5f}")
    return losses, size


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--base", choices=("nf4", "fp8"), default="nf4")
    for name, default in (("tokens", 512), ("width", 1024), ("hidden", 2816), ("rank", 16), ("steps", 40)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    losses, size = train(a.base, a.tokens, a.width, a.hidden, a.rank, a.steps)
    plain = 2 * a.tokens * (a.width + 3 * a.hidden)
    print(f"kept for the backward pass: {size / 1e6:.2f} MB (the activations alone in bf16: {plain / 1e6:.2f} MB)")
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
