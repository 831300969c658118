"""One data-parallel training step of a gated block whose activations live in 8 bits.

    python examples/int8_layer_step.py [--tokens T] [--width D] [--hidden F] [--steps S]

The block is y = W2 (silu(G x) * U x) with G and U stacked in W1.  The forward pass
encodes its input once (rowwise_int8) and multiplies from the codes; what it keeps for
the backward pass are those codes, the codes of gate and up, and the codes of the
gated product: 8 bits an element, and no activation in 16.  The backward pass reads
them again.  The two weight gradients are flat fp32 tensors, which the sender half of
the communication codec compresses with error feedback (encode_ef) and the receiver
half decodes; the decoded gradients update fp32 master weights, and the step's loss is
the mean square of y - target.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import embedding_communication_codecs_gb300 as q  # noqa: E402


class GatedBlock:
    def __init__(self, width, hidden, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w1 = torch.randn(2 * hidden, width, generator=gen, device="cuda") / width ** 0.5
        self.w2 = torch.randn(width, hidden, generator=gen, device="cuda") / hidden ** 0.5
        self.err = [torch.zeros_like(self.w1), torch.zeros_like(self.w2)]  # what compression has held back

    def encode_weights(self):
        self.c1, self.s1 = q.rowwise_int8(self.w1)
        self.c2, self.s2 = q.rowwise_int8(self.w2)

    def forward(self, x):
        xc, xs = q.rowwise_int8(x)
        gate_up = q.int8_matmul(xc, xs, self.c1, self.s1)
        hc, hs, saved, saved_scale = q.swiglu_encode(gate_up)
        self.kept = (xc, xs, hc, hs, saved, saved_scale)
        return q.int8_matmul(hc, hs, self.c2, self.s2, dtype=torch.float32)

    def backward(self, dy):
        """(dx, dW1, dW2) from the codes that forward() kept."""
        xc, xs, hc, hs, saved, saved_scale = self.kept
        dw2, _ = q.int8_weight_grad(dy, hc, hs)
        dgate_up = q.swiglu_backward(q.int8_input_grad(dy, self.c2, self.s2), saved, saved_scale)
        dw1, _ = q.int8_weight_grad(dgate_up, xc, xs)
        return q.int8_input_grad(dgate_up, self.c1, self.s1), dw1, dw2

    def update(self, grads, lr, step, bits=8, bucket=2048):
        """Each gradient through the wire: encoded with error feedback, decoded, applied."""
        for w, e, g in zip((self.w1, self.w2), self.err, grads):
            payload = q.encode_ef(g.view(-1), e.view(-1), bits=bits, bucket=bucket, seed=1, step=step)
            w.view(-1).sub_(q.decode_accumulate(*payload, n=w.numel(), bits=bits, bucket=bucket), alpha=lr)


def train(tokens=2048, width=1024, hidden=4096, steps=10, lr=None):
    """The losses of `steps` steps on one fixed batch, whose target another block made."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(torch.bfloat16)
    teacher = GatedBlock(width, hidden, seed=2)
    teacher.encode_weights()
    target = teacher.forward(x)
    block = GatedBlock(width, hidden, seed=1)
    lr = tokens * width / 40.0 if lr is None else lr
    losses = []
    for step in range(steps):
        block.encode_weights()
        d = block.forward(x) - target
        losses.append(d.square().mean())
        dy = (2.0 / d.numel() * d).to(torch.bfloat16)
        _, dw1, dw2 = block.backward(dy)
        block.update((dw1, dw2), lr / tokens, step)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    losses = train(a.tokens, a.width, a.hidden, a.steps)
    for i, v in enumerate(losses):
        print(f"step {i}: loss {v:.5f}")
    if q.qc_take_device_errors():
        raise SystemExit("a pipeline wait timed out")


if __name__ == "__main__":
    main()
