"""The example's training step: every call of the 8-bit layer with the codec around the
weight gradients, against the same step in 64 bits from the same codes."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

from tests import _layer_plain as plain

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_block_against_64_bits():
    import embedding_communication_codecs_gb300 as q
    import int8_layer_step as example
    T, D, F = 96, 64, 160
    block = example.GatedBlock(D, F)
    block.encode_weights()
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, D), generator=gen, device="cuda").to(torch.bfloat16)
    y = block.forward(x)
    dy = (1e-2 * torch.randn((T, D), generator=gen, device="cuda")).to(torch.bfloat16)
    dx, dw1, dw2 = block.backward(dy)

    def value(c, s):
        return plain.decoded(c.cpu().numpy(), s.cpu().numpy())
    xc, xs, hc, hs, saved, saved_scale = block.kept
    X, H, W1, W2 = value(xc, xs), value(hc, hs), value(block.c1, block.s1), value(block.c2, block.s2)
    D_ = dy.double().cpu().numpy()

    def rel(got, want):
        got = got.double().cpu().numpy()
        return np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel(y, H @ W2.T) <= 1e-6                                   # fp32 out, sums below 2^24
    assert rel(dw2, D_.T @ H) <= (T + 1) * 2.0 ** -23
    G, U = value(saved[:, :F].contiguous(), saved_scale[:, 0]), value(saved[:, F:].contiguous(), saved_scale[:, 1])
    dg, du = plain.swiglu_grad(G, U, D_ @ W2)
    dgu = np.concatenate([dg, du], 1)
    # dh and dgate_up are rounded to bf16 on the way: one rounding each, relative to elements
    assert rel(dw1, dgu.T @ X) <= 2 * plain.U16
    assert rel(dx, dgu @ W1) <= 3 * plain.U16
    # what the codes stand for is the activation, to half a step
    assert np.abs(X - x.double().cpu().numpy()).max() <= 0.5 * float(xs.max())
    assert q.qc_take_device_errors() == 0


def test_training_lowers_the_loss():
    import int8_layer_step as example
    losses = example.train(tokens=512, width=256, hidden=1024, steps=8)
    assert all(np.isfinite(losses)) and all(b < a for a, b in zip(losses, losses[1:])), losses
