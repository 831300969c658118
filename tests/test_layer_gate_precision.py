"""The fp32 gated activation keeps fp32's precision for gates of any size.

The bounds are in units of U = 2^-24, a rounding of fp32, relative to the exact result's
terms.  The exponential of a negative magnitude is within 2 units in the last place (4 U),
its sum with 1 and the reciprocal and the product that make sigma or 1 - sigma of it add
1 + 2 + 1, the decoded gate is exact here, and so

    dup   = dh * (g * sigma)                           8 U + 2 products             = 10 U
    dgate = (dh * u) * (sigma * (1 + g * (1 - sigma))) 8 + 1 (sum) + 8 + 3 products = 20 U

with dgate's relative to |dh u| sigma (1 + |g| (1 - sigma)), as its two terms cancel near
g = -1.28.  Below 2^-126, at gates under -87.3, sigma itself has an absolute step of 2^-149."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _layer_plain as plain

pytestmark = pytest.mark.gpu


def gates():
    """int8 codes and fp32 scales whose products are exact: every gate from -88 to 88 in steps of 1/1.4."""
    codes = np.tile(np.arange(-127, 128, dtype=np.int8), (4, 1))
    scale = np.array([88 / 128, 0.25, 2.0 ** -6, 2.0 ** -12], dtype=np.float32)
    return codes, scale


@pytest.mark.parametrize("lead", [0, 1])        # rows on vector boundaries, and anywhere
def test_gradients_of_gates_of_any_size(lead):
    import embedding_communication_codecs_gb300 as q
    gc, gs = gates()
    rows, dim = gc.shape[0], 256
    gc = np.concatenate([gc, np.zeros((rows, 1), np.int8)], 1)[:, :dim]
    rng = np.random.default_rng(1)
    uc = rng.integers(-127, 128, (rows, dim)).astype(np.int8)
    us = np.full(rows, 0.125, np.float32)
    dh = rng.standard_normal((rows, dim)).astype(np.float32)
    G, U_ = plain.decoded(gc, gs), plain.decoded(uc, us)
    assert np.array_equal(G, G.astype(np.float32))
    base = torch.zeros(rows * dim + 8, device="cuda")
    t = base[lead:lead + rows * dim].view(rows, dim)
    t.copy_(torch.from_numpy(dh))
    d = q.swiglu_backward(t, torch.from_numpy(np.concatenate([gc, uc], 1)).cuda(),
                          torch.from_numpy(np.stack([gs, us], 1)).cuda()).double().cpu().numpy()
    D = dh.astype(np.float64)
    sig, other = 1 / (1 + np.exp(-G)), 1 / (1 + np.exp(G))      # sigma and 1 - sigma, each to its own precision
    want = D * G * sig
    tol = 10 * plain.U * np.abs(want) + np.abs(D * G) * 2.0 ** -149
    bad = np.abs(d[:, dim:] - want) > tol
    assert not bad.any(), f"dup: {bad.sum()} outside, gates {G[bad][:5]}, worst {np.nanmax(np.abs(d[:, dim:] - want) / (tol + 1e-300)):.3g}"
    want = D * U_ * sig * (1 + G * other)
    size = np.abs(D * U_) * sig * (1 + np.abs(G) * other)
    tol = 20 * plain.U * size + np.abs(D * U_) * (1 + np.abs(G)) * 2.0 ** -149
    bad = np.abs(d[:, :dim] - want) > tol
    assert not bad.any(), f"dgate: {bad.sum()} outside, gates {G[bad][:5]}, worst {np.nanmax(np.abs(d[:, :dim] - want) / (tol + 1e-300)):.3g}"


@pytest.mark.parametrize("dim", [256, 259])
@pytest.mark.parametrize("rows", [5, 2000])
def test_product_of_a_far_gate_and_a_large_up(rows, dim):
    """silu(-87.5 .. -88.5) is below 1e-35 and its product with an up of 1e36 is of ordinary
    size: it is not lost on the way."""
    import embedding_communication_codecs_gb300 as q
    g = torch.linspace(-88.5, -87.5, dim, device="cuda").repeat(rows, 1)
    u = torch.full((rows, dim), 1e36, device="cuda")
    hc, hs, _, _ = q.swiglu_encode(torch.cat([g, u], 1))
    h = g.double() * torch.sigmoid(g.double()) * u.double()
    err = (hc.double() * hs.double()[:, None] - h).abs()
    # sigma is below 2^-126 here: an absolute step of 2^-149, times gate and up
    assert bool((err <= 0.5 * hs.double()[:, None] + h.abs() * 10 * plain.U + g.double().abs() * u.double() * 2.0 ** -149).all())
