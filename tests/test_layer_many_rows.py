"""The decoder and the gated activation's backward pass with more rows than the grid covers at
once, where a team goes round several times, on and off vector boundaries."""
from __future__ import annotations

import pytest
import torch

from tests import _layer_plain as plain

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SIZES = [(60000, 64), (70000, 71), (5000, 4096), (5000, 4099), (3000, 8200), (20000, 1001)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_restored_rows(rows, dim, dtype):
    import embedding_communication_codecs_gb300 as q
    gen = torch.Generator(device="cuda").manual_seed(rows)
    codes = torch.randint(-128, 128, (rows, dim), generator=gen, device="cuda", dtype=torch.int8)
    scale = torch.exp2(torch.randint(-100, 100, (rows,), generator=gen, device="cuda").float())
    got = q.rowwise_int8_dequant(codes, scale, dtype=dtype)
    assert torch.equal(got.double(), codes.double() * scale.double()[:, None])       # exact in both types


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_gate_gradients(rows, dim, dtype):
    import embedding_communication_codecs_gb300 as q
    gen = torch.Generator(device="cuda").manual_seed(dim)
    saved = torch.randint(-127, 128, (rows, 2 * dim), generator=gen, device="cuda", dtype=torch.int8)
    scale = torch.exp2(torch.randint(-7, -3, (rows, 2), generator=gen, device="cuda").float())
    dh = torch.randn((rows, dim), generator=gen, device="cuda").to(dtype)
    d = q.swiglu_backward(dh, saved, scale)
    g = saved[:, :dim].double() * scale[:, :1].double()
    u = saved[:, dim:].double() * scale[:, 1:].double()
    sig, x = torch.sigmoid(g), dh.double()
    u16 = 1.01 * plain.U16 if dtype == BF16 else 0.0
    # the terms' sizes times a few fp32 roundings (gates below 16 in magnitude), and the output's own
    for got, want, size in ((d[:, :dim], x * u * sig * (1 + g * (1 - sig)), (x * u).abs() * (1 + g.abs())),
                            (d[:, dim:], x * g * sig, (x * g * sig).abs())):
        assert bool(((got.double() - want).abs() <= u16 * want.abs() + size * 2.0 ** -18 + 1e-40).all())
