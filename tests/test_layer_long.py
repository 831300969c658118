"""Matrices of more than 2^32 elements: every call's last rows, which lie beyond what 32 bits
count, against the same call on those rows by themselves.  Integers, so one right answer."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

TAIL = 300


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.get_device_properties(0).total_memory < 150 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def ints(shape, lim, seed, dtype=torch.int8):
    """Filled a slice at a time."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.split(1 << 16):
        part.copy_(torch.randint(-lim, lim + 1, part.shape, generator=gen, device="cuda", dtype=torch.int8))
    return out


@pytest.mark.parametrize("rows,dim", [((1 << 20) + 5000, 4096), ((1 << 19) + 5000, 8195)])
def test_rows_and_gates(rows, dim):
    import embedding_communication_codecs_gb300 as q
    assert rows * dim > 1 << 32
    x = ints((rows, dim), 100, 1, torch.bfloat16)
    tail = slice(rows - TAIL, rows)
    codes, scale = q.rowwise_int8(x)
    want, ws = q.rowwise_int8(x[tail].contiguous())
    assert torch.equal(codes[tail], want) and torch.equal(scale[tail], ws)
    back = q.rowwise_int8_dequant(codes, scale)
    del codes
    assert torch.equal(back[tail], q.rowwise_int8_dequant(want, ws)) and torch.equal(back[:TAIL], x[:TAIL])
    del back
    if dim % 2:
        gate_up = x[:, :dim - 1]        # an even number of strided elements
    else:
        gate_up = x
    got = q.swiglu_encode(gate_up)
    ref = q.swiglu_encode(gate_up[tail].contiguous())
    for a, b in zip(got, ref):
        assert torch.equal(a[tail], b)
    dh = x[:, :gate_up.shape[1] // 2]
    d = q.swiglu_backward(dh, got[2], got[3])
    assert torch.equal(d[tail], q.swiglu_backward(dh[tail].contiguous(), ref[2], ref[3]))


@pytest.mark.parametrize("K", [4096, 4099])
def test_products(K):
    import embedding_communication_codecs_gb300 as q
    T, N = (1 << 20) + 5000, 48
    x, w = ints((T, K), 3, 2), ints((N, K), 3, 3)
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    tail = slice(T - TAIL, T)
    y = q.int8_matmul(x, one_t, w, one_n, dtype=torch.float32)
    assert torch.equal(y[tail].double(), x[tail].double() @ w.double().t())
    assert torch.equal(y[:TAIL].double(), x[:TAIL].double() @ w.double().t())
    # as the gradient's long sums: dy of one live row at either end
    dy = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    dy[0, 1], dy[T - 1, 2], dy[T - 7, 2] = 1, 2, -1
    dw, db = q.int8_weight_grad(dy, x, one_t, with_bias=True)
    want = torch.zeros((N, K), device="cuda")
    want[1], want[2] = x[0].float(), 2 * x[T - 1].float() - x[T - 7].float()
    assert torch.equal(dw, want) and db[1] == 1 and db[2] == 1 and db.abs().sum() == 2
    del dw, want
    dy.copy_(ints((T, N), 2, 4))
    dx = q.int8_input_grad(dy, w, one_n, dtype=torch.float32)      # more than 2^32 results
    assert torch.equal(dx[tail].double(), dy[tail].double() @ w.double())
    assert torch.equal(dx[:TAIL].double(), dy[:TAIL].double() @ w.double())
    assert q.qc_take_device_errors() == 0


def test_products_of_many_outputs():
    """More than 2^32 weights and results."""
    import embedding_communication_codecs_gb300 as q
    N, K = (1 << 20) - 7, 4112
    w = ints((N, K), 3, 5)
    one_n = torch.ones(N, device="cuda")
    tail = slice(N - TAIL, N)
    for T in (2, 40, 4200):
        x = ints((T, K), 3, 6)
        y = q.int8_matmul(x, torch.ones(T, device="cuda"), w, one_n, dtype=torch.bfloat16)
        assert torch.equal(y[:, tail].double(), (x.double() @ w[tail].double().t()).to(torch.bfloat16).double())
        del y
    assert q.qc_take_device_errors() == 0
