"""Gradients added to what is there, by each of the three ways that the kernels write:
TMA additions, element by element, and the join of a cut contraction."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# rows of dw on 16 bytes, off them, cut (whole and odd rows); with more tokens than one range
SIZES = [(130, 200, 264), (130, 200, 263), (4096, 256, 256), (4096, 257, 255), (4096, 1024, 1024), (1001, 776, 1505),
         (64, 24, 40), (1, 5, 7)]


def case(T, N, K):
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)

    def ints(lim, *shape):
        return torch.randint(-lim, lim + 1, shape, generator=gen, device="cuda")
    return ints(2, T, N).to(torch.bfloat16), ints(127, T, K).to(torch.int8), ints


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_integers(T, N, K, bias):
    """Integers whose sums stay below 2^24: one right answer, twice over."""
    import embedding_communication_codecs_gb300 as q
    dy, x, ints = case(T, N, K)
    dw0, db0 = ints(100, N, K).float(), ints(100, N).float()
    dw, db = dw0.clone(), db0.clone()
    one = torch.ones(T, device="cuda")
    want, wb = dy.double().t() @ x.double(), dy.double().sum(0)
    for times in (1, 2):
        got = q.int8_weight_grad(dy, x, one, into=(dw, db if bias else None))
        assert got[0] is dw and got[1] is (db if bias else None)
        assert torch.equal(dw.double(), dw0.double() + times * want)
        assert torch.equal(db.double(), db0.double() + (times * wb if bias else 0))
    assert q.qc_take_device_errors() == 0


@pytest.mark.parametrize("T,N,K", SIZES)
def test_what_is_there_may_be_small(T, N, K):
    """Subnormal and other tiny gradients that a zero is added to are kept, by all three ways."""
    import embedding_communication_codecs_gb300 as q
    rng = np.random.default_rng(T)
    there = rng.integers(0, 1 << 32, N * K, dtype=np.uint64).astype(np.uint32) & 0x807FFFFF       # subnormals of both signs
    dw0 = torch.from_numpy(there.view(np.float32).reshape(N, K).copy()).cuda()
    dw = dw0.clone()
    q.int8_weight_grad(torch.zeros((T, N), dtype=torch.bfloat16, device="cuda"), torch.ones((T, K), dtype=torch.int8, device="cuda"),
                       torch.ones(T, device="cuda"), into=(dw, None))
    assert bool((dw == dw0).all())


@pytest.mark.parametrize("extra", [8, 3])
@pytest.mark.parametrize("T,N,K", [(6, 40, 72), (140, 264, 320), (4096, 256, 256)])
def test_gaps_between_the_rows_of_dy(T, N, K, extra):
    """dy as a slice of a wider tensor, through the calls that take tensors only."""
    import embedding_communication_codecs_gb300 as q
    dense, x, ints = case(T, N, K)
    wide = torch.full((T, N + extra), 1e30, dtype=torch.bfloat16, device="cuda")
    dy = wide[:, :N]
    dy.copy_(dense)
    one, w = torch.ones(T, device="cuda"), ints(31, N, K).to(torch.int8)
    ones = torch.ones(N, device="cuda")
    assert torch.equal(q.int8_input_grad(dy, w, ones, dtype=torch.float32).double(), dense.double() @ w.double())
    dw, db = q.int8_weight_grad(dy, x, one, with_bias=True)
    assert torch.equal(dw.double(), dense.double().t() @ x.double()) and torch.equal(db.double(), dense.double().sum(0))
    dw0, db0 = dw.clone(), db.clone()
    q.int8_weight_grad(dy, x, one, into=(dw, db))
    assert torch.equal(dw, 2 * dw0) and torch.equal(db, 2 * db0)
