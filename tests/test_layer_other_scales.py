"""The gradients from codes under scales that are not powers of two: the decoded operand is an fp32
product rounded to bf16, so each term is off by one bf16 rounding (and the fp32 one before
it), and the sum by its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _layer_plain as plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [(3, 40, 64), (20, 136, 200), (140, 264, 320), (131, 257, 333), (2000, 96, 104)])
def test_gradients(T, N, K):
    import embedding_communication_codecs_gb300 as q
    rng = np.random.default_rng([T, N, K])
    x, w = rng.integers(-128, 128, (T, K)).astype(np.int8), rng.integers(-128, 128, (N, K)).astype(np.int8)
    sx = (np.abs(rng.standard_normal((T, 5))).max(1) / 127).astype(np.float32)       # as max|x| / 127 gives them
    sw = (np.abs(rng.standard_normal((N, 5))).max(1) / 127).astype(np.float32)
    dy = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda().to(torch.bfloat16)
    D = dy.double().cpu().numpy()

    def cu(a):
        return torch.from_numpy(a).cuda()

    def check(got, want, terms, length):
        tol = terms * (plain.U16 * (1 + 2.0 ** -7) + 2 * plain.U) + plain.sum_error(terms, length) * (1 + 2.0 ** -7)
        assert (np.abs(got.double().cpu().numpy() - want) <= tol + plain.rounded(np.abs(want) + tol, False)).all()
    W, X = plain.decoded(w, sw), plain.decoded(x, sx)
    check(q.int8_input_grad(dy, cu(w), cu(sw), dtype=torch.float32), D @ W, np.abs(D) @ np.abs(W), N)
    check(q.int8_weight_grad(dy, cu(x), cu(sx))[0], D.T @ X, np.abs(D).T @ np.abs(X), T)
    # the forward product takes any scale as it is
    y = q.int8_matmul(cu(x), cu(sx), cu(w), cu(sw), dtype=torch.float32).double().cpu().numpy()
    want = X @ W.T
    assert (np.abs(y - want) <= plain.sum_error(np.abs(X) @ np.abs(W).T, K) + 4 * plain.U * np.abs(want)).all()
