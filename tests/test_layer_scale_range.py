"""int8_matmul's two scales where their product leaves fp32's range: the result is that of
the formula wherever it is in range.

One unit is U = 2^-24: an exact sum, two products and the bias are at most 4 U of their
largest term off, and a subnormal result half a subnormal step."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _layer_plain as plain

pytestmark = pytest.mark.gpu

# one kernel each: few tokens (aligned, anywhere), weights as codes (whole, cut and joined), widened tiles
# (TMA stores, element stores, cut and joined)
SIZES = [(1, 40, 64), (3, 40, 65), (40, 300, 128), (40, 300, 1024), (40, 301, 333), (700, 4100, 1024), (700, 4101, 1030),
         (2100, 328, 136), (2100, 331, 136), (3000, 256, 4096)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_scales_whose_product_leaves_the_range(T, N, K, bias):
    import embedding_communication_codecs_gb300 as q
    rng = np.random.default_rng([T, N, K])
    lim = 16                                        # sums below 2^24: exact
    x = rng.integers(-lim, lim + 1, (T, K)).astype(np.int8)
    w = rng.integers(-lim, lim + 1, (N, K)).astype(np.int8)
    x[0] = 0                                        # a row of zeros, whose scale may be anything
    ex = rng.choice([-125, -100, -60, 0, 60, 100, 120], T)
    ew = rng.choice([-125, -100, -60, 0, 60, 100, 120], N)
    sx = (np.exp2(ex.astype(np.float64)) * rng.uniform(1, 2, T)).astype(np.float32)
    sw = (np.exp2(ew.astype(np.float64)) * rng.uniform(1, 2, N)).astype(np.float32)
    sx[0] = 2.0 ** 120
    sx[1 % T], sw[1] = (0.0 if T > 1 else sx[0]), 0.0
    b = rng.standard_normal(N).astype(np.float32) if bias else None

    def cu(a):
        return torch.from_numpy(a).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        y = q.int8_matmul(cu(x), cu(sx), cu(w), cu(sw), None if b is None else cu(b), dtype=dtype).double().cpu().numpy()
        prod = (x.astype(np.float64) @ w.astype(np.float64).T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
        want = prod + (b.astype(np.float64) if bias else 0.0)
        rel = plain.U16 * 1.01 if dtype == torch.bfloat16 else 0.0
        tol = 3 * plain.U * np.abs(prod) + (plain.U * 1.01 + rel) * np.abs(want) + 2.0 ** -133
        big = np.finfo(np.float32).max
        inside = np.abs(prod) < big * (1 - 2.0 ** -7)
        bad = inside & ~(np.abs(y - want) <= tol)
        assert not bad.any(), f"{dtype}: {bad.sum()} of {inside.sum()} wrong, first {y[bad][:4]} for {want[bad][:4]}"
        out = np.abs(prod) > big * (1 + 2.0 ** -7)
        assert np.array_equal(np.isposinf(y[out]), prod[out] > 0) and np.isinf(y[out]).all()


def test_scales_that_are_not_finite():
    """A NaN scale reaches its row (or column) and nothing else, for every kernel."""
    import embedding_communication_codecs_gb300 as q
    for T, N, K in SIZES:
        x = torch.ones((T, K), dtype=torch.int8, device="cuda")
        w = torch.ones((N, K), dtype=torch.int8, device="cuda")
        sx, sw = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
        sx[T - 1], sw[2] = float("nan"), float("nan")
        y = q.int8_matmul(x, sx, w, sw, dtype=torch.float32)
        want = torch.full((T, N), float(K), device="cuda")
        want[T - 1], want[:, 2] = float("nan"), float("nan")
        assert torch.equal(torch.nan_to_num(y, nan=-1.0), torch.nan_to_num(want, nan=-1.0))


@pytest.mark.parametrize("T,N,K", SIZES)
def test_subnormal_scales(T, N, K):
    """Scales below 2^-126, whole in fp32 whatever the other one is, against large ones."""
    import embedding_communication_codecs_gb300 as q
    rng = np.random.default_rng([T, N, K, 1])
    x = rng.integers(-16, 17, (T, K)).astype(np.int8)
    w = rng.integers(-16, 17, (N, K)).astype(np.int8)
    small = (rng.integers(1, 1 << 22, T).astype(np.uint32)).view(np.float32)       # subnormal
    large = (np.exp2(rng.integers(100, 127, N).astype(np.float64)) * rng.uniform(1, 1.9, N)).astype(np.float32)
    for sx, sw in ((small, large), (np.resize(large, T), np.resize(small, N))):
        y = q.int8_matmul(*(torch.from_numpy(a).cuda() for a in (x, sx, w, sw)), dtype=torch.float32).double().cpu().numpy()
        want = (x.astype(np.float64) @ w.astype(np.float64).T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
        # two roundings of the three fractions, and a subnormal result's own
        assert (np.abs(y - want) <= 3 * plain.U * np.abs(want) + 2.0 ** -149).all()
