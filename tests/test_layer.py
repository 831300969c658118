"""The 8-bit layer on the GPU against its formulas in 64 bits.

Integer-valued cases, whose sums stay below 2^24, have one right answer in fp32
whatever the order of the additions, and are compared bit for bit; the others are
held to bounds that follow from the arithmetic (tests/_layer_plain.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _layer_plain as plain

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def q():
    import embedding_communication_codecs_gb300 as q
    return q


def cu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def rng_of(*key):
    return np.random.default_rng([int(k) for k in key])


def strided(rows, dim, dtype, extra, lead=0, fill=-7.0):
    """A rows x dim view with `extra` elements between rows, starting `lead` elements
    into its buffer, and the buffer."""
    base = torch.full((rows * (dim + extra) + lead + 64,), fill, dtype=dtype, device="cuda")
    return base[lead:lead + rows * (dim + extra)].view(rows, dim + extra)[:, :dim], base


def untouched(base, view, fill=-7.0):
    """Every element of base outside view still holds the fill value."""
    keep = torch.ones_like(base, dtype=torch.bool)
    off = view.storage_offset() - base.storage_offset()
    torch.as_strided(keep, view.shape, view.stride(), off)[:] = False
    return bool((base[keep] == fill).all())


def check(got, want, tol, what=""):
    d = np.abs(got - want)
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst {np.nanmax(d / tol):.3g} of the bound"


# --------------------------------------------------------------- row codes

ROWS = [(1, 1), (1, 4096), (3, 5), (7, 33), (5, 128), (4, 129), (33, 1000), (9, 1001), (2, 8192), (3, 8200),
        (2, 20000), (40, 64), (1000, 16), (6, 2056)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", ROWS)
def test_row_codes(q, rows, dim, dtype):
    g = rng_of(rows, dim, dtype == BF16)
    x = g.standard_normal((rows, dim)) * np.exp2(g.integers(-100, 100, (rows, 1)).astype(np.float64))
    x[0] = 0.0
    t = cu(x.astype(np.float32), dtype)
    codes, scale = q.rowwise_int8(t)
    want, ws = plain.row_codes(f64(t))
    assert np.array_equal(scale.cpu().numpy(), ws)
    assert np.array_equal(codes.cpu().numpy(), want)
    for out in (F32, BF16):        # a power of two times at most 7 bits: exact in both
        assert np.array_equal(f64(q.rowwise_int8_dequant(codes, scale, dtype=out)), plain.decoded(want, ws))


def test_row_codes_at_the_edges(q):
    """Largest magnitudes either side of the step to the next power of two, ties,
    subnormals, the type's largest value, and rows that are not finite."""
    big = np.finfo(np.float32).max
    rows = np.zeros((14, 24), dtype=np.float32)
    rows[0, :3] = [127.5, 1, -0.5]                     # 127.5: the next scale
    rows[1, :3] = [np.nextafter(np.float32(127.5), np.float32(0)), 0.5, 1.5]
    rows[2, :4] = [127, 0.5, 1.5, 2.5]                 # ties go to even
    rows[3, :3] = [-127, -0.5, -1.5]
    rows[4, :2] = [1e-45, -1e-45]
    rows[5, :2] = [2.0 ** -126, 2.0 ** -127]
    rows[6, :2] = [big, -big / 3]
    rows[7, 5] = np.nan
    rows[8, 23] = np.inf
    rows[9, 0] = -np.inf
    rows[10, :2] = [np.nan, np.inf]
    rows[11, 20] = -1e-30
    rows[12, :2] = [64, 63.5]
    rows[13, :2] = [-0.0, 0.0]
    codes, scale = q.rowwise_int8(cu(rows))
    want, ws = plain.row_codes(rows)
    assert np.array_equal(scale.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want)
    back = f64(q.rowwise_int8_dequant(codes, scale, dtype=F32))
    assert np.isnan(back[7:11]).all() and np.isfinite(back[:7]).all() and np.isfinite(back[11:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,extra,lead", [(128, 8, 0), (100, 3, 1), (1000, 24, 5), (64, 1, 3), (1, 1, 0), (4096, 16, 8)])
def test_row_codes_of_strided_rows(q, dim, extra, lead, dtype):
    rows = 9
    g = rng_of(dim, extra, lead)
    x, base = strided(rows, dim, dtype, extra, lead, fill=1e30)   # what lies between the rows is not read
    x.copy_(cu(g.standard_normal((rows, dim)).astype(np.float32)))
    codes, scale = q.rowwise_int8(x)
    want, ws = plain.row_codes(f64(x))
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scale.cpu().numpy(), ws)
    out, obase = strided(rows, dim, dtype, extra, lead)
    code = q.QC_DTYPE_BF16 if dtype == BF16 else q.QC_DTYPE_F32
    q.qc_rowwise_int8_dequant(codes, scale, rows, dim, out, code, dim + extra)
    assert np.array_equal(f64(out), plain.decoded(want, ws))
    assert untouched(obase, out)
    # codes that start anywhere
    cbase = torch.zeros(rows * dim + 16, dtype=torch.int8, device="cuda")
    q.qc_rowwise_int8(x, code, dim + extra, rows, dim, cbase[lead:lead + rows * dim], scale)
    assert np.array_equal(cbase[lead:lead + rows * dim].cpu().numpy().reshape(rows, dim), want)
    assert not cbase[:lead].any() and not cbase[lead + rows * dim:].any()


def test_dequant_of_other_scales(q):
    """Scales that are not powers of two: one rounding to the output's type."""
    g = rng_of(5)
    codes = g.integers(-128, 128, (7, 300)).astype(np.int8)
    scale = g.standard_normal(7).astype(np.float32)
    want = plain.decoded(codes, scale)
    check(f64(q.rowwise_int8_dequant(cu(codes), cu(scale), dtype=F32)), want, plain.rounded(want, False))
    # bf16 after the fp32 product: two roundings
    check(f64(q.rowwise_int8_dequant(cu(codes), cu(scale), dtype=BF16)), want,
          plain.rounded(want, True) * (1 + 2.0 ** -10))


# ---------------------------------------------------------------- products

PRODUCTS = [(1, 1, 1), (1, 64, 64), (1, 257, 4096), (1, 33, 1001), (2, 16, 32), (3, 130, 259), (4, 1000, 512),
            (7, 64, 2056), (8, 500, 1504), (9, 129, 96), (16, 256, 1024), (17, 40, 333), (24, 1100, 640),
            (31, 65, 130), (33, 128, 257), (48, 1000, 512), (64, 256, 256), (65, 77, 1000), (100, 300, 200),
            (128, 128, 64), (129, 257, 385), (200, 1031, 72), (255, 256, 1000), (256, 512, 2048),
            (300, 520, 1030), (513, 768, 1025), (1000, 264, 520), (2049, 130, 261),
            (2050, 66, 2500), (2100, 328, 136)]


def int_case(T, N, K, kind):
    """Codes over all of int8 whose products' sums stay below 2^24, scales all 1."""
    g = rng_of(T, N, K, kind)
    lim = 128 if K * 16384 < 2 ** 24 else 64 if K * 4096 < 2 ** 24 else 32
    x = g.integers(-lim, lim, (T, K)).astype(np.int8)
    w = g.integers(-lim, lim, (N, K)).astype(np.int8)
    return g, x, w


@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_matmul_integers(q, T, N, K):
    _, x, w = int_case(T, N, K, 0)
    y = q.int8_matmul(cu(x), torch.ones(T, device="cuda"), cu(w), torch.ones(N, device="cuda"), dtype=F32)
    assert np.array_equal(f64(y), x.astype(np.float64) @ w.astype(np.float64).T)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_matmul_scales(q, T, N, K, bias, bf16):
    """Any fp32 scales, on both axes, and a bias."""
    g = rng_of(T, N, K, bias, bf16)
    x = g.integers(-128, 128, (T, K)).astype(np.int8)
    w = g.integers(-128, 128, (N, K)).astype(np.int8)
    sx = np.exp(g.standard_normal(T) - 3).astype(np.float32)
    sw = np.exp(g.standard_normal(N) - 3).astype(np.float32)
    b = g.standard_normal(N).astype(np.float32) if bias else None
    y = q.int8_matmul(cu(x), cu(sx), cu(w), cu(sw), None if b is None else cu(b), dtype=BF16 if bf16 else F32)
    s = sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    want = x.astype(np.float64) @ w.astype(np.float64).T * s
    terms = np.abs(x.astype(np.float64)) @ np.abs(w.astype(np.float64)).T * s
    tol = (plain.sum_error(terms, K) if K * 16384 >= 2 ** 24 else 0) + 3 * plain.U * np.abs(want)
    if bias:
        want = want + b.astype(np.float64)
    check(f64(y), want, (tol + plain.rounded(want, False)) + (1.01 * plain.rounded(want, True) + tol if bf16 else 0))


def bf16_ints(g, lim, shape):
    return g.integers(-lim, lim + 1, shape).astype(np.float32)


@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_gradients_integers(q, T, N, K):
    """dy of small integers and scales that are small powers of two: exact."""
    g = rng_of(T, N, K, 3)
    dy = bf16_ints(g, 2, (T, N))
    x = g.integers(-127, 128, (T, K)).astype(np.int8)
    w = g.integers(-127, 128, (N, K)).astype(np.int8)
    sx = np.exp2(g.integers(-1, 2, T)).astype(np.float32)
    sw = np.exp2(g.integers(-1, 2, N)).astype(np.float32)
    dyc = cu(dy, BF16)
    dx = q.int8_input_grad(dyc, cu(w), cu(sw), dtype=F32)
    assert np.array_equal(f64(dx), dy.astype(np.float64) @ plain.decoded(w, sw))
    dw, db = q.int8_weight_grad(dyc, cu(x), cu(sx), with_bias=True)
    assert np.array_equal(f64(dw), dy.astype(np.float64).T @ plain.decoded(x, sx))
    assert np.array_equal(f64(db), dy.astype(np.float64).sum(0))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_gradients_real(q, T, N, K, bf16):
    """Codes and scales as rowwise_int8 makes them, bf16 gradients."""
    g = rng_of(T, N, K, 4)
    out = BF16 if bf16 else F32
    xc, xs = q.rowwise_int8(cu(g.standard_normal((T, K)).astype(np.float32)))
    wc, ws = q.rowwise_int8(cu((g.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32)))
    dy = cu((1e-3 * g.standard_normal((T, N))).astype(np.float32), BF16)
    d = f64(dy)
    X, W = plain.decoded(xc.cpu().numpy(), xs.cpu().numpy()), plain.decoded(wc.cpu().numpy(), ws.cpu().numpy())
    want = d @ W
    tol = plain.sum_error(np.abs(d) @ np.abs(W), N)
    check(f64(q.int8_input_grad(dy, wc, ws, dtype=out)), want, tol + 1.01 * plain.rounded(np.abs(want) + tol, bf16))
    dw, db = q.int8_weight_grad(dy, xc, xs, dtype=out, with_bias=True)
    want = d.T @ X
    tol = plain.sum_error(np.abs(d).T @ np.abs(X), T)
    check(f64(dw), want, tol + 1.01 * plain.rounded(np.abs(want) + tol, bf16))
    check(f64(db), d.sum(0), plain.sum_error(np.abs(d).sum(0), T) + 1e-40)


@pytest.mark.parametrize("T,N,K", [(5, 24, 40), (130, 200, 264)])
def test_weight_grad_accumulates(q, T, N, K):
    g = rng_of(T, N, K, 5)
    dy = bf16_ints(g, 2, (T, N))
    x = g.integers(-127, 128, (T, K)).astype(np.int8)
    dw0, db0 = bf16_ints(g, 100, (N, K)), bf16_ints(g, 100, N)
    dw, db = cu(dw0), cu(db0)
    got = q.int8_weight_grad(cu(dy, BF16), cu(x), torch.ones(T, device="cuda"), into=(dw, db))
    assert got[0] is dw and got[1] is db
    assert np.array_equal(f64(dw), dw0 + dy.astype(np.float64).T @ x.astype(np.float64))
    assert np.array_equal(f64(db), db0 + dy.astype(np.float64).sum(0))
    q.int8_weight_grad(cu(dy, BF16), cu(x), torch.ones(T, device="cuda"), into=(dw, None))
    assert np.array_equal(f64(dw), dw0 + 2 * dy.astype(np.float64).T @ x.astype(np.float64))


def test_no_tokens(q):
    N, K = 24, 40
    w, sw = torch.ones((N, K), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    none = torch.empty((0, K), dtype=torch.int8, device="cuda")
    s0 = torch.empty(0, device="cuda")
    assert q.int8_matmul(none, s0, w, sw).shape == (0, N)
    dy = torch.empty((0, N), dtype=BF16, device="cuda")
    assert q.int8_input_grad(dy, w, sw).shape == (0, K)
    for dtype in (F32, BF16):
        dw, db = q.int8_weight_grad(dy, none, s0, dtype=dtype, with_bias=True)
        assert not dw.any() and not db.any()
    dw, db = torch.full((N, K), 3.0, device="cuda"), torch.full((N,), 4.0, device="cuda")
    q.int8_weight_grad(dy, none, s0, into=(dw, db))
    assert bool((dw == 3).all()) and bool((db == 4).all())
    codes, scale = q.rowwise_int8(torch.empty((0, K), device="cuda"))
    assert codes.shape == (0, K) and q.rowwise_int8_dequant(codes, scale).shape == (0, K)
    got = q.swiglu_encode(torch.empty((0, 2 * K), device="cuda"))
    assert q.swiglu_backward(torch.empty((0, K), device="cuda"), got[2], got[3]).shape == (0, 2 * K)


@pytest.mark.parametrize("T,N,K", [(3, 40, 64), (20, 136, 200), (140, 264, 320)])
def test_rows_that_are_not_finite(q, T, N, K):
    """A row of codes with a NaN scale makes its own outputs NaN and no others; in the
    weight gradient it reaches every weight."""
    g = rng_of(T, N, K, 6)
    x = g.standard_normal((T, K)).astype(np.float32)
    x[1, 3] = np.inf
    xc, xs = q.rowwise_int8(cu(x))
    wc, ws = q.rowwise_int8(cu(g.standard_normal((N, K)).astype(np.float32)))
    y = f64(q.int8_matmul(xc, xs, wc, ws))
    assert np.isnan(y[1]).all() and np.isfinite(np.delete(y, 1, 0)).all()
    dy = cu(g.standard_normal((T, N)).astype(np.float32), BF16)
    assert np.isnan(f64(q.int8_weight_grad(dy, xc, xs)[0])).all()
    dy[2, 5] = float("inf")
    dx = f64(q.int8_input_grad(dy, wc, ws))
    assert not np.isfinite(dx[2]).any()      # infinity times a zero weight is NaN
    assert np.isfinite(np.delete(dx, 2, 0)).all()


@pytest.mark.parametrize("T,N,K,extra,lead", [(6, 40, 72, 8, 0), (6, 41, 71, 3, 1), (33, 130, 100, 1, 3),
                                              (140, 256, 264, 8, 8), (140, 257, 263, 5, 1), (130, 64, 128, 0, 4)])
@pytest.mark.parametrize("bf16", [False, True])
def test_products_of_strided_and_shifted_buffers(q, T, N, K, extra, lead, bf16):
    """Rows with gaps, buffers that start anywhere, codes off every alignment; the
    gaps are neither read (they hold 1e30) nor written."""
    g = rng_of(T, N, K, extra, lead, bf16)
    out, code = (BF16, q.QC_DTYPE_BF16) if bf16 else (F32, q.QC_DTYPE_F32)

    def shifted(a):
        base = torch.zeros(a.size + 64, dtype=torch.int8, device="cuda")
        v = base[lead:lead + a.size]
        v.copy_(cu(a).reshape(-1))
        return v

    x = g.integers(-32, 32, (T, K)).astype(np.int8)
    w = g.integers(-32, 32, (N, K)).astype(np.int8)
    dyv, _ = strided(T, N, BF16, extra, lead, fill=1e30)
    dy = bf16_ints(g, 2, (T, N))
    dyv.copy_(cu(dy))
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")

    def ws(n):
        return torch.full((n + 256,), 0x7F, dtype=torch.uint8, device="cuda")[:n]   # 256-byte aligned; NaN patterns

    y, ybase = strided(T, N, out, extra, lead)
    n = q.qc_int8_matmul_workspace(T, N, K)
    q.qc_int8_matmul(shifted(x), one_t, shifted(w), one_n, None, T, N, K, y, code, N + extra, ws(n), n)
    X, W, D = x.astype(np.float64), w.astype(np.float64), dy.astype(np.float64)

    def same(got, want):
        assert np.array_equal(f64(got), f64(cu(want).to(out)))
    same(y, X @ W.T)
    assert untouched(ybase, y)
    dx, dxbase = strided(T, K, out, extra, lead)
    n = q.qc_int8_input_grad_workspace(T, N, K)
    q.qc_int8_input_grad(dyv, N + extra, shifted(w), one_n, T, N, K, dx, code, K + extra, ws(n), n)
    same(dx, D @ W)
    assert untouched(dxbase, dx)
    dwbase = torch.full((N * K + lead + 64,), -7.0, dtype=out, device="cuda")
    dw = dwbase[lead:lead + N * K].view(N, K)
    n = q.qc_int8_weight_grad_workspace(T, N, K)
    q.qc_int8_weight_grad(dyv, N + extra, shifted(x), one_t, T, N, K, dw, code, None, 0, ws(n), n)
    same(dw, D.T @ X)
    assert untouched(dwbase, dw)


def test_gradients_against_differences(q):
    """The layer's gradients are those of its forward formula: difference quotients of
    sum(r * y), in 64 bits, by the decoded inputs and weights."""
    T, N, K = 12, 20, 28
    g = rng_of(7)
    xc, xs = q.rowwise_int8(cu(g.standard_normal((T, K)).astype(np.float32)))
    wc, ws = q.rowwise_int8(cu(g.standard_normal((N, K)).astype(np.float32)))
    r = cu(g.standard_normal((T, N)).astype(np.float32), BF16)
    X, W, R = plain.decoded(xc.cpu().numpy(), xs.cpu().numpy()), plain.decoded(wc.cpu().numpy(), ws.cpu().numpy()), f64(r)
    loss = lambda X, W: float((R * (X @ W.T)).sum())   # noqa: E731
    dx = f64(q.int8_input_grad(r, wc, ws, dtype=F32))
    dw = f64(q.int8_weight_grad(r, xc, xs)[0])
    for _ in range(20):
        t, n, k = int(g.integers(T)), int(g.integers(N)), int(g.integers(K))
        for A, grad, at in ((X, dx, (t, k)), (W, dw, (n, k))):
            hi, lo = A.copy(), A.copy()
            hi[at] += 0.5
            lo[at] -= 0.5
            diff = loss(hi if A is X else X, hi if A is W else W) - loss(lo if A is X else X, lo if A is W else W)
            # the loss is linear in A: the quotient is exact up to 64-bit rounding; the kernel's sum has
            # at most 28 terms of about 4 each
            assert abs(diff - grad[at]) <= 29 * 2 * plain.U * 28 * 16 + 1e-9


# ------------------------------------------------------------------ swiglu

SWIGLU = [(1, 1), (1, 64), (3, 7), (5, 128), (33, 1408), (4, 1001), (2, 8192), (3, 11008), (2, 20000), (300, 40)]

# silu(g) * u in fp32: an exponential within 4 units in the last place (2 from the
# function and |g| < 16 times half a unit of the rounded argument are together
# below 2^-19), one division and one product: 2^-18 relative covers them.
H_REL = 2.0 ** -18


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", SWIGLU)
def test_swiglu(q, rows, dim, dtype):
    g = rng_of(rows, dim, dtype == BF16, 8)
    gu = g.standard_normal((rows, 2 * dim)) * 2
    gu[-1, :dim] = 0.0                                  # a row of zero gates: h is zero
    t = cu(gu.astype(np.float32), dtype)
    hc, hs, sc, ss = q.swiglu_encode(t)
    v = f64(t)
    gate, up = v[:, :dim], v[:, dim:]
    gc, gs = plain.row_codes(gate)
    uc, us = plain.row_codes(up)
    assert np.array_equal(sc.cpu().numpy(), np.concatenate([gc, uc], 1))
    assert np.array_equal(ss.cpu().numpy(), np.stack([gs, us], 1))
    h = plain.swiglu(gate, up)
    scale = hs.cpu().numpy().astype(np.float64)
    got = plain.decoded(hc.cpu().numpy(), hs.cpu().numpy())
    # the scale is the power of two for the row's maximum, or its neighbour where that is within H_REL of the step
    a = np.abs(h).max(1)
    for r in range(rows):
        lo, hi = (plain.row_codes(np.array([[a[r] * f]]))[1][0] for f in (1 - H_REL, 1 + H_REL))
        assert scale[r] in (lo, hi), (r, scale[r], lo, hi)
    check(got, h, 0.5 * scale[:, None] + np.abs(h) * H_REL + 1e-44)
    dh = cu((1e-2 * g.standard_normal((rows, dim))).astype(np.float32), dtype)
    d = f64(q.swiglu_backward(dh, sc, ss))
    G, U_ = plain.decoded(gc, gs), plain.decoded(uc, us)
    dg, du = plain.swiglu_grad(G, U_, f64(dh))
    bf = dtype == BF16
    # slope = sig (1 + g (1 - sig)) cancels where it is near zero (g near -1.28): its error is absolute,
    # a few units of its terms sig and sig |g| (1 - sig), both below 1
    for got_, want, size in ((d[:, :dim], dg, np.abs(f64(dh) * U_) * (1 + np.abs(G))), (d[:, dim:], du, np.abs(du))):
        check(got_, want, 1.01 * plain.rounded(want, bf) + size * H_REL + 1e-40)


def test_swiglu_extremes(q):
    """Gates far out: silu saturates to g or to zero without overflow; rows that are
    not finite decode to NaN and touch no other row."""
    v = np.array([[1e4, -1e4, 88.8, -88.8, 1.0, -1.0, 0.0, -0.0],
                  [np.nan, 1, 1, 1, 1, 1, 1, 1],
                  [1, 1, 1, np.inf, 1, 1, 1, 1],
                  [1, 1, 1, 1, -np.inf, 1, 1, 1],
                  [0.5] * 8], dtype=np.float32)
    up = np.ones_like(v)
    up[4, 2] = np.nan
    hc, hs, sc, ss = q.swiglu_encode(cu(np.concatenate([v, up], 1)))
    h = f64(q.rowwise_int8_dequant(hc, hs, dtype=F32))
    with np.errstate(over="ignore", invalid="ignore"):
        want = plain.swiglu(v[0].astype(np.float64), 1.0)
    check(h[0], want, 0.5 * float(hs[0]) + 1e-6)
    assert np.isnan(h[1:]).all()
    s = ss.cpu().numpy()
    assert np.isnan(s[1:4, 0]).all() and np.isfinite(s[1:4, 1]).all()
    assert np.isfinite(s[4, 0]) and np.isnan(s[4, 1]) and np.isfinite(s[0]).all()
    d = f64(q.swiglu_backward(torch.ones((5, 8), device="cuda"), sc, ss))
    assert np.isfinite(d[0]).all() and np.isnan(d[1:4, :8]).all() and np.isnan(d[4, :8]).all()
    assert np.isfinite(d[4, 8:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,extra,lead", [(64, 8, 0), (33, 3, 1), (1000, 24, 8), (128, 1, 3)])
def test_swiglu_of_strided_rows(q, dim, extra, lead, dtype):
    rows = 7
    g = rng_of(dim, extra, lead, 9)
    x, _ = strided(rows, 2 * dim, dtype, extra, lead, fill=1e30)
    x.copy_(cu(g.standard_normal((rows, 2 * dim)).astype(np.float32)))
    dh, _ = strided(rows, dim, dtype, extra, lead, fill=1e30)
    dh.copy_(cu(g.standard_normal((rows, dim)).astype(np.float32)))
    strided_, dense = q.swiglu_encode(x), q.swiglu_encode(x.contiguous())
    for a, b in zip(strided_, dense):
        assert torch.equal(a, b)
    out, base = strided(rows, 2 * dim, dtype, extra, lead)
    code = q.QC_DTYPE_BF16 if dtype == BF16 else q.QC_DTYPE_F32
    q.qc_swiglu_backward(dh, code, dim + extra, dense[2], dense[3], rows, dim, out, 2 * dim + extra)
    assert torch.equal(out, q.swiglu_backward(dh.contiguous(), dense[2], dense[3]))
    assert untouched(base, out)


def test_swiglu_gradient_against_differences(q):
    """(dgate, dup) against central differences of sum(dh * h) in 64 bits."""
    g = rng_of(10)
    rows, dim = 4, 30
    _, _, sc, ss = q.swiglu_encode(cu((2 * g.standard_normal((rows, 2 * dim))).astype(np.float32)))
    codes, scale = sc.cpu().numpy(), ss.cpu().numpy()
    G, U_ = plain.decoded(codes[:, :dim], scale[:, 0]), plain.decoded(codes[:, dim:], scale[:, 1])
    dh = g.standard_normal((rows, dim)).astype(np.float32)
    d = f64(q.swiglu_backward(cu(dh), sc, ss))
    e = 1e-4
    dg = dh * (plain.swiglu(G + e, U_) - plain.swiglu(G - e, U_)) / (2 * e)
    du = dh * (plain.swiglu(G, U_ + e) - plain.swiglu(G, U_ - e)) / (2 * e)
    # e^2 / 6 times the third derivative (below 1 in magnitude) times |dh u|, and the kernel's rounding
    size = np.abs(dh) * (1 + np.abs(U_)) * (1 + np.abs(G))
    check(d[:, :dim], dg, size * (e * e + plain.U * 64 + 1e-9))
    check(d[:, dim:], du, size * (plain.U * 64 + 1e-9))


# ------------------------------------- the kernels that only larger sizes reach

def by_torch(codes, scale):
    return codes.double() * scale.double()[:, None]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", [(2000, 4096), (1001, 2056), (500, 8200), (460, 16384), (60000, 64), (3700, 1000),
                                      (1300, 4099), (70000, 71), (500, 9001)])
def test_many_rows(q, rows, dim, dtype):
    """Row counts that fill the device: the streaming gated activation and the ragged
    rows' one-warp teams, against torch in 64 bits; some rows are zero, infinite or NaN."""
    gen = torch.Generator(device="cuda").manual_seed(rows * 31 + dim)
    x = 2 * torch.randn((rows, 2 * dim), generator=gen, device="cuda")
    x[3] = 0
    x[7, dim + 1] = float("nan")
    x[rows - 1, 5] = float("inf")
    x = x.to(dtype)
    hc, hs, sc, ss = q.swiglu_encode(x)
    g, u = x[:, :dim].contiguous(), x[:, dim:].contiguous()
    for half, part in ((0, g), (1, u)):        # gate and up are coded as rows of their own
        codes, scale = q.rowwise_int8(part)
        assert torch.equal(sc[:, half * dim:(half + 1) * dim], codes)
        assert torch.equal(ss[:, half].view(torch.int32), scale.view(torch.int32))
        live = torch.isfinite(part).all(1)
        a = part.double().abs().amax(1)
        assert bool((torch.isnan(scale) == ~live).all())
        s = scale.double()[live]
        assert bool((torch.frexp(s)[0] == 0.5).logical_or(s == 0).all())
        assert bool(((a[live] < 127.5 * s) & (a[live] >= 63.75 * s)).logical_or(s == 0).all())
        err = (by_torch(codes, scale) - part.double()).abs()[live]
        assert bool((err <= 0.5 * s[:, None]).all())
    h = g.double() * torch.sigmoid(g.double()) * u.double()
    live = torch.isfinite(h).all(1)
    assert bool((torch.isnan(hs) == ~live).all())
    err = (by_torch(hc, hs) - h).abs()[live]
    assert bool((err <= 0.5 * hs.double()[live][:, None] + h.abs()[live] * H_REL + 1e-44).all())
    assert q.qc_take_device_errors() == 0


@pytest.mark.parametrize("T,N,K", [(20, 20000, 512), (100, 33000, 256), (300, 10000, 1024), (2100, 2300, 600),
                                   (4, 6000, 4096), (8, 4864, 320), (600, 512, 12000), (130, 128, 16384)])
def test_larger_products(q, T, N, K):
    """Several units of work to a block, split contractions with a short last range,
    every token tile: integers below 2^24 in all sums, so one right answer."""
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)

    def ints(lim, *shape):
        return torch.randint(-lim, lim + 1, shape, generator=gen, device="cuda")
    lim = 127 if K * 127 * 127 < 2 ** 24 else 32 if K * 32 * 32 < 2 ** 24 else 31
    x, w = ints(lim, T, K).to(torch.int8), ints(lim, N, K).to(torch.int8)
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    y = q.int8_matmul(x, one_t, w, one_n, dtype=F32)
    assert torch.equal(y.double(), x.double() @ w.double().t())
    dy = ints(2, T, N).to(BF16)
    assert torch.equal(q.int8_input_grad(dy, w, one_n, dtype=F32).double(), dy.double() @ w.double())
    dw, db = q.int8_weight_grad(dy, x, one_t, with_bias=True)
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))
    assert q.qc_take_device_errors() == 0


def test_long_sums_keep_their_precision(q):
    """A weight gradient over 16384 tokens: cut into parts, the sum's error stays that of
    a part of 2048 terms (each addition off by at most a unit in the last place of the
    running sum, which for terms of random sign is the root of their number times one)."""
    T, N, K = 16384, 256, 256
    gen = torch.Generator(device="cuda").manual_seed(3)
    xc, xs = q.rowwise_int8(torch.randn((T, K), generator=gen, device="cuda"))
    dy = torch.randn((T, N), generator=gen, device="cuda").to(BF16)
    dw, _ = q.int8_weight_grad(dy, xc, xs)
    want = dy.double().t() @ by_torch(xc, xs)
    # 2048 / 16 additions of at most 2^-23 of a sum no larger than the result, plus the joins
    assert float((dw.double() - want).norm() / want.norm()) <= (2048 / 16 + 8 + 16) * 2.0 ** -23


@pytest.mark.parametrize("T,N,K", [(300, 10000, 1024), (128, 33000, 1024), (96, 33000, 1024), (64, 33000, 4096),
                                   (48, 33000, 1024), (32, 33000, 1024)])
def test_many_units_many_times(q, T, N, K):
    """Every token tile with several units to a block and the memory busy, fifty times: the
    stages of codes are refilled as fast as they are given back."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    lim = 127 if K <= 1024 else 31
    x = torch.randint(-lim, lim + 1, (T, K), generator=gen, device="cuda").to(torch.int8)
    w = torch.randint(-lim, lim + 1, (N, K), generator=gen, device="cuda").to(torch.int8)
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    want = (x.double() @ w.double().t()).float()
    for _ in range(50):
        assert torch.equal(q.int8_matmul(x, one_t, w, one_n, dtype=F32), want)
    assert q.qc_take_device_errors() == 0


@pytest.mark.parametrize("T,N,K", [(5, 300, 131072), (12, 300, 131072), (30, 20000, 16384), (48, 20000, 16384), (64, 20000, 16384),
                                   (96, 20000, 16384), (128, 20000, 16384), (300, 20000, 16384), (700, 2000, 16384)])
def test_sums_of_one_sign_keep_their_precision(q, T, N, K):
    """Codes of 64 to 127 only, whose sums pass 2^24: each part of 2048 terms is 128 additions
    that lose at most a unit in the last place of a sum no larger than the result; the
    parts (up to 64) are added in fp32, and the scales are ones."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randint(64, 128, (T, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(64, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    y = q.int8_matmul(x, torch.ones(T, device="cuda"), w, torch.ones(N, device="cuda"), dtype=F32)
    for part in (slice(0, 200), slice(N - 200, N)):
        want = x.double() @ w[part].double().t()
        assert bool(((y[:, part].double() - want).abs() <= (128 + 64) * 2.0 ** -23 * want).all())
    assert q.qc_take_device_errors() == 0


# ------------------------------------------------------------ how it is run

def test_other_stream_and_repeat(q):
    """On a stream of its own behind a long queue of work, with the inputs made on that
    stream; twice, with equal bits."""
    s = torch.cuda.Stream()
    g = rng_of(11)
    x = cu(g.standard_normal((260, 520)).astype(np.float32))
    w = cu(g.standard_normal((300, 520)).astype(np.float32))
    r = cu(g.standard_normal((260, 300)).astype(np.float32))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            big = big @ big * 1e-3
        x2, w2, dy = x * 1.0, w * 1.0, r.to(BF16)
    runs = []
    for _ in range(2):
        xc, xs = q.rowwise_int8(x2, stream=s)
        wc, ws = q.rowwise_int8(w2, stream=s)
        y = q.int8_matmul(xc, xs, wc, ws, dtype=F32, stream=s.cuda_stream)
        y1 = q.int8_matmul(xc[:1], xs[:1], wc, ws, dtype=F32, stream=s)
        dx = q.int8_input_grad(dy, wc, ws, dtype=F32, stream=s)
        dw, db = q.int8_weight_grad(dy, xc, xs, with_bias=True, stream=s)
        runs.append((y, y1, dx, dw, db))
    s.synchronize()
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    X, W = plain.decoded(*plain.row_codes(f64(x))), plain.decoded(*plain.row_codes(f64(w)))
    y, y1, dx, dw, db = runs[0]
    D = f64(dy)
    for got, want, terms, n in ((y, X @ W.T, np.abs(X) @ np.abs(W).T, 520), (y1, X[:1] @ W.T, np.abs(X[:1]) @ np.abs(W).T, 520),
                                (dx, D @ W, np.abs(D) @ np.abs(W), 300), (dw, D.T @ X, np.abs(D).T @ np.abs(X), 260)):
        check(f64(got), want, plain.sum_error(terms, n) + 4 * plain.U * np.abs(want))
    assert q.qc_take_device_errors() == 0


def test_in_a_graph(q):
    """Every call captured once and replayed on new inputs."""
    g = rng_of(12)
    T, N, F = 140, 256, 128
    x = torch.zeros((T, 264), device="cuda")
    w1, w2 = (cu(g.standard_normal(s).astype(np.float32)) for s in ((2 * F, 264), (N, F)))
    (w1c, w1s), (w2c, w2s) = q.rowwise_int8(w1), q.rowwise_int8(w2)
    dy = torch.zeros((T, N), dtype=BF16, device="cuda")

    def step():
        xc, xs = q.rowwise_int8(x)
        hc, hs, sc, ss = q.swiglu_encode(q.int8_matmul(xc, xs, w1c, w1s))
        y = q.int8_matmul(hc, hs, w2c, w2s)
        dw2, db2 = q.int8_weight_grad(dy, hc, hs, with_bias=True)
        dgu = q.swiglu_backward(q.int8_input_grad(dy, w2c, w2s), sc, ss)
        return y, dw2, db2, q.int8_weight_grad(dgu, xc, xs)[0], q.int8_input_grad(dgu, w1c, w1s)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    x.copy_(cu(g.standard_normal((T, 264)).astype(np.float32)))
    dy.copy_(cu(g.standard_normal((T, N)).astype(np.float32)))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, step()):
        assert a.abs().sum() > 0 and torch.equal(a, b)
