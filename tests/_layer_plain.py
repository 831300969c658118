"""The 8-bit layer's formulas in 64 bits (numpy), and the tolerances of its kernels.

Shares no code with the package: scales come from frexp, products from float64
matmul, the gated activation from its definition."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # half a unit in the last place of fp32, relative
U16 = 2.0 ** -8          # the same of bf16: 8 significant bits, as fp32 has 24


def row_codes(x):
    """(codes int8, scale float32) of the rows of x."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, dtype=np.int8)
    scale = np.zeros(x.shape[0], dtype=np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            scale[r] = np.nan
            continue
        a = np.abs(row).max()
        if a == 0:
            continue
        s = 2.0 ** -126
        _, e = np.frexp(a)             # a in [2^(e-1), 2^e)
        s = max(s, 2.0 ** (int(e) - 7))
        if a / s >= 127.5:
            s *= 2
        s = min(s, 2.0 ** 121)         # 127 s stays finite; codes saturate
        codes[r] = np.clip(np.rint(row / s), -127, 127).astype(np.int8)
        scale[r] = s
    return codes, scale


def decoded(codes, scale):
    with np.errstate(invalid="ignore"):
        return codes.astype(np.float64) * scale.astype(np.float64)[:, None]


def sum_error(terms, length):
    """Bound on an fp32 sum of `length` exact products in any order, whether each
    addition rounds to nearest or truncates (one unit in the last place each);
    `terms` is the sum of the products' magnitudes."""
    return (length + 1) * 2 * U * terms


def rounded(y, bf16):
    """Bound on rounding y once to the output's type."""
    return np.abs(y) * (U16 if bf16 else U) + 2.0 ** -133


def bf16_to_f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def silu(g):
    return g / (1.0 + np.exp(-g))


def swiglu(g, u):
    return silu(g) * u


def swiglu_grad(g, u, dh):
    sig = 1.0 / (1.0 + np.exp(-g))
    return dh * u * (sig + g * sig * (1.0 - sig)), dh * g * sig
