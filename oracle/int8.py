"""Oracle of the 8-bit path (numpy, fp64): row codes, the RMS norm that gives
them, and the int8 linears.

TEST INFRASTRUCTURE ONLY, like the rest of this package, sharing no code with
the CUDA library.

Row codes: a = max |v_c|, q_c = the whole number nearest to 127 v_c / a (ties
to even), scale a / 127; an all-zero row has codes 0 and scale 1; a row with an
infinity or NaN has codes 0 and scale NaN.  For values of at most 24
significant bits 127 v is exact in fp64 and a quotient that is not a tie is
further from one than fp64's rounding, so rint of the fp64 quotient is exact.
"""
from __future__ import annotations

import numpy as np


def row_codes(v):
    """(codes int8 [M, d], scales fp64 [M]) of fp64 rows that hold values of at most 24 bits."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a = np.abs(v).max(axis=1)
    ok = np.isfinite(v).all(axis=1)
    a = np.where(ok, a, 0.0)
    div = np.where(a > 0, a, 1.0)
    q = np.rint(127.0 * np.where(ok[:, None], v, 0.0) / div[:, None]).astype(np.int8)
    s = np.where(a > 0, a / 127.0, 1.0)
    return q, np.where(ok, s, np.nan)


def rms_norm_codes(h, gain=None, eps=1e-6):
    """Row codes of h_c g_c / sqrt(mean h^2 + eps) for hidden states h [M, d] already in their
    type; h g is taken as fp32 holds it (exact, or infinite beyond fp32)."""
    h = np.asarray(h, dtype=np.float64)
    g = np.ones(h.shape[1]) if gain is None else np.asarray(gain, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        v = (h * g[None, :]).astype(np.float32).astype(np.float64)
        q, s = row_codes(v)
        r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    zero = (np.abs(np.nan_to_num(v)).max(axis=1) == 0) & np.isfinite(v).all(axis=1)
    return q, np.where(zero, 1.0, s * r)


def w8a8_linear(q, sx, w, sw, bias=None):
    """y [M, d_out] in fp64."""
    whole = np.asarray(q, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T  # exact: below 2^53
    y = whole * np.asarray(sx, dtype=np.float64)[:, None] * np.asarray(sw, dtype=np.float64)[None, :]
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)[None, :]


def w8a8_swiglu(q, sx, wg, sg, wu, su):
    """(silu(gate) * up, gate, up) in fp64."""
    g, u = w8a8_linear(q, sx, wg, sg), w8a8_linear(q, sx, wu, su)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u, g, u
