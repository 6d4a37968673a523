"""CPU oracle of the norms, the rotary positions, the page bounds and the selection of
pages (plain numpy, fp64).

TEST INFRASTRUCTURE, like moe_oracle.py: imports nothing from the product path.

Definitions
  rmsnorm   y = s / sqrt(mean s^2 + eps) * w, s = x + residual
  rope      pairs (a, b) of the first rot channels -> m (a cos t - b sin t, a sin t + b cos t),
            t = position * freq; pairs are (2i, 2i + 1) or (i, i + rot / 2)
  bounds    per page, head and channel the smallest and largest key, a zero as +0, NaN where
            one is
  select    score = fp32(sum over heads and channels of max(q lo, q hi)); the first pages, the
            last ones and the best of the others, ties to the lower page, NaN last
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, w, eps, residual=None):
    s = x if residual is None else x + residual
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w, s


def norm_terms(d):
    """Relative error, in units of 2^-24, of y before its rounding: the sum s (1), its square root's
    argument (half of: twice s's, at most 32 products and 20 additions of partial sums of positive
    terms, the mean and eps), the root and its reciprocal, 1 + w and two products."""
    return 1 + 0.5 * (2 + 32 + 20 + 2) + 2 + 1 + 2


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rope(x, positions, freqs, interleaved=False, magnitude=1.0):
    """x fp64 [T, H, D]; also the sum of the two magnitudes that go into each value."""
    a, b = pairs(2 * len(freqs), interleaved)
    t = positions.astype(np.float64)[:, None, None] * freqs.astype(np.float64)
    c, s = magnitude * np.cos(t), magnitude * np.sin(t)
    y, size = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = magnitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def bounds(values, total):
    """values fp64 [pages, page, D] of one sequence and head, of which the first `total` rows count
    -> [pages, 2, D]."""
    n, page, D = values.shape
    out = np.zeros((n, 2, D))
    for i in range(n):
        v = values[i, :max(min(page, total - i * page), 0)]
        if len(v):
            out[i, 0], out[i, 1] = v.min(0), v.max(0)  # numpy's keep a NaN
    return out + 0.0


def select(q, lo, hi, exists, position, page, top, first, recent):
    """Pages [<= first + top + recent] that a token takes: q fp64 [heads, D], lo and hi [pages, D]."""
    last = min(position, len(exists) * page - 1)
    if last < 0:
        return np.zeros(0, dtype=np.int64)
    own = last // page
    c = np.arange(own + 1)
    scored = (c >= first) & (c <= own - recent)
    with np.errstate(all="ignore"):
        s = np.maximum(q[:, None] * lo[None, :own + 1], q[:, None] * hi[None, :own + 1]).sum((0, 2)).astype(np.float32)
    ok = exists[:own + 1]
    order = sorted((i for i in c if scored[i] and ok[i]),
                   key=lambda i: (np.isnan(s[i]), -s[i] if not np.isnan(s[i]) else 0.0, i))
    return np.sort(np.array([i for i in c if not scored[i] and ok[i]] + order[:top], dtype=np.int64))
