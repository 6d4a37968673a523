"""CPU oracle of the int4-g64 key/value cache, its attention and the int4-g64
linear projection (plain numpy, fp64).

TEST INFRASTRUCTURE, like moe_oracle.py: imports nothing from the product path.

Definitions
  quantise  per group of 64 channels x (fp32 values): b = bf16(min x) (a
            zero is +0), s = bf16(fp32(fp32(max x - b) * fp32(1/15))), 0 below 2^-126; code =
            (fp32(x - b) / s) rounded to nearest, ties to even, clamped to
            0..15 (0 where s = 0). A group with a NaN or an infinity, or whose
            bias or span overflows, has s = b = NaN and codes 0.
  value     s * code + b
  attention softmax over the seen positions of scale * q . k, weighted sum of
            v; a query that sees nothing gives zeros
  linear    act(x W^T + bias) + residual, W = bf16(fp32(s * code + b))
"""
from __future__ import annotations

import math

import numpy as np

from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits

GROUP = 64
NAN_BITS = 0x7FC0


def _bf16(v):
    """bf16 bits of fp32 values, and their value in fp32."""
    bits = round_to_bf16_bits(np.asarray(v, dtype=np.float64))
    return bits, bf16_to_f64(bits).astype(np.float32)


def quantise(x: np.ndarray):
    """x fp32 [..., D] -> codes uint8 [..., D] (one a byte), scale and bias bits [..., D/64]."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1) + np.float32(0.0), g.max(-1)  # a zero minimum is +0
        b_bits, b = _bf16(lo)
        span = hi - b
        s_bits, s = _bf16(span * np.float32(1.0 / 15.0))
        bad = ~np.isfinite(g).all(-1) | ~np.isfinite(b) | ~np.isfinite(span)
        zero = ~(s >= np.float32(2.0 ** -126))
        s_bits = np.where(zero, 0, s_bits)
        t = (g - b[..., None]).astype(np.float64)
        d = np.where(zero | bad, 1.0, s.astype(np.float64))
        q = np.clip(np.rint(np.where(bad[..., None], 0.0, t) / d[..., None]), 0, 15)
    q = np.where((zero | bad)[..., None], 0, q).astype(np.uint8).reshape(x.shape)
    return (q, np.where(bad, NAN_BITS, s_bits).astype(np.uint16),
            np.where(bad, NAN_BITS, b_bits).astype(np.uint16))


def pack(q: np.ndarray) -> np.ndarray:
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes: np.ndarray) -> np.ndarray:
    q = np.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=np.uint8)
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    return q


def values(codes, s_bits, b_bits) -> np.ndarray:
    """fp64 [..., D] of packed codes [..., D/2] and bf16 bits [..., D/64]."""
    s = np.repeat(bf16_to_f64(s_bits), GROUP, axis=-1)
    b = np.repeat(bf16_to_f64(b_bits), GROUP, axis=-1)
    return s * unpack(codes) + b


def token_slots(cu, kv_len, table, page, T):
    """(sequence, page, slot) of each of T token rows; page -1 where it has no place, and
    sequence -1 for rows past the last one."""
    seq, pg, sl = (np.full(T, -1, dtype=np.int64) for _ in range(3))
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t, pos = cu[b] + i, int(kv_len[b]) - n + i
            seq[t] = b
            if 0 <= pos < table.shape[1] * page:
                pg[t], sl[t] = table[b, pos // page], pos % page
    return seq, pg, sl


class Paged:
    """A paged cache (codes [pages, H, page, D/2], scale and bias bits [pages, H, page, D/64]
    of k and of v) seen through a page table; entries outside the cache have no place."""

    def __init__(self, k, v, table):
        self.planes, self.table = {"k": k, "v": v}, np.asarray(table)
        self.pages, self.heads, self.page, _ = k[0].shape

    def rows(self, name, b, h, n):
        """(codes [n, D], scale [n, D], bias [n, D]) of the first n positions, and which exist."""
        pos = np.arange(n)
        inside = pos < self.table.shape[1] * self.page
        pg = self.table[b, np.where(inside, pos, 0) // self.page]
        ok = inside & (pg >= 0) & (pg < self.pages)
        at = (np.where(ok, pg, 0), h, pos % self.page)
        c, s, z = (a[at] for a in self.planes[name])
        return (unpack(c).astype(np.float64), np.repeat(bf16_to_f64(s), GROUP, -1),
                np.repeat(bf16_to_f64(z), GROUP, -1), ok)


def attention(q, cache, cu, kv_len, scale, causal=True, window=0):
    """out fp64 [T, Hq, D], and what an implementation may be off by, element by element:
      2^-8 |out|                     the result's rounding to bf16,
      2^-8 sum p s |code - 8|        each weight p s rounded to bf16,
      (n + 64) 2^-24 sum p (55 s + |b|)   fp32 sums of n keys with codes kept as 16 + code,
      2 d sum p |v|                  scores off by d: fp32 sums of 64 products with codes as
                                     16 + code, and an exponential good to 2^-22 of its range.
    """
    T, Hq, D = q.shape
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    G = Hq // cache.heads
    for b in range(len(kv_len)):
        n, total = cu[b + 1] - cu[b], int(kv_len[b])
        if n == 0:
            continue
        pos = np.arange(total)
        at = total - n + np.arange(n)[:, None]
        for h in range(cache.heads):
            kc, ks, kb, ok = cache.rows("k", b, h, total)
            vc, vs, vb, _ = cache.rows("v", b, h, total)
            see = np.broadcast_to(ok, (n, total)).copy()
            if causal:
                see &= pos <= at
            if window:
                see &= pos > at - window
            some = see.any(1)
            # what no query sees is dropped before any arithmetic
            keep = see.any(0)
            kc, ks, kb, vc, vs, vb = (a[keep] for a in (kc, ks, kb, vc, vs, vb))
            see = see[:, keep]
            for g in range(h * G, (h + 1) * G):
                rows = slice(cu[b], cu[b] + n)
                x = q[rows, g]
                if not some.any():
                    continue
                z = np.where(see, scale * (x @ (ks * kc + kb).T), -np.inf)
                top = np.where(some, z.max(1), 0.0)[:, None]
                p = np.exp(z - top)
                p /= np.where(some, p.sum(1), 1.0)[:, None]
                v = vs * vc + vb
                o = weigh(p, v)
                d = scale * 80 * 2.0 ** -24 * (np.abs(x) @ (47 * np.abs(ks) + np.abs(kb)).T)
                d = np.where(see, d + 2.0 ** -22 * (np.abs(np.where(see, z, 0)) + 1), 0).max(1)[:, None]
                out[rows, g] = o
                tol[rows, g] = (2.0 ** -8 * (np.abs(o) + weigh(p, np.abs(vs * (vc - 8))))
                                + (total + 64) * 2.0 ** -24 * weigh(p, 55 * np.abs(vs) + np.abs(vb))
                                + 2 * d * weigh(p, np.abs(v)))
    return out, tol


def weigh(p, v):
    """p @ v where a weight of zero takes nothing, whatever v holds there."""
    if np.isfinite(v).all():
        return p @ v
    return np.array([row[row != 0] @ v[row != 0] for row in p])


ACT = {
    "none": lambda z: z,
    "relu": lambda z: np.maximum(z, 0.0),
    "silu": lambda z: z / (1.0 + np.exp(-z)),
    "gelu": lambda z: 0.5 * z * (1.0 + np.vectorize(math.erf)(z / math.sqrt(2.0))),
}


def weights(codes, s_bits, b_bits) -> np.ndarray:
    """The projection's weights: fp32(s q + b) rounded to bf16, as fp64."""
    w = values(codes, s_bits, b_bits).astype(np.float32)
    return bf16_to_f64(round_to_bf16_bits(w.astype(np.float64)))


def linear(x, w, bias=None, act="none", residual=None):
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = ACT[act](z)
    return y if residual is None else y + residual
