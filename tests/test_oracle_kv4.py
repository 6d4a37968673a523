"""The cache, attention and projection oracle against hand-worked cases and properties (CPU)."""
import math

import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle.moe_oracle import bf16_to_f64


def group(values, fill):
    x = np.full(64, fill, dtype=np.float32)
    x[:len(values)] = values
    return x


def test_quantise_by_hand():
    # min 0, max 15: scale 1, codes the values themselves; 0.5, 1.5, 2.5 are ties to even
    q, s, b = K.quantise(group([0, 15, 7, 0.5, 1.5, 2.5, 2.4999], 3))
    assert q[:8].tolist() == [0, 15, 7, 0, 2, 2, 2, 3]
    assert bf16_to_f64(s).tolist() == [1.0] and bf16_to_f64(b).tolist() == [0.0]


def test_quantise_constant_group_has_no_scale():
    q, s, b = K.quantise(group([], 1.25))
    assert not q.any() and s.tolist() == [0] and bf16_to_f64(b).tolist() == [1.25]


def test_bias_rounded_above_the_minimum_clamps():
    # 1.00390625 + 2^-9 rounds up to 1.0078125: the span is negative, the group is its bias
    x = group([], 1.0 + 2.0 ** -8 + 2.0 ** -9)
    q, s, b = K.quantise(x)
    assert not q.any() and s.tolist() == [0]
    assert bf16_to_f64(b)[0] == 1.0078125


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, -3.4e38])
def test_quantise_bad_groups_read_back_as_nan(bad):
    x = np.concatenate([group([bad], 1.0), group([2.0], 1.0)])
    if bad == -3.4e38:
        x[1] = 3.4e38  # a span past fp32
    q, s, b = K.quantise(x)
    v = K.values(K.pack(q), s, b)
    assert np.isnan(v[:64]).all() and np.isfinite(v[64:]).all()


def test_quantise_error_is_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 128)).astype(np.float32)
    q, s, b = K.quantise(x)
    step = np.repeat(bf16_to_f64(s), 64, axis=-1)
    # half a step, plus the scale's and the bias's own rounding: 15 s 2^-9 and |b| 2^-9
    slack = 15 * step * 2.0 ** -8 + np.repeat(np.abs(bf16_to_f64(b)), 64, -1) * 2.0 ** -8
    assert (np.abs(K.values(K.pack(q), s, b) - x) <= 0.5 * step + slack).all()


def test_pack_order():
    q = np.arange(16, dtype=np.uint8)
    assert K.pack(q).tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert (K.unpack(K.pack(q)) == q).all()


def test_token_slots():
    table = np.array([[5, 2], [7, 9]])
    seq, pg, sl = K.token_slots([0, 2, 3], [17, 40], table, 16, 4)
    assert seq.tolist() == [0, 0, 1, -1]
    assert pg.tolist() == [5, 2, -1, -1]  # position 39 is past two pages of 16
    assert sl.tolist()[:2] == [15, 0]


def paged(codes_k, codes_v, s=1.0, b=0.0, page=16, pages=2):
    """One head of 64 channels; channel 0 of key and value i is codes_k[i], codes_v[i]."""
    def plane(first):
        q = np.zeros((pages, 1, page, 64), dtype=np.uint8)
        q.reshape(-1, 64)[:len(first), 0] = first
        bits = lambda v: np.full((pages, 1, page, 1), K._bf16(np.float32(v))[0])  # noqa: E731
        return K.pack(q), bits(s), bits(b)
    return K.Paged(plane(codes_k), plane(codes_v), np.array([[0, 1]]))


def test_attention_by_hand():
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = 1.0
    c = paged([0, 0, 0], [3, 6, 9])
    # equal scores: means of what is seen; two new tokens of three
    o, tol = K.attention(q, c, [0, 2], [3], 1.0)
    assert np.allclose(o[:, 0, 0], [4.5, 6]) and not o[:, 0, 1:].any() and (tol >= 0).all()
    assert np.allclose(K.attention(q, c, [0, 2], [3], 1.0, window=1)[0][:, 0, 0], [6, 9])
    assert np.allclose(K.attention(q, c, [0, 2], [3], 1.0, causal=False)[0][:, 0, 0], [6, 6])
    # the first of two tokens lies before the start of a sequence of one
    assert np.allclose(K.attention(q, c, [0, 2], [1], 1.0)[0][:, 0, 0], [0, 3])
    # a score of ln 2 more is twice the weight
    c = paged([0, 0, 1], [3, 6, 9])
    o, _ = K.attention(q, c, [0, 2], [3], math.log(2.0))
    assert np.allclose(o[1, 0, 0], (3 + 6 + 18) / 4)


def test_attention_skips_pages_that_do_not_exist():
    q = np.zeros((1, 1, 64))
    c = paged([0] * 32, [4] * 16 + [8] * 16)
    c.table = np.array([[-1, 1]])
    assert K.attention(q, c, [0, 1], [32], 1.0)[0][0, 0, 0] == 8
    c.table = np.array([[0, 2]])
    assert K.attention(q, c, [0, 1], [32], 1.0)[0][0, 0, 0] == 4
    c.table = np.array([[7, -3]])
    assert not K.attention(q, c, [0, 1], [32], 1.0)[0].any()


def test_unseen_nan_stays_out():
    q = np.ones((2, 1, 64))
    c = paged([1, 2, 3], [3, 6, 9])
    for p in ("k", "v"):
        c.planes[p][1][0, 0, 2] = K.NAN_BITS  # scale of position 2
    o, _ = K.attention(q, c, [0, 2], [3], 1.0)
    assert np.isfinite(o[0]).all() and np.isnan(o[1]).all()


def test_activations():
    z = np.array([-30.0, -1.0, 0.0, 2.0])
    assert K.ACT["relu"](z).tolist() == [0, 0, 0, 2]
    assert np.allclose(K.ACT["silu"](z)[1:], [-1 / (1 + math.e), 0, 2 / (1 + math.exp(-2))])
    assert np.allclose(K.ACT["gelu"](z)[1:], [-0.158655254, 0, 1.954499736])


def test_linear():
    x = np.array([[1.0, 2.0]])
    w = np.array([[3.0, 4.0], [-5.0, 0.5]])
    assert K.linear(x, w, bias=np.array([1.0, 1.0]), act="relu", residual=np.array([[0.5, 0.5]])).tolist() == [[12.5, 0.5]]
