"""The 4-bit key/value cache and its attention on the GPU against the fp64 oracle.

Cache contents (codes, scales, biases) and what is read back are compared bit for bit.
Attention is held to the oracle's element-wise bound of what its roundings may cost."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
from oracle import kv4_oracle as K
from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits
from parity_util import dev_bits, host_bits, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def bf16_values(a):
    return bf16_to_f64(round_to_bf16_bits(a)).astype(np.float32)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make_cache(num_pages, Hkv, page, D, fill=None):
    c = M.KV4Cache.empty(num_pages, Hkv, page, D)
    for m in (c.k, c.v):
        m.codes.fill_(0xA5)
        for t in (m.scales, m.biases):
            t.fill_(float("nan") if fill is None else fill)
    return c


def host_planes(c):
    return [(m.codes.cpu().numpy(), host_bits(m.scales), host_bits(m.biases)) for m in (c.k, c.v)]


class Batch:
    """Ragged sequences on shuffled pages."""

    def __init__(self, rng, new, past, page, spare=2, width=0):
        self.new, self.len = list(new), [n + p for n, p in zip(new, past)]
        self.page, self.B, self.T = page, len(new), sum(new)
        self.cu = [0] + list(np.cumsum(new))
        width = max(width, max(1, max(-(-t // page) for t in self.len)) + 1)
        self.num_pages = self.B * width + spare
        self.table = rng.permutation(self.num_pages)[:self.B * width].reshape(self.B, width)
        self.dev = (i32(self.table), i32(self.cu), i32(self.len))

    def max_new(self):
        return max(max(self.new), 1)


def tokens(rng, T, H, D, dtype):
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x[:, :, :3] *= 6.0
    return bf16_values(x) if dtype == BF16 else x


def filled(rng, b, Hkv, D):
    """A cache holding every token of every sequence (written through the framework), NaN elsewhere."""
    c = make_cache(b.num_pages, Hkv, b.page, D)
    T = sum(b.len)
    kv = [tokens(rng, T, Hkv, D, BF16) for _ in range(2)]
    k, v = (torch.from_numpy(a).cuda().to(BF16) for a in kv)
    M.moe_kv4_append(c, k, v, b.dev[0], i32([0] + list(np.cumsum(b.len))), b.dev[2])
    return c


def queries(rng, T, Hq, D):
    x = bf16_values(rng.standard_normal((T, Hq, D)))
    return x.astype(np.float64), torch.from_numpy(x).cuda().to(BF16)


def check(got, want, tol, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    assert (np.isnan(got) == np.isnan(want)).all(), what
    ok = ~np.isnan(want)
    off = np.abs(got - want)[ok]
    t = tol[ok]
    if off.size:
        say(f"  {what}: worst {float((off / np.maximum(t, 1e-30)).max()):.3f} of the bound, "
            f"rms {np.sqrt((off ** 2).mean()):.2e} of {np.sqrt((want[ok] ** 2).mean()):.2e}")
    assert (off <= t).all(), what


# ------------------------------------------------------------------ write and read

CACHE_CASES = [  # new tokens, earlier tokens, Hkv, D, page
    ([1], [0], 1, 64, 16),
    ([1] * 8, [15, 16, 31, 0, 5, 700, 63, 64], 2, 256, 16),
    ([3, 0, 17, 1], [14, 2, 0, 100], 1, 128, 32),
    ([5, 70], [60, 0], 3, 64, 64),
    ([2] * 70, list(range(70)), 1, 64, 16),          # more sequences than lanes
    ([1, 0, 2] * 50, [3] * 150, 2, 128, 256),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,past,Hkv,D,page", CACHE_CASES)
def test_append_and_read(new, past, Hkv, D, page, dtype):
    rng = np.random.default_rng(len(new) * 1000 + D)
    b = Batch(rng, new, past, page)
    kv = [tokens(rng, b.T, Hkv, D, dtype) for _ in range(2)]
    c = make_cache(b.num_pages, Hkv, page, D)
    # keys and values as slices of one projection's output: strided rows
    both = torch.from_numpy(np.concatenate(kv, axis=1)).cuda().to(dtype)
    before = host_planes(c)
    M.moe_kv4_append(c, both[:, :Hkv], both[:, Hkv:], *b.dev)
    after = host_planes(c)
    _, pg, sl = K.token_slots(b.cu, b.len, b.table, page, b.T)
    for name, x, old, got in zip("kv", kv, before, after):
        q, s, z = K.quantise(x)
        for field, a, o, g in zip(("codes", "scales", "biases"), (K.pack(q), s, z), old, got):
            want = o.copy()
            for t in range(b.T):
                want[pg[t], :, sl[t]] = a[t]
            assert (want == g).all(), f"{name}.{field}"
    for out in (BF16, F32):
        k, v = M.moe_kv4_read(c, *b.dev, b.T, dtype=out)
        for x, got in zip(kv, (k, v)):
            q, s, z = K.quantise(x)
            want = K.values(K.pack(q), s, z).astype(np.float32)
            if out == F32:
                assert (got.cpu().numpy() == want).all()
            else:
                assert (host_bits(got) == round_to_bf16_bits(want)).all()


def test_quantiser_edges():
    """Ties, constant and subnormal groups, outliers, biases above the minimum, NaN and
    infinities, spans past fp32: codes, scales and biases bit for bit."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((200, 1, 64)).astype(np.float32)
    x[0], x[1], x[2] = 0.0, 1.25, -0.0
    x[3] = np.linspace(0, 15, 64)
    x[4] = np.arange(64) / 4.0 - 0.5          # many exact ties
    x[5] = np.arange(64) % 31 / 2.0            # every half
    x[6] *= np.float32(1e-38)
    x[7] *= np.float32(1e-44)
    x[8, 0, 7], x[9, 0, 8], x[10, 0, 9] = np.nan, np.inf, -np.inf
    x[11, 0, :2] = 3.4e38, -3.4e38
    x[12] = 1.0 + 2.0 ** -8 + 2.0 ** -9        # rounds up to a bias above everything
    x[13] = 1000.0 + x[13]
    x[14, 0, 0] = 1e30
    x[15] = -3.39e38
    x[16, 0, 0] = -3.4028e38                   # its bias rounds to -inf
    x[17:60] = np.round(x[17:60] * 4) / 4      # coarse lattices: ties everywhere
    x[60:90] = np.round(x[60:90] * 8) * np.float32(2.0 ** 20)
    x[90:120] *= np.float32(2.0) ** rng.integers(-120, 120, (30, 1, 1)).astype(np.float32)
    for dtype in (F32, BF16):
        y = x.copy()
        if dtype == BF16:
            y = bf16_values(y)
        b = Batch(rng, [200], [0], 16)
        c = make_cache(b.num_pages, 1, 16, 64)
        d = torch.from_numpy(y).cuda().to(dtype)
        M.moe_kv4_append(c, d, -d, *b.dev)
        _, pg, sl = K.token_slots(b.cu, b.len, b.table, 16, 200)
        for sign, got in zip((1, -1), host_planes(c)):
            q, s, z = K.quantise(sign * y)
            for name, a, g in zip(("scales", "biases", "codes"), (s, z, K.pack(q)), (got[1], got[2], got[0])):
                bad = (a != g[pg, :, sl]).reshape(200, -1).any(1)
                assert not bad.any(), (name, dtype, sign, np.nonzero(bad)[0][:10])
        k, _ = M.moe_kv4_read(c, *b.dev, 200, dtype=F32)
        k = k.cpu().numpy()
        assert np.isnan(k[[8, 9, 10, 11]]).all() and np.isfinite(k[[0, 1, 2, 3, 6, 7, 12, 13, 14]]).all()


def test_dequant_w4_sees_the_same_page():
    rng = np.random.default_rng(6)
    b = Batch(rng, [16], [0], 16)
    c = make_cache(b.num_pages, 2, 16, 128, fill=0.0)
    x = torch.from_numpy(tokens(rng, 16, 2, 128, BF16)).cuda().to(BF16)
    M.moe_kv4_append(c, x, x, *b.dev)
    k, _ = M.moe_kv4_read(c, *b.dev, 16)
    m = M.W4Matrix(c.k.codes.view(-1, 16, 64), c.k.scales.view(-1, 16, 2), c.k.biases.view(-1, 16, 2))
    for h in range(2):
        page = M.moe_dequant_w4(m, index=int(b.table[0, 0]) * 2 + h)
        assert torch.equal(page, k[:, h])


def test_tokens_without_a_place():
    """Pages outside the cache, positions past the table and rows past the last sequence:
    nothing is written anywhere else; read gives zeros for the first two and leaves the rest."""
    rng = np.random.default_rng(7)
    b = Batch(rng, [20, 20, 4], [12, 30, 0], 16)
    table = b.table.copy()
    table[0, 1] = b.num_pages       # one past the end
    table[1, 2] = -5
    lens = [b.len[0], b.len[1], table.shape[1] * 16 + 2]
    dev = (i32(table), i32(b.cu), i32(lens))
    T = b.T + 3
    x = torch.from_numpy(tokens(rng, T, 1, 64, F32)).cuda()
    c = make_cache(b.num_pages, 1, 16, 64)
    before = host_planes(c)
    M.moe_kv4_append(c, x, x, *dev)
    _, pg, sl = K.token_slots(b.cu, lens, table, 16, T)
    placed = (pg >= 0) & (pg < b.num_pages)
    assert 0 < placed.sum() < b.T
    q, s, z = K.quantise(x.cpu().numpy())
    for old, got in zip(before, host_planes(c)):
        for o, g, a in zip(old, got, (K.pack(q), s, z)):
            o[pg[placed], :, sl[placed]] = a[placed]
            assert (o == g).all()
    k = torch.full((T, 1, 64), 7.0, device="cuda")
    v = torch.full((T, 1, 64), 7.0, device="cuda")
    M.moe_kv4_read(c, *dev, T, dtype=F32, k=k, v=v)
    want = np.where(placed[:, None, None], K.values(K.pack(q), s, z).astype(np.float32), 0)
    want[b.T:] = 7.0
    assert (k.cpu().numpy() == want).all() and (v.cpu().numpy() == want).all()


# ------------------------------------------------------------------ attention

ATTENTION = [  # new, past, Hq, Hkv, D, page, causal, window
    ([1], [0], 1, 1, 64, 16, True, 0),
    ([1], [15], 8, 1, 128, 16, True, 0),
    ([1], [16], 16, 2, 256, 16, True, 0),
    ([1, 1, 1], [30, 31, 32], 16, 2, 128, 32, True, 0),
    ([1] * 9, [0, 7, 63, 64, 65, 127, 128, 500, 1200], 16, 2, 256, 64, True, 0),
    ([1, 0, 2], [333, 100, 0], 6, 2, 64, 16, True, 0),       # 3 heads a group, an idle sequence
    ([5, 3], [100, 0], 12, 1, 128, 128, True, 0),            # 12 heads a group
    ([1], [5000], 8, 8, 64, 256, True, 0),                   # split over workgroups
    ([1, 1], [9000, 40], 16, 2, 128, 16, True, 0),
    ([2], [3000], 32, 1, 256, 64, True, 0),                  # two row tiles, split
    ([3] * 4, [700, 10, 0, 95], 8, 8, 64, 32, True, 100),    # sliding window
    ([1], [4000], 16, 2, 128, 16, True, 1),                  # sees itself only
    ([40], [50], 4, 2, 128, 16, True, 17),
    ([33], [0], 8, 2, 128, 16, True, 0),                     # prompts
    ([200, 1, 77], [0, 300, 129], 16, 2, 128, 64, True, 0),
    ([130], [65], 8, 1, 64, 16, True, 0),
    ([100, 31], [3, 200], 16, 2, 256, 32, True, 0),
    ([64, 9], [0, 80], 4, 4, 128, 16, False, 0),             # every token sees all
    ([20], [200], 4, 2, 64, 16, False, 50),
    ([150], [700], 20, 4, 256, 128, True, 333),
    ([300], [0], 2, 2, 64, 16, True, 0),                     # one head a group, three tiles of 128 rows
    ([257], [1000], 8, 2, 256, 64, True, 0),
    ([129], [31], 3, 1, 128, 16, True, 40),
    ([70], [333], 4, 2, 128, 32, False, 0),
    ([700, 3, 0, 8, 1], [100, 2000, 50, 900, 5000], 16, 2, 128, 64, True, 0),  # prompts and single tokens
    ([9, 2, 90], [300, 700, 0], 8, 1, 64, 16, True, 150),    # on both sides of 64 rows
]


@pytest.mark.parametrize("new,past,Hq,Hkv,D,page,causal,window", ATTENTION)
def test_attention(new, past, Hq, Hkv, D, page, causal, window):
    rng = np.random.default_rng(Hq * 7 + D + len(new) + sum(past))
    b = Batch(rng, new, past, page)
    c = filled(rng, b, Hkv, D)
    q64, q = queries(rng, b.T, Hq, D)
    out = M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), causal=causal, window=window)
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, D ** -0.5, causal, window)
    check(out, want, tol, f"{new} {past} {Hq}/{Hkv}x{D}")
    again = M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), causal=causal, window=window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("prompt", [0, 270])
def test_hundreds_of_sequences(prompt):
    """More than are spread by their lengths, keys split; and with a prompt among them."""
    rng = np.random.default_rng(36)
    new = [1] * 300
    past = [int(x) for x in np.exp(rng.uniform(0, 7.9, 300))]
    new[17], past[40] = max(prompt, 1), 2900
    b = Batch(rng, new, past, 16, width=8192 // 16 if prompt else 0)
    c = filled(rng, b, 1, 64)
    q64, q = queries(rng, b.T, 16, 64)
    out = M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new())
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, 0.125)
    check(out, want, tol, "300 sequences")


def test_attention_in_place_and_wide_bounds():
    rng = np.random.default_rng(37)
    for new, past, width in (([1, 2], [3000, 40], 0), ([300], [3000], 512)):
        b = Batch(rng, new, past, 16, width=width)
        c = filled(rng, b, 2, 128)
        _, q = queries(rng, b.T, 16, 128)
        want = M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new())
        for kw in (dict(max_new=2 ** 32 + 1), dict(max_new=b.T, window=2 ** 32 + 3)):
            kw.setdefault("window", 0)
            assert torch.allclose(M.moe_kv4_attention(c, q, *b.dev, **kw).float(), want.float(), atol=2e-2)
        M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), out=q)
        assert torch.equal(q, want)
    for bad in (dict(max_new=-1), dict(max_new=1, window=-2 ** 32), dict(max_new=1, scale=2.0 ** 65)):
        with pytest.raises(M.MoeError):
            M.moe_kv4_attention(c, q, *b.dev, **bad)


def test_attention_scales_and_strides():
    """Large scores, another scale, queries inside a wider row, an output of its own strides,
    rows past the last sequence left as they were."""
    rng = np.random.default_rng(21)
    b = Batch(rng, [2, 1], [90, 300], 16)
    c = filled(rng, b, 2, 128)
    T = b.T + 2
    x = bf16_values(rng.standard_normal((T, 12, 128)) * 4)
    wide = torch.from_numpy(x).cuda().to(BF16)
    room = torch.full((T, 10, 128), 3.0, dtype=BF16, device="cuda")
    q, out = wide[:, 2:10], room[:, 1:9]
    for scale in (0.5, 1e-3):
        M.moe_kv4_attention(c, q, *b.dev, max_new=2, scale=scale, out=out)
        want, tol = K.attention(x[:b.T, 2:10].astype(np.float64), K.Paged(*host_planes(c), b.table), b.cu,
                                b.len, float(np.float32(scale)))
        check(out[:b.T], want, tol, f"scale {scale}")
        assert (room[b.T:] == 3).all() and (room[:, 0] == 3).all() and (room[:, 9] == 3).all()


def test_rows_that_see_nothing():
    """Positions before the start, empty sequences and missing pages: zeros, never NaN, though
    the cache holds NaN there; bad pages are skipped."""
    rng = np.random.default_rng(22)
    b = Batch(rng, [4, 3, 2, 2], [0, 60, 40, 0], 16)
    c = filled(rng, b, 2, 64)
    q64, q = queries(rng, b.T, 4, 64)
    table = b.table.copy()
    table[1, 1], table[2, :] = b.num_pages + 3, -1
    lens = [2, b.len[1], b.len[2], 0]
    out = M.moe_kv4_attention(c, q, i32(table), i32(b.cu), i32(lens), max_new=4)
    want, tol = K.attention(q64, K.Paged(*host_planes(c), table), b.cu, lens, 64 ** -0.5)
    check(out, want, tol, "holes")
    assert not out[:2].any() and not out[7:].any() and out[2:4].any()


def test_hostile_batches_stay_in_their_buffers():
    """Offsets and lengths that make no sense are clamped: no fault, and rows no sequence
    claims are left alone."""
    rng = np.random.default_rng(23)
    b = Batch(rng, [3, 3], [20, 40], 16)
    c = filled(rng, b, 2, 64)
    _, q = queries(rng, b.T, 4, 64)
    big = 2 ** 31 - 1
    for cu, lens in (([-5, 3, 900], [23, 43]), ([0, 3, 6], [big, -4]), ([6, 3, 0], [23, 43]),
                     ([big, -big, 2], [5, 5])):
        out = torch.full((b.T, 4, 64), 5.0, dtype=BF16, device="cuda")
        M.moe_kv4_attention(c, q, b.dev[0], i32(cu), i32(lens), max_new=6, out=out)
        M.moe_kv4_read(c, b.dev[0], i32(cu), i32(lens), b.T)
    torch.cuda.synchronize()


@pytest.mark.parametrize("past", [40, 3000])
def test_nan_reaches_only_those_who_see_it(past):
    """A NaN key and a NaN value at one position: queries at or behind it are NaN (the value's
    only in its own group of channels), earlier ones are not."""
    rng = np.random.default_rng(24)
    b = Batch(rng, [5], [past], 16)
    q64, q = queries(rng, 5, 2, 128)
    at = past + 2
    for which in "kv":
        c = filled(rng, b, 1, 128)
        m = getattr(c, which)
        pg, sl = int(b.table[0, at // 16]), at % 16
        m.scales[pg, 0, sl, 1] = float("nan")
        m.biases[pg, 0, sl, 1] = float("nan")
        out = M.moe_kv4_attention(c, q, *b.dev, max_new=5).float().cpu().numpy()
        want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, 128 ** -0.5)
        check(torch.from_numpy(out), want, tol, which)
        assert np.isfinite(out[:2]).all() and np.isnan(out[2:, :, 64:]).all()
        assert np.isnan(out[2:, :, :64]).all() == (which == "k")


def test_outlier_values_keep_their_neighbours():
    """A huge value that weighs next to nothing does not cost the others their digits."""
    rng = np.random.default_rng(25)
    b = Batch(rng, [1], [99], 16)
    c = make_cache(b.num_pages, 1, 16, 64)
    k = bf16_values(rng.standard_normal((100, 1, 64)) * 0.1)
    v = bf16_values(rng.standard_normal((100, 1, 64)))
    k[50], v[50] = -40.0, bf16_values(np.array(1e6) * rng.standard_normal(64))
    x = np.ones((1, 1, 64), dtype=np.float32)
    cu = i32([0, 100])
    M.moe_kv4_append(c, *(torch.from_numpy(a).cuda().to(BF16) for a in (k, v)), b.dev[0], cu, b.dev[2])
    out = M.moe_kv4_attention(c, torch.from_numpy(x).cuda().to(BF16), *b.dev, max_new=1)
    want, tol = K.attention(x.astype(np.float64), K.Paged(*host_planes(c), b.table), b.cu, b.len, 0.125)
    check(out, want, tol, "outlier")


# ------------------------------------------------------------------ prompts
# Enough query rows (4096 in all, more than 64 a sequence and head), and a page
# table of 8192 positions, for the kernel that prompts take.

PROMPTS = [  # new, past, Hq, Hkv, D, page, causal, window
    ([129], [31], 32, 1, 128, 16, True, 0),                  # 32 heads a group
    ([70], [0], 64, 64, 64, 16, True, 0),                    # one
    ([70], [0], 60, 20, 128, 32, True, 0),                   # three: tiles begin inside a token
    ([300], [0], 16, 4, 64, 16, True, 0),
    ([257], [1000], 16, 2, 256, 64, True, 0),
    ([128], [333], 32, 4, 128, 32, False, 0),                # every token sees all
    ([300, 3, 0, 8, 1], [100, 2000, 50, 900, 5000], 16, 2, 128, 64, True, 0),  # with single tokens
    ([9, 2, 250], [300, 700, 0], 24, 3, 64, 16, True, 0),    # on both sides of 64 rows
    ([1100], [500], 32, 1, 64, 16, True, 1000),              # sliding windows
    ([520], [200], 128, 2, 64, 32, False, 550),
    ([260], [3000], 16, 2, 128, 64, True, 0),                # keys split over workgroups
    ([256], [2500], 16, 1, 256, 32, True, 0),
    ([520], [1500], 8, 8, 64, 16, True, 0),
    ([140, 126, 1], [4000, 900, 4095], 16, 2, 64, 64, True, 0),
    ([130], [2200], 32, 1, 128, 128, False, 0),
]


def prompt_batch(rng, new, past, page):
    return Batch(rng, new, past, page, width=8192 // page)


@pytest.mark.parametrize("new,past,Hq,Hkv,D,page,causal,window", PROMPTS)
def test_prompts(new, past, Hq, Hkv, D, page, causal, window):
    rng = np.random.default_rng(Hq * 5 + D + len(new) + sum(past))
    b = prompt_batch(rng, new, past, page)
    assert b.T * Hq >= 4096 and max(new) * (Hq // Hkv) > 64
    c = filled(rng, b, Hkv, D)
    q64, q = queries(rng, b.T, Hq, D)
    out = M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), causal=causal, window=window)
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, D ** -0.5, causal, window)
    check(out, want, tol, f"{new} {past} {Hq}/{Hkv}x{D}")
    again = M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), causal=causal, window=window)
    assert torch.equal(out, again)


def test_prompt_scales_and_strides():
    rng = np.random.default_rng(31)
    b = prompt_batch(rng, [140], [90], 16)
    c = filled(rng, b, 2, 128)
    T = b.T + 2
    x = bf16_values(rng.standard_normal((T, 40, 128)) * 4)
    wide = torch.from_numpy(x).cuda().to(BF16)
    room = torch.full((T, 34, 128), 3.0, dtype=BF16, device="cuda")
    q, out = wide[:, 2:34], room[:, 1:33]
    for scale in (0.5, 1e-3):
        M.moe_kv4_attention(c, q, *b.dev, max_new=140, scale=scale, out=out)
        want, tol = K.attention(x[:b.T, 2:34].astype(np.float64), K.Paged(*host_planes(c), b.table), b.cu,
                                b.len, float(np.float32(scale)))
        check(out[:b.T], want, tol, f"scale {scale}")
        assert (room[b.T:] == 3).all() and (room[:, 0] == 3).all() and (room[:, 33] == 3).all()


@pytest.mark.parametrize("past", [60, 3000])
def test_prompt_rows_that_see_nothing(past):
    """Positions before the start, a sequence of length zero and bad pages, among keys that are
    split and not: zeros, and bad pages are skipped."""
    rng = np.random.default_rng(32)
    b = prompt_batch(rng, [140, 130, 70], [0, past, 0], 16)
    c = filled(rng, b, 2, 64)
    q64, q = queries(rng, b.T, 16, 64)
    table = b.table.copy()
    table[1, 1], table[1, 5], table[1, -1] = b.num_pages + 3, -1, 2 ** 31 - 1
    lens = [20, b.len[1], 0]
    out = M.moe_kv4_attention(c, q, i32(table), i32(b.cu), i32(lens), max_new=140)
    want, tol = K.attention(q64, K.Paged(*host_planes(c), table), b.cu, lens, 64 ** -0.5)
    check(out, want, tol, "holes")
    assert not out[:120].any() and not out[270:].any() and out[120:270].any()


def test_hostile_prompts_stay_in_their_buffers():
    rng = np.random.default_rng(33)
    b = prompt_batch(rng, [150, 150], [20, 2000], 16)
    c = filled(rng, b, 2, 64)
    _, q = queries(rng, b.T, 16, 64)
    big = 2 ** 31 - 1
    for cu, lens in (([-5, 100, 900], [23, 4300]), ([0, 300, 300], [big, -4]), ([300, 150, 0], [23, 43]),
                     ([big, -big, 200], [5, 5]), ([0, 200, 300], [8193, 100000])):
        out = torch.full((b.T, 16, 64), 5.0, dtype=BF16, device="cuda")
        M.moe_kv4_attention(c, q, b.dev[0], i32(cu), i32(lens), max_new=b.T, out=out)
    torch.cuda.synchronize()


def test_prompt_max_new_bounds_what_is_computed():
    rng = np.random.default_rng(34)
    b = prompt_batch(rng, [300], [10], 16)
    c = filled(rng, b, 1, 64)
    _, q = queries(rng, 300, 16, 64)
    whole = M.moe_kv4_attention(c, q, *b.dev, max_new=300)
    assert torch.equal(whole, M.moe_kv4_attention(c, q, *b.dev, max_new=100000))
    out = torch.full_like(whole, 9.0)
    M.moe_kv4_attention(c, q, *b.dev, max_new=270, out=out)
    assert torch.equal(out[:270], whole[:270]) and (out[270:] == 9).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["large", "small", "query", "faint query", "mixed", "split"])
def test_prompts_outside_fp16(D, kind):
    """Prompts whose keys, values or queries leave fp16's range (the kernel turns to bf16
    operands, whose rounding, 2^-8 of every key and value, is added to the bound)."""
    rng = np.random.default_rng(D)
    b = prompt_batch(rng, [40, 33], [3000 if kind == "split" else 70, 0], 16)
    T = sum(b.len)
    f = 1e6 if kind == "large" else 1e-6 if kind == "small" else 1.0
    k = bf16_values(tokens(rng, T, 2, D, BF16) * min(f, 1.0))
    v = bf16_values(tokens(rng, T, 2, D, BF16) * f)
    if kind in ("mixed", "split"):
        v[95] *= 1e6  # far into the first sequence: the run starts over there
    x = bf16_values(rng.standard_normal((b.T, 64, D)))
    scale = D ** -0.5
    if kind == "query":
        x, scale = bf16_values(x * 1e5), scale * 1e-5
    if kind == "faint query":
        x[:, :9], scale = bf16_values(x[:, :9] * 1e-7), scale * 1e5
        x[:, 9:] = bf16_values(x[:, 9:] * 1e-5)
    c = make_cache(b.num_pages, 2, 16, D)
    M.moe_kv4_append(c, *(torch.from_numpy(a).cuda().to(BF16) for a in (k, v)), b.dev[0],
                     i32([0] + list(np.cumsum(b.len))), b.dev[2])
    out = M.moe_kv4_attention(c, torch.from_numpy(x).cuda().to(BF16), *b.dev, max_new=40, scale=scale)
    scale = float(np.float32(scale))
    planes = K.Paged(*host_planes(c), b.table)
    want, tol = K.attention(x.astype(np.float64), planes, b.cu, b.len, scale)
    # scores off by 2^-8 scale sum |q k|, values by 2^-8 of themselves
    extra = np.zeros_like(tol)
    for s in range(b.B):
        for h in range(2):
            kc, ks, kb, _ = planes.rows("k", s, h, b.len[s])
            vc, vs, vb, _ = planes.rows("v", s, h, b.len[s])
            vmax = np.abs(vs * vc + vb).max(0)
            for g in range(32 * h, 32 * h + 32):
                rows = slice(b.cu[s], b.cu[s + 1])
                d = 2.0 ** -8 * scale * (np.abs(x[rows, g]).astype(np.float64) @ np.abs(ks * kc + kb).T).max(1)
                extra[rows, g] = (2 * d[:, None] + 2.0 ** -8) * vmax
    check(out, want, tol + extra, f"{kind} {D}")


@pytest.mark.parametrize("Hq", [4, 64])
def test_long_faint_tail_is_not_lost(Hq):
    """Keys that weigh 2^-27 of the largest each, whose value is all there is to see."""
    rng = np.random.default_rng(35)
    b = prompt_batch(rng, [72], [7900], 16)
    k = np.zeros((7972, 1, 64), dtype=np.float32)
    v = np.ones((7972, 1, 64), dtype=np.float32)
    k[0], v[0] = 2.34375, 0.0   # 8 x 2.34 = 18.75 = 27.05 ln 2
    c = make_cache(b.num_pages, 1, 16, 64)
    M.moe_kv4_append(c, *(torch.from_numpy(a).cuda() for a in (k, v)), b.dev[0], i32([0, 7972]), b.dev[2])
    x = np.ones((72, Hq, 64))
    out = M.moe_kv4_attention(c, torch.from_numpy(x).cuda().to(BF16), *b.dev, max_new=72)
    want, tol = K.attention(x, K.Paged(*host_planes(c), b.table), b.cu, b.len, 0.125)
    # Prompts: weights are rounded to fp16 times 2^7. The reference they are relative to is a
    # score of the row, so their sum is at least 1; below 2^-14 fp16 steps by 2^-24, so each is
    # off by up to 2^-25 / 2^7 = 2^-32 beside what larger ones are. 7972 of them, of value 1:
    check(out, want, tol + 7972 * 2.0 ** -32, "tail")  # 1.9e-6 of the 5.7e-5 that the tail adds up to


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("past", [50, 3000])
def test_prompt_nan_reaches_only_those_who_see_it(D, past):
    rng = np.random.default_rng(29)
    b = prompt_batch(rng, [80], [past], 16)
    q64, q = queries(rng, 80, 64, D)
    at = past + 37
    for which in "kv":
        c = filled(rng, b, 1, D)
        m = getattr(c, which)
        pg, sl = int(b.table[0, at // 16]), at % 16
        m.scales[pg, 0, sl, -1] = float("nan")
        m.biases[pg, 0, sl, -1] = float("nan")
        out = M.moe_kv4_attention(c, q, *b.dev, max_new=80).float().cpu().numpy()
        want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, D ** -0.5)
        assert (np.isnan(out) == np.isnan(want)).all()
        assert np.isfinite(out[:37]).all() and np.isnan(out[37:, :, -64:]).all()
        ok = ~np.isnan(want)
        assert np.abs(out[ok] - want[ok]).max() < 0.05 * np.abs(want[ok]).max()


def test_offsets_past_32_bits():
    """Pages whose codes lie beyond 2^31 bytes of the cache."""
    rng = np.random.default_rng(26)
    Hkv, page, D = 2, 256, 256
    num_pages = (5 << 30) // (Hkv * page * D // 2)   # 5 GiB of codes a plane
    c = M.KV4Cache.empty(num_pages, Hkv, page, D)
    table = np.array([[num_pages - 1, num_pages // 2 + 1, 3]])
    n = 600
    kv = [tokens(rng, n, Hkv, D, BF16) for _ in range(2)]
    k, v = (torch.from_numpy(a).cuda().to(BF16) for a in kv)
    M.moe_kv4_append(c, k, v, i32(table), i32([0, n]), i32([n]))
    rk, rv = M.moe_kv4_read(c, i32(table), i32([0, n]), i32([n]), n)
    planes = []
    for x, got in zip(kv, (rk, rv)):
        qc, s, z = K.quantise(x)
        assert (host_bits(got) == round_to_bf16_bits(K.values(K.pack(qc), s, z).astype(np.float32))).all()
        full = []
        for a in (K.pack(qc), s, z):  # the same three pages in a small cache
            p = np.zeros((3, page, Hkv, a.shape[-1]), dtype=a.dtype)
            p.reshape(3 * page, Hkv, -1)[:n] = a
            full.append(p.transpose(0, 2, 1, 3))
        planes.append(tuple(full))
    q64, q = queries(rng, 2, 4, D)
    out = M.moe_kv4_attention(c, q, i32(table), i32([0, 2]), i32([n]), max_new=2)
    want, tol = K.attention(q64, K.Paged(*planes, np.array([[0, 1, 2]])), [0, 2], [n], D ** -0.5)
    check(out, want, tol, "far pages")
    q64, q = queries(rng, n, 80, D)   # rows enough for the prompts' kernel
    out = M.moe_kv4_attention(c, q, i32(table), i32([0, n]), i32([n]), max_new=n)
    want, tol = K.attention(q64, K.Paged(*planes, np.array([[0, 1, 2]])), [0, n], [n], D ** -0.5)
    check(out, want, tol, "far pages, prompt")


def test_max_new_bounds_what_is_computed():
    rng = np.random.default_rng(27)
    b = Batch(rng, [6], [10], 16)
    c = filled(rng, b, 1, 64)
    q64, q = queries(rng, 6, 2, 64)
    whole = M.moe_kv4_attention(c, q, *b.dev, max_new=6)
    assert torch.equal(whole, M.moe_kv4_attention(c, q, *b.dev, max_new=1000))
    out = torch.full_like(whole, 9.0)
    M.moe_kv4_attention(c, q, *b.dev, max_new=4, out=out)
    assert torch.equal(out[:4], whole[:4]) and (out[4:] == 9).all()


def test_empty_calls():
    c = make_cache(2, 1, 16, 64)
    e = torch.empty((0, 1, 64), dtype=BF16, device="cuda")
    dev = (i32([[0]]), i32([0, 0]), i32([5]))
    M.moe_kv4_append(c, e, e, *dev)
    assert M.moe_kv4_read(c, *dev, 0)[0].shape == (0, 1, 64)
    assert M.moe_kv4_attention(c, e, *dev, max_new=0).shape == (0, 1, 64)


def test_binding_refusals():
    c = make_cache(4, 2, 16, 64)
    q = torch.zeros((2, 4, 64), dtype=BF16, device="cuda")
    kv = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    dev = (i32([[0, 1]]), i32([0, 2]), i32([5]))
    out = torch.empty_like(q)
    bad_attention = [dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()),
                     dict(out=out[:1]), dict(out=out.float()), dict(scale=0.0), dict(window=-1),
                     dict(max_new=0), dict(table=dev[0].long()), dict(cu=i32([0, 1, 2])), dict(ln=i32([5, 5])),
                     dict(table=dev[0][0])]
    for bad in bad_attention:
        a = dict(q=q, table=dev[0], cu=dev[1], ln=dev[2], max_new=2)
        a.update(bad)
        with pytest.raises(M.MoeError):
            M.moe_kv4_attention(c, a.pop("q"), a.pop("table"), a.pop("cu"), a.pop("ln"), **a)
    for k, v in ((kv[:, :1], kv), (kv, kv.float()), (kv.half(), kv.half()), (kv.transpose(0, 1), kv), (kv, kv.cpu())):
        with pytest.raises(M.MoeError):
            M.moe_kv4_append(c, k, v, *dev)
    with pytest.raises(M.MoeError):
        M.moe_kv4_read(c, *dev, 2, dtype=torch.float16)
    with pytest.raises(M.MoeError):
        M.moe_kv4_read(c, *dev, 2, k=torch.zeros((2, 2, 64), device="cuda"))
    long = M.KV4Cache(c.k, c.v)
    table = i32([[0] * 4096])
    with pytest.raises(M.MoeError):
        M.moe_kv4_attention(long, q, table, dev[1], dev[2], max_new=2,
                            ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ prompts whose rows fill the card
# No keys are split (no workspace), so a causal call's tiles go in the order that pairs
# long ones with short ones: 257 to 512 tiles over several heads, of which some begin
# before and end behind workgroup 256.

UNSPLIT = [  # new, past, Hq, Hkv, D, page, causal
    ([3000], [0], 16, 2, 128, 64, True),
    ([3000], [40], 16, 2, 64, 16, True),
    ([1500], [0], 32, 8, 128, 16, True),
    ([1500], [7], 32, 4, 64, 32, True),
    ([640, 640, 640], [0, 100, 33], 32, 8, 64, 16, True),
    ([640, 411, 500], [0, 100, 33], 32, 8, 128, 64, True),
    ([869, 800, 869, 869, 640, 750, 801, 777, 869], [0, 90, 3, 0, 200, 1, 20, 0, 4], 6, 2, 128, 16, True),
    ([2049], [0], 24, 8, 64, 128, True),
    ([2100], [300], 64, 2, 64, 16, True),                    # more tiles than are paired
    ([1500], [0], 32, 8, 64, 16, False),
    ([1500], [0], 32, 8, 256, 64, True),
]


@pytest.mark.parametrize("new,past,Hq,Hkv,D,page,causal", UNSPLIT)
def test_prompts_that_fill_the_card(new, past, Hq, Hkv, D, page, causal):
    rng = np.random.default_rng(Hq * 3 + D + len(new) + sum(past))
    b = Batch(rng, new, past, page)
    width = b.table.shape[1]
    c = filled(rng, b, Hkv, D)
    # rows and pairs enough for the prompts' kernel, and its keys in one piece
    assert b.T * Hq >= 4096 and b.T * Hq * width * page >= 2 ** 25 and max(new) * (Hq // Hkv) > 64
    assert M.moe_kv4_attention_workspace_bytes(c, b.T, Hq, b.B, width, b.max_new()) == 0
    q64, q = queries(rng, b.T, Hq, D)
    out = torch.full((b.T, Hq, D), float("nan"), dtype=BF16, device="cuda")
    M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), causal=causal, out=out)
    assert not torch.isnan(out).any()
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, D ** -0.5, causal)
    check(out, want, tol, f"{new} {past} {Hq}/{Hkv}x{D}")
    M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), causal=causal, out=q)
    assert torch.equal(out, q)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("past", [50, 3000])
def test_prompt_values_past_the_range_stay_with_those_who_see_them(D, past):
    """A finite scale whose rebuilt values (or keys) overflow, at a position that the first 37
    tokens do not see, some of them in a block of rows with tokens that do: their results are
    those beside a NaN there, bit for bit. Who sees it gets no finite number in its group."""
    rng = np.random.default_rng(41)
    b = prompt_batch(rng, [80], [past], 16)
    q64, q = queries(rng, 80, 64, D)
    at = past + 37
    for which in "kv":
        c = filled(rng, b, 1, D)
        m = getattr(c, which)
        pg, sl = int(b.table[0, at // 16]), at % 16
        outs = []
        for s, z in ((float("nan"), float("nan")), (2.5e37, 0.0), (-2.5e37, -1e38), (3e38, 3e38)):
            m.codes[pg, 0, sl] = 0xFF      # 15 s + z is past 3.4e38
            m.scales[pg, 0, sl, -1] = s
            m.biases[pg, 0, sl, -1] = z
            outs.append(M.moe_kv4_attention(c, q, *b.dev, max_new=80).float().cpu().numpy())
        for i, out in enumerate(outs):
            same = bool(np.isfinite(out[:37]).all() and (out[:37] == outs[0][:37]).all())
            assert same, (which, i)
            if which == "v":
                kept = bool(np.isfinite(out[37:, :, -64:]).any())
                others = bool(np.isfinite(out[37:, :, :-64]).all())
                assert others and not kept, i


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,past,Hq", [(2, 30, 4), (1, 5000, 4), (80, 50, 64), (80, 3000, 64)])
def test_scores_of_any_size(D, new, past, Hq):
    """Scores far past fp32's integers, and past fp32 once they are scaled (scales up to 2^64):
    keys a_t u with u = +-1 a group, exact in the cache and in every product, where a token's own
    key scores highest of all it sees; by 64 and more, its result is its own value."""
    rng = np.random.default_rng(43)
    b = prompt_batch(rng, [new], [past], 16)
    n = new + past
    u = rng.choice([-1.0, 1.0], D // 64).repeat(64)
    back = np.arange(n - 1, -1, -1)              # tokens behind this one
    far = np.exp2(rng.integers(3, 12, n)) * (1 + rng.integers(0, 128, n) / 128)
    up = np.where(back < 128, 2.0 ** 13 * (1 - back / 256), far)
    down = -np.where(back < 128, 1 + back / 128, far)
    v = bf16_values(rng.standard_normal((n, 1, D)))
    q, s, z = K.quantise(v)
    val = K.values(K.pack(q), s, z)[:, 0]
    s, z = (np.abs(np.repeat(bf16_to_f64(a)[:, 0], 64, -1)) for a in (s, z))
    # 2^-8 each: the result, the values or weights as bf16 (few rows: weight times scale, on
    # codes - 8), and weights beside a sum of unrounded ones; then the fp32 sums of n keys
    tol = (2.0 ** -8 * (3 * np.abs(val) + 8 * s) + (n + 64) * 2.0 ** -24 * (55 * s + z))[past:, None]
    for a in (up, down):
        k = (a[:, None] * u).astype(np.float32)
        assert (k == bf16_values(k)).all()
        c = make_cache(b.num_pages, 1, 16, D)
        M.moe_kv4_append(c, torch.from_numpy(k).cuda()[:, None], torch.from_numpy(v).cuda(),
                         b.dev[0], i32([0, n]), b.dev[2])
        for size in (0, 100):
            x = torch.from_numpy(np.broadcast_to(u * 2.0 ** size, (new, Hq, D)).copy()).cuda().to(BF16)
            for scale in (D ** -0.5, 2.0 ** 20, 2.0 ** 64):
                out = M.moe_kv4_attention(c, x, *b.dev, max_new=new, scale=scale).double().cpu().numpy()
                finite = bool(np.isfinite(out).all())
                assert finite, (size, scale)
                gap = 2.0 ** size * scale * D * (32 if a is up else 2.0 ** -7)
                worst = float((np.abs(out - val[past:, None]) / tol).max())
                assert gap < 64 or worst <= 1, (size, scale, worst)


def test_more_rows_than_a_launch_dimension_holds():
    """2^26 rows and a few: those of a sequence without a place, then 100 that have one."""
    rng = np.random.default_rng(45)
    T, n = 2 ** 26 + 300, 100
    b = Batch(rng, [n], [0], 16)
    table = np.concatenate([b.table, b.table])
    dev = (i32(table), i32([0, T - n, T]), i32([0, n]))
    x = tokens(rng, n, 1, 64, BF16)
    c = make_cache(b.num_pages, 1, 16, 64)
    k, v = (torch.empty((T, 1, 64), dtype=BF16, device="cuda") for _ in range(2))
    k[T - n:] = torch.from_numpy(x)
    M.moe_kv4_append(c, k, k, *dev)
    q, s, z = K.quantise(x)
    at = np.arange(n)
    for plane in host_planes(c):
        for got, want in zip(plane, (K.pack(q), s, z)):
            assert bool((got[b.table[0, at // 16], :, at % 16] == want).all())
    k.fill_(1.0), v.fill_(1.0)
    M.moe_kv4_read(c, *dev, T, k=k, v=v)
    want = round_to_bf16_bits(K.values(K.pack(q), s, z).astype(np.float32))
    for t in (k, v):
        assert bool((host_bits(t[T - n:]) == want).all())
        assert not bool(t[:T - n].view(torch.int16).any())


def test_empty_attention_with_a_wide_bound():
    c = make_cache(2, 1, 16, 64)
    e = torch.empty((0, 1, 64), dtype=BF16, device="cuda")
    for bound in (0, 5, 2 ** 31, 2 ** 32 + 7):
        assert M.moe_kv4_attention(c, e, i32([[0]]), i32([0, 0]), i32([5]), max_new=bound).shape == (0, 1, 64)


@pytest.mark.parametrize("new,past,Hq,Hkv,D", [([300, 1, 2], [0, 8000, 5000], 16, 2, 128), ([1, 300, 1], [7000, 20, 0], 16, 1, 64),
                                                ([2, 3, 260, 1], [8100, 900, 5, 4000], 24, 2, 256)])
def test_single_tokens_beside_a_prompt_in_their_own_workspace(new, past, Hq, Hkv, D):
    """Split keys of the few rows, parts kept by sequence: within the bytes asked for."""
    rng = np.random.default_rng(47)
    b = prompt_batch(rng, new, past, 32)
    c = filled(rng, b, Hkv, D)
    q64, q = queries(rng, b.T, Hq, D)
    need = M.moe_kv4_attention_workspace_bytes(c, b.T, Hq, b.B, b.table.shape[1], b.max_new())
    assert 0 < need
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((b.T, Hq, D), float("nan"), dtype=BF16, device="cuda")
    M.moe_kv4_attention(c, q, *b.dev, max_new=b.max_new(), out=out, ws=ws[:need])
    assert bool((ws[need:] == 0xA5).all())
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, D ** -0.5)
    check(out, want, tol, f"{new} {past}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_split_keys_in_a_padded_batch(D):
    """More rows than the sequences have tokens for: parts are kept by sequence."""
    rng = np.random.default_rng(49)
    b = Batch(rng, [1, 2, 0, 1], [5000, 900, 40, 2500], 32)
    c = filled(rng, b, 2, D)
    T = b.T + 200
    x = bf16_values(rng.standard_normal((T, 8, D)))
    q = torch.from_numpy(x).cuda().to(BF16)
    need = M.moe_kv4_attention_workspace_bytes(c, T, 8, b.B, b.table.shape[1], 2)
    assert 0 < need
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((T, 8, D), 5.0, dtype=BF16, device="cuda")
    M.moe_kv4_attention(c, q, *b.dev, max_new=2, out=out, ws=ws[:need])
    assert bool((ws[need:] == 0xA5).all()) and bool((out[b.T:] == 5).all())
    want, tol = K.attention(x[:b.T].astype(np.float64), K.Paged(*host_planes(c), b.table), b.cu, b.len, D ** -0.5)
    check(out[:b.T], want, tol, f"padded {D}")


@pytest.mark.parametrize("scale", [2.0, 90.0, 700.0, 1500.0])
@pytest.mark.parametrize("new,past,Hq,width", [(2, 5000, 4, 8192), (80, 2000, 64, 8192), (1500, 600, 16, 2112)])
def test_close_scores_far_from_zero(new, past, Hq, width, scale):
    """Scores of 2^13 and small multiples of 2^-9 more, exact in the cache and in every product: a
    softmax over small differences of scaled scores of up to 2^24, whose reference moves within
    a workgroup and differs between splits."""
    rng = np.random.default_rng(51)
    n, D = new + past, 128
    b = Batch(rng, [new], [past], 16, width=width // 16)
    t = np.arange(n)
    j = np.where(t % 512 < 256, (t // 512) % 3, 0.0)
    j = np.where(np.isin(t % 512, (300, 400)), 9.0 + (t // 512) % 3, j) * (355 / max(scale, 16.0))
    j = np.clip(np.round(j), 0, 255)
    k = np.zeros((n, 1, D), dtype=np.float32)
    k[:, :, :64], k[:, :, 64:] = 2.0 ** 13, (j * 2.0 ** -9)[:, None, None]
    assert (k == bf16_values(k)).all()
    v = bf16_values(rng.standard_normal((n, 1, D)))
    q, s, z = K.quantise(v)
    code, val = q[:, 0].astype(np.float64), K.values(K.pack(q), s, z)[:, 0]
    s = np.repeat(bf16_to_f64(s)[:, 0], 64, -1)
    c = make_cache(b.num_pages, 1, 16, D)
    M.moe_kv4_append(c, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), b.dev[0], i32([0, n]), b.dev[2])
    x = torch.zeros((new, Hq, D), dtype=BF16, device="cuda")
    x[:, :, 3], x[:, :, 70] = 1.0, 1.0
    out = torch.full((new, Hq, D), float("nan"), dtype=BF16, device="cuda")
    M.moe_kv4_attention(c, x, *b.dev, max_new=new, scale=scale, out=out)
    out = out.double().cpu().numpy()
    w = np.exp(scale * (j - j.max()) * 2.0 ** -9)
    total = np.cumsum(w)[past:, None]
    mean = lambda a: np.cumsum(w[:, None] * a, axis=0)[past:] / total  # noqa: E731  over what a token sees
    # the result's rounding and weight times scale as bf16 (few rows), or weights and values as
    # fp16, or both as bf16 (scaled scores past 2^23); arguments of up to 60 off by 2^-22 of
    # themselves, and fp32 sums of n keys
    bf16 = 2.0 ** 13 * scale * 1.45 > 2.0 ** 23 and new > 2
    tol = (2.0 ** -8 * (np.abs(mean(val)) + mean(np.abs(s * (code - 8)))) + (2.0 ** -7 if bf16 else 2.0 ** -10) * mean(np.abs(val))
           + (2 * 60 * 2.0 ** -22 + (n + 64) * 2.0 ** -24) * mean(55 * s + np.abs(val)))
    worst = float((np.abs(out - mean(val)[:, None]) / tol[:, None]).max())
    say(f"  scale {scale}: worst {worst:.3f} of the bound")
    assert worst <= 1
