"""Page bounds and attention over selected pages on the GPU against the fp64 oracle.

Bounds and the pages taken are compared exactly; outputs with the oracle's bound of what the
attention's roundings may cost, over the keys of the oracle's own selection."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
from oracle import block_oracle as B
from oracle import kv4_oracle as K
from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits
from parity_util import dev_bits, host_bits, say
from test_gpu_kv4 import BF16, Batch, bf16_values, check, filled, host_planes, i32, make_cache, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def whole(c):
    """Values of the keys as bf16, fp64 [pages, Hkv, page, D]."""
    codes, s, z = host_planes(c)[0]
    with np.errstate(all="ignore"):
        v = K.values(codes, s, z).astype(np.float32)
        return bf16_to_f64(round_to_bf16_bits(v.astype(np.float64)))


def empty_bounds(c, fill=9.0):
    return torch.full((c.num_pages, c.Hkv, 2, c.D), fill, dtype=BF16, device="cuda")


def all_bounds(c, b):
    """Bounds of every page of every sequence, through the framework."""
    out = empty_bounds(c, float("nan"))
    T = sum(b.len)
    M.moe_kv4_bounds(c, out, b.dev[0], i32([0] + list(np.cumsum(b.len))), b.dev[2], T)
    return out


# ------------------------------------------------------------------ bounds

BOUNDS = [  # new tokens, earlier tokens, Hkv, D, page
    ([1], [0], 1, 64, 16), ([1] * 8, [15, 16, 31, 0, 5, 700, 63, 64], 2, 256, 16), ([3, 0, 17, 1], [14, 2, 0, 100], 1, 128, 32),
    ([5, 70], [60, 0], 3, 64, 64), ([2] * 70, list(range(70)), 1, 64, 16), ([1, 0, 2] * 50, [3] * 150, 2, 128, 256),
    ([9000, 40, 1], [3, 1000, 500], 2, 128, 64), ([20000], [0], 1, 256, 16), ([1], [2047], 1, 128, 2048),
]


@pytest.mark.parametrize("new,past,Hkv,D,page", BOUNDS)
def test_bounds(new, past, Hkv, D, page):
    rng = np.random.default_rng(len(new) + D)
    b = Batch(rng, new, past, page)
    c = filled(rng, b, Hkv, D)
    got = empty_bounds(c)
    M.moe_kv4_bounds(c, got, *b.dev, b.T)
    want = np.full((c.num_pages, Hkv, 2, D), 9.0)
    keys = whole(c)
    for s in range(b.B):
        if b.new[s]:
            at = np.arange((b.len[s] - b.new[s]) // page, (b.len[s] - 1) // page + 1)
            for h in range(Hkv):
                want[b.table[s, at], h] = B.bounds(keys[b.table[s, at], h], b.len[s] - at[0] * page)
    assert (host_bits(got) == round_to_bf16_bits(want)).all()


def test_bounds_special_keys():
    """NaN keys give NaN bounds in their channels only, infinities stay, zeros of both signs are +0,
    negative scales; slots past the sequence are not looked at."""
    rng = np.random.default_rng(3)
    b = Batch(rng, [40], [0], 32)
    c = filled(rng, b, 2, 128)
    pg = b.table[0]
    c.k.scales[pg[0], 0, 5, 1] = float("nan")
    c.k.biases[pg[0], 1, 31, 0] = float("nan")
    c.k.scales[pg[0], 1, 3, 1] = -0.5
    c.k.biases[pg[1], 0, 2, 0] = float("inf")
    c.k.scales[pg[1], 0, 3, 1] = float("inf")     # inf * 0 + b is NaN where the code is 0
    c.k.codes[pg[1], 1, :, :] = 0
    c.k.biases[pg[1], 1] = -0.0
    got = empty_bounds(c)
    M.moe_kv4_bounds(c, got, *b.dev, b.T)
    keys = whole(c)
    bits = host_bits(got)
    for i in range(2):
        for h in range(2):
            with np.errstate(all="ignore"):
                want = B.bounds(keys[pg[i:i + 1], h], 32 if i == 0 else 8)[0]
            have = bf16_to_f64(bits[pg[i], h])
            assert np.array_equal(have, want, equal_nan=True) and (have[~np.isnan(have)] == want[~np.isnan(want)]).all()
            assert not (bits[pg[i], h] == 0x8000).any()
    assert np.isnan(bf16_to_f64(bits[pg[0], 0, :, 64:])).all() and not np.isnan(bf16_to_f64(bits[pg[0], 0, :, :64])).any()


def test_bounds_without_a_place():
    rng = np.random.default_rng(5)
    b = Batch(rng, [20, 20, 4, 30], [12, 30, 0, 0], 16)
    c = filled(rng, b, 1, 64)
    table = b.table.copy()
    table[0, 1], table[1, 2] = b.num_pages, -5
    lens = [b.len[0], b.len[1], table.shape[1] * 16 + 2, 25]
    got = empty_bounds(c)
    M.moe_kv4_bounds(c, got, i32(table), i32(b.cu), i32(lens), b.T + 5)
    want = np.full((c.num_pages, 1, 2, 64), 9.0)
    keys = whole(c)
    for s in range(4):
        for at in range(max(lens[s] - b.new[s], 0) // 16, min((lens[s] - 1) // 16 + 1, table.shape[1])):
            if 0 <= table[s, at] < b.num_pages:
                want[table[s, at], 0] = B.bounds(keys[table[s, at]], lens[s] - at * 16)[0]
    assert (host_bits(got) == round_to_bf16_bits(want)).all()


# ------------------------------------------------------------------ attention

def expected(q64, c, bounds, table, cu, lens, T, top, first, recent, scale=None, max_new=10 ** 9):
    """(out, tolerance, blocks) and which rows are computed."""
    n, Hkv, page, D = c.sizes()
    table = np.asarray(table)
    size, Hq = top + first + recent, q64.shape[1]
    G = Hq // Hkv
    bb = bf16_to_f64(host_bits(bounds))
    blocks = np.full((T, Hkv, size), -1)
    taken = np.zeros((T, Hkv, table.shape[1]), dtype=bool)
    done = np.zeros(T, dtype=bool)
    for s in range(len(lens)):
        ok = (table[s] >= 0) & (table[s] < n)
        pages = np.where(ok, table[s], 0)
        for i in range(min(cu[s + 1] - cu[s], max_new)):
            t = cu[s] + i
            done[t] = True
            for h in range(Hkv):
                p = B.select(q64[t, h * G:(h + 1) * G], bb[pages, h, 0], bb[pages, h, 1], ok,
                             lens[s] - (cu[s + 1] - cu[s]) + i, page, top, first, recent)
                blocks[t, h, :len(p)] = p
                taken[t, h, p] = True
    want, tol = K.attention(q64, K.Paged(*host_planes(c), table), cu, lens, D ** -0.5 if scale is None else scale, taken=taken)
    return want, tol, blocks, done


CASES = [  # new, earlier, Hq, Hkv, D, page, top, first, recent
    ([1], [0], 1, 1, 64, 16, 1, 1, 1),
    ([1], [500], 16, 2, 256, 16, 4, 1, 1),
    ([1], [40000], 16, 2, 128, 64, 13, 1, 2),
    ([1] * 9, [3, 15, 16, 17, 100, 900, 2000, 63, 64], 8, 2, 128, 16, 5, 2, 2),
    ([3, 0, 1, 5], [300, 20, 0, 1000], 12, 4, 64, 32, 3, 0, 3),
    ([70, 33], [200, 900], 8, 2, 64, 16, 6, 1, 2),
    ([17], [3000], 3, 1, 256, 64, 8, 0, 1),
    ([1, 2], [70000, 5000], 4, 4, 64, 16, 40, 3, 4),
    ([1, 1], [1000, 70], 40, 1, 128, 16, 7, 1, 1),     # more query heads than a tile has rows
    ([2], [900], 8, 8, 64, 16, 0, 1, 2),               # nothing but the first and the last pages
    ([1], [20000], 2, 1, 64, 16, 300, 10, 20),         # a long list
    ([1] * 300, list(range(0, 1500, 5)), 4, 2, 64, 16, 3, 1, 1),
    ([1], [3000], 16, 2, 128, 1024, 1, 0, 1),
]


@pytest.mark.parametrize("new,past,Hq,Hkv,D,page,top,first,recent", CASES)
def test_sparse_attention(new, past, Hq, Hkv, D, page, top, first, recent):
    rng = np.random.default_rng(sum(past) + D)
    b = Batch(rng, new, past, page)
    c = filled(rng, b, Hkv, D)
    bounds = all_bounds(c, b)
    q64, q = queries(rng, b.T, Hq, D)
    blocks = torch.full((b.T, Hkv, top + first + recent), -7, dtype=torch.int32, device="cuda")
    out = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, b.max_new(), top, first, recent, blocks=blocks)
    want, tol, pages, _ = expected(q64, c, bounds, b.table, b.cu, b.len, b.T, top, first, recent)
    assert (blocks.cpu().numpy() == pages).all()
    check(out, want, tol, "sparse")
    # strided queries and outputs, in place, without the list
    wide = torch.full((b.T, Hq + 2, D), float("nan"), dtype=BF16, device="cuda")
    wide[:, 1:Hq + 1] = q
    M.moe_kv4_sparse_attention(c, bounds, wide[:, 1:Hq + 1], *b.dev, b.max_new(), top, first, recent,
                               out=wide[:, 1:Hq + 1])
    assert torch.equal(wide[:, 1:Hq + 1], out) and torch.isnan(wide[:, 0]).all() and torch.isnan(wide[:, -1]).all()


def test_all_pages_is_causal_attention():
    rng = np.random.default_rng(11)
    b = Batch(rng, [5, 1, 30], [100, 300, 0], 16)
    c = filled(rng, b, 2, 128)
    bounds = all_bounds(c, b)
    q64, q = queries(rng, b.T, 8, 128)
    out = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 30, top=50)
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, 128 ** -0.5)
    check(out, want, tol, "everything taken")


def test_ties_go_to_the_lower_page():
    """Pages with the same bounds, in groups, at every border of the list."""
    rng = np.random.default_rng(12)
    page, W, D = 16, 700, 64
    b = Batch(rng, [1], [W * page - 1], page)
    c = filled(rng, b, 1, D)
    bounds = torch.zeros((c.num_pages, 1, 2, D), dtype=BF16, device="cuda")
    level = rng.integers(0, 5, W)
    bounds[b.dev[0][0, :W].long()] = torch.from_numpy(level).cuda().to(BF16)[:, None, None, None]
    q = torch.ones((1, 1, D), dtype=BF16, device="cuda")
    for top in (1, 2, 100, 139, 140, 141, 200, 333, 697, 698, 699, 800):
        blocks = torch.empty((1, 1, top + 2), dtype=torch.int32, device="cuda")
        M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 1, top, blocks=blocks)
        order = sorted(range(1, W - 1), key=lambda i: (-level[i], i))[:top]
        want = sorted([0, W - 1] + order)
        assert blocks[0, 0].tolist() == want + [-1] * (top + 2 - len(want)), top


def test_near_scores_are_told_apart():
    """Scores that differ in the 24th bit only, of terms that cancel: decided as in 64 bits."""
    rng = np.random.default_rng(13)
    page, W, D = 16, 400, 128
    b = Batch(rng, [1], [W * page - 1], page)
    c = filled(rng, b, 1, D)
    v = bf16_values(rng.standard_normal((1, 1, 1, D)) * 8).repeat(c.num_pages, 0)
    v[:, 0, 0, :2] += bf16_values(rng.standard_normal((c.num_pages, 2)) * 2.0 ** -9)  # some round away
    bounds = dev_bits(round_to_bf16_bits(np.concatenate([v, v], axis=2))).view(BF16)
    q64, q = queries(rng, 1, 4, D)
    blocks = torch.empty((1, 1, 52), dtype=torch.int32, device="cuda")
    M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 1, 50, blocks=blocks)
    _, _, pages, _ = expected(q64, c, bounds, b.table, b.cu, b.len, 1, 50, 1, 1)
    assert (blocks.cpu().numpy() == pages).all()


def test_nan_and_infinite_bounds():
    rng = np.random.default_rng(14)
    b = Batch(rng, [2], [1000], 16)
    c = filled(rng, b, 2, 64)
    bounds = all_bounds(c, b)
    pg = b.dev[0][0].long()
    bounds[pg[3], 0, 0, 5] = float("nan")
    bounds[pg[4], 1, 1, 6] = float("inf")
    bounds[pg[5], 0, 0, 7] = -float("inf")
    bounds[pg[6]] = float("nan")
    q64, q = queries(rng, 2, 4, 64)
    q64[:, :, 6], q[:, :, 6] = 0.0, 0.0  # 0 * inf is NaN
    for top in (3, 50, 60, 61):
        blocks = torch.empty((2, 2, top + 2), dtype=torch.int32, device="cuda")
        out = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 2, top, blocks=blocks)
        want, tol, pages, _ = expected(q64, c, bounds, b.table, b.cu, b.len, 2, top, 1, 1)
        assert (blocks.cpu().numpy() == pages).all(), top
        check(out, want, tol, f"top {top}")


def test_unseen_keys_never_reach_a_result():
    """NaN in pages that are not taken and in slots behind the token's own leave no trace."""
    rng = np.random.default_rng(15)
    b = Batch(rng, [4, 1], [500, 130], 32)
    c = filled(rng, b, 1, 128)
    bounds = all_bounds(c, b)
    _, q = queries(rng, b.T, 4, 128)
    blocks = torch.empty((b.T, 1, 6), dtype=torch.int32, device="cuda")
    out = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 4, 4, blocks=blocks)
    used = {int(b.table[s, p]) for t, s in enumerate([0, 0, 0, 0, 1]) for p in blocks[t, 0].tolist() if p >= 0}
    for m in (c.k, c.v):
        for p in set(range(c.num_pages)) - used:
            m.scales[p], m.biases[p] = float("nan"), float("inf")
        for s in range(2):  # behind the last token
            m.scales[int(b.table[s, (b.len[s] - 1) // 32]), 0, (b.len[s] - 1) % 32 + 1:] = float("nan")
    assert torch.equal(M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 4, 4), out)


def test_hostile_batches():
    """Pages outside the cache, positions past the table or before it, rows of no sequence and tokens
    past max_new."""
    rng = np.random.default_rng(16)
    b = Batch(rng, [3, 2, 4, 6, 5], [200, 330, 0, 0, 90], 16)
    c = filled(rng, b, 2, 64)
    bounds = all_bounds(c, b)
    table = b.table.copy()
    table[0, 1], table[0, 5], table[1, 20], table[4, 5] = b.num_pages, -1, 2 ** 31 - 1, -2 ** 31
    lens = [b.len[0], b.len[1], table.shape[1] * 16 + 2, 3, b.len[4]]
    T = b.T + 3
    q64, q = queries(rng, T, 4, 64)
    for max_new in (6, 3):
        blocks = torch.full((T, 2, 7), -9, dtype=torch.int32, device="cuda")
        out = torch.full((T, 4, 64), 6.0, dtype=BF16, device="cuda")
        M.moe_kv4_sparse_attention(c, bounds, q, i32(table), i32(b.cu), i32(lens), max_new, 4, 1, 2, blocks=blocks, out=out)
        want, tol, pages, done = expected(q64, c, bounds, table, b.cu, lens, T, 4, 1, 2, max_new=max_new)
        got = blocks.cpu().numpy()
        assert (got[done] == pages[done]).all() and (got[~done] == -9).all()
        assert (out[torch.from_numpy(~done).cuda()] == 6.0).all() and (~done).sum() >= 3
        check(out[torch.from_numpy(done).cuda()], want[done], tol[done], f"max_new {max_new}")


def test_no_page_at_all():
    """A token whose pages do not exist gets zeros and an empty list."""
    rng = np.random.default_rng(17)
    b = Batch(rng, [1, 1], [100, 40], 16)
    c = filled(rng, b, 1, 64)
    _, q = queries(rng, 2, 2, 64)
    table = np.full_like(b.table, -1)
    table[1] = b.table[1]
    for top in (0, 4):
        blocks = torch.empty((2, 1, top + 2), dtype=torch.int32, device="cuda")
        out = M.moe_kv4_sparse_attention(c, all_bounds(c, b), q, i32(table), *b.dev[1:], 1, top, blocks=blocks)
        assert (out[0] == 0).all() and (blocks[0] == -1).all() and (out[1] != 0).any()


def test_many_rows_in_parts():
    """More rows than one part's score keys hold: the same as the rows on their own."""
    rng = np.random.default_rng(18)
    page, D, W = 16, 64, 2 ** 16
    b = Batch(rng, [1100], [900], page, width=W)
    c = filled_pages(rng, b, 1, D)
    bounds = all_bounds(c, b)
    _, q = queries(rng, b.T, 2, D)
    need = M.moe_kv4_sparse_attention_workspace_bytes(c, b.T, 2, 1, W, 1100, 4)
    assert need >= 256 << 20
    blocks = torch.empty((b.T, 1, 6), dtype=torch.int32, device="cuda")
    out = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 1100, 4, blocks=blocks)
    # the same batch with a table of the pages that are used
    small = torch.empty_like(blocks)
    short = (b.dev[0][:, :126].contiguous(), *b.dev[1:])
    assert torch.equal(M.moe_kv4_sparse_attention(c, bounds, q, *short, 1100, 4, blocks=small), out)
    assert torch.equal(small, blocks)


def filled_pages(rng, b, Hkv, D):
    """As filled(), for a table much wider than the sequences: pages past theirs repeat."""
    used = -(-max(b.len) // b.page) + 1
    b.num_pages = used + 3
    b.table = np.arange(b.table.shape[1])[None] % b.num_pages
    b.dev = (i32(b.table), *b.dev[1:])
    return filled(rng, b, Hkv, D)


def test_refusals():
    rng = np.random.default_rng(19)
    b = Batch(rng, [2], [40], 16)
    c = filled(rng, b, 1, 64)
    bounds = all_bounds(c, b)
    _, q = queries(rng, 2, 2, 64)
    ok = dict(cache=c, bounds=bounds, q=q, page_table=b.dev[0], cu=b.dev[1], kv_len=b.dev[2], max_new=2, top=2)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for bad in (dict(bounds=bounds[:-1]), dict(bounds=bounds.float()), dict(bounds=bounds.transpose(2, 3)), dict(top=-1),
                dict(first=-1), dict(recent=0), dict(top=5000), dict(blocks=i(2, 1, 5)), dict(blocks=i(2, 1, 4).long()),
                dict(max_new=0), dict(max_new=-1), dict(q=q[:, :, :32]), dict(q=q.float()), dict(scale=0.0),
                dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(bounds=bounds.cpu()), dict(top=2 ** 40)):
        with pytest.raises(M.MoeError):
            M.moe_kv4_sparse_attention(**{**ok, **bad})
    with pytest.raises(M.MoeError):
        M.moe_kv4_bounds(c, bounds[:, :, :1], *b.dev, 2)
    with pytest.raises(M.MoeError):
        M.moe_kv4_bounds(c, bounds, *b.dev, -1)
    assert M.moe_kv4_sparse_attention(**{**ok, "q": q[:0], "cu": i(2)}).shape == (0, 2, 64)


MORE = [  # prompts and rows of several kinds: new, earlier, Hq, Hkv, D, page, top, first, recent
    ([100], [5000], 8, 2, 256, 32, 6, 1, 2),
    ([64], [3000], 5, 1, 128, 16, 9, 0, 1),
    ([80] + [1] * 69, [900] + list(range(10, 1390, 20)), 4, 2, 64, 16, 3, 1, 1),   # many sequences, one of them a prompt
    ([150, 0, 65, 1], [0, 40, 2000, 700], 64, 1, 64, 16, 4, 2, 1),
    ([300], [0], 4, 4, 128, 16, 5, 1, 1),
    ([400], [300], 16, 16, 256, 16, 3, 1, 1),     # three lists and more for each wavefront of the card
    ([480], [200], 32, 32, 64, 16, 2, 0, 2),
    ([290, 0, 1], [300, 60, 700], 64, 32, 128, 16, 3, 1, 1),
    ([100], [700], 18, 2, 128, 16, 3, 1, 1),      # 9 heads a list
    ([5, 1], [700, 90], 14, 2, 64, 16, 3, 1, 1),  # 7
]


@pytest.mark.parametrize("new,past,Hq,Hkv,D,page,top,first,recent", MORE)
def test_sparse_prompts(new, past, Hq, Hkv, D, page, top, first, recent):
    test_sparse_attention(new, past, Hq, Hkv, D, page, top, first, recent)


@pytest.mark.parametrize("W", [3000, 9000])
def test_ties_in_long_tables(W):
    """Lists from tables whose keys are held eight a lane, or not held: the border inside ties of more
    and of fewer pages than are ranked at once."""
    rng = np.random.default_rng(W)
    b = Batch(rng, [1], [W * 16 - 1], 16)
    c = filled(rng, b, 1, 64)
    level = np.where(rng.random(W) < 0.01, 3, rng.integers(0, 3, W))
    bounds = torch.zeros((c.num_pages, 1, 2, 64), dtype=BF16, device="cuda")
    bounds[b.dev[0][0, :W].long()] = torch.from_numpy(level).cuda().to(BF16)[:, None, None, None]
    q = torch.ones((1, 2, 64), dtype=BF16, device="cuda")
    many = int((level[1:-1] == 3).sum())
    for top in (1, many - 1, many, many + 1, many + 300):
        blocks = torch.empty((1, 1, top + 2), dtype=torch.int32, device="cuda")
        M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, 1, top, blocks=blocks)
        order = sorted(range(1, W - 1), key=lambda i: (-level[i], i))[:top]
        assert blocks[0, 0].tolist() == sorted([0, W - 1] + order), top


@pytest.mark.parametrize("new", [[3], [70]])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 66, 2.0 ** -100, 2.0 ** 120])
def test_queries_of_any_size(scale, new):
    """Queries outside the range that the fast scores are bounded for, zeros, infinities and NaN: the
    pages are still those of the scores in 64 bits, and other tokens' do not change."""
    rng = np.random.default_rng(31)
    b = Batch(rng, new, [1500], 16)
    c = filled(rng, b, 2, 128)
    bounds = all_bounds(c, b)
    q64, q = queries(rng, b.T, 6, 128)
    q64, q = q64 * scale, q * scale
    q64[1, :, :64] = 0
    q[1, :, :64] = 0
    blocks = torch.empty((b.T, 2, 12), dtype=torch.int32, device="cuda")
    out = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, b.T, 10, blocks=blocks)
    with np.errstate(over="ignore", invalid="ignore"):
        bb = bf16_to_f64(host_bits(bounds))
        for t in range(b.T):
            for h in range(2):
                p = B.select(q64[t, 3 * h:3 * h + 3], bb[b.table[0], h, 0], bb[b.table[0], h, 1],
                             np.ones(b.table.shape[1], bool), 1500 + t, 16, 10, 1, 1)
                assert blocks[t, h].tolist() == p.tolist() + [-1] * (12 - len(p)), (t, h)
    q[0, 0, 5], q[2, 3, 7] = float("nan"), float("inf")
    more = torch.empty_like(blocks)
    again = M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, b.T, 10, blocks=more)
    rest = [t for t in range(b.T) if t not in (0, 2)]
    assert torch.equal(again[rest].nan_to_num(7.0), out[rest].nan_to_num(7.0)) and torch.equal(more[rest], blocks[rest])
    # a NaN query's scores are all NaN: its pages are the first ones
    assert more[0, 0].tolist() == list(range(11)) + [(b.len[0] - b.T) // 16]
    assert torch.equal(more[0, 1], blocks[0, 1]) and torch.equal(more[2, 0], blocks[2, 0])


def test_far_pages():
    """Cache offsets past 2^32: the write, the bounds and attention on the last pages of a large cache,
    against a small one."""
    rng = np.random.default_rng(33)
    n, Hkv, page, D = 70000, 8, 64, 256
    big, small = M.KV4Cache.empty(n, Hkv, page, D), M.KV4Cache.empty(9, Hkv, page, D)
    assert big.k.codes.numel() > 2 ** 32
    bb = torch.empty((n, Hkv, 2, D), dtype=BF16, device="cuda")
    bs = torch.empty((9, Hkv, 2, D), dtype=BF16, device="cuda")
    T = 500
    _, x = queries(rng, T, 3 * Hkv, D)
    order = rng.permutation(9)[:8]
    rope = M.Rope.make(128)
    outs = []
    for cache, bounds, table in ((big, bb, n - 1 - order), (small, bs, order)):
        batch = (i32(table[None]), i32([0, T]), i32([T]))
        q = M.moe_kv4_rope_append(cache, x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], rope, *batch)
        M.moe_kv4_bounds(cache, bounds, *batch, T)
        outs.append((q, M.moe_kv4_sparse_attention(cache, bounds, q, *batch, T, 2), bounds[i32(table).long()],
                     *M.moe_kv4_read(cache, *batch, T)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_bounds_follow_a_rejected_draft():
    """A sequence cut back and refilled: its pages' bounds are those of the tokens it has now."""
    rng = np.random.default_rng(34)
    b = Batch(rng, [5], [30], 16)
    c = filled(rng, b, 1, 64)
    got = all_bounds(c, b)
    x = torch.from_numpy(100 * rng.standard_normal((2, 1, 64))).cuda().to(BF16)
    M.moe_kv4_append(c, x, x, b.dev[0], i32([0, 2]), i32([33]))  # tokens 31 and 32 anew, 33 and 34 gone
    M.moe_kv4_bounds(c, got, b.dev[0], i32([0, 2]), i32([33]), 2)
    keys = whole(c)
    want = B.bounds(keys[b.table[0, :3], 0], 33)
    assert (host_bits(got)[b.table[0, :3], 0] == round_to_bf16_bits(want)).all()


@pytest.mark.parametrize("new", [[2], [66]])
def test_scores_next_to_the_largest_number(new):
    """Scores on both sides of fp32's largest number: infinite ones tie, finite ones next to them do not."""
    rng = np.random.default_rng(37)
    b = Batch(rng, new, [16 * 200], 16)
    c = filled(rng, b, 1, 64)
    n = c.num_pages
    top = 3.3e38 * (1 - 2.0 ** -rng.integers(3, 12, size=(n, 1, 1, 64)))
    bounds = torch.from_numpy(np.concatenate([-top, top], axis=2).astype(np.float32)).cuda().to(BF16)
    # 128 terms of 0.0083 times 3.3e38 (1 - 0.0277 on average) are 3.409e38, the largest number 3.403e38
    q = torch.full((b.T, 2, 64), 0.0083, device="cuda").to(BF16)
    q[:, 1] *= -1
    blocks = torch.empty((b.T, 1, 42), dtype=torch.int32, device="cuda")
    M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, b.T, 40, blocks=blocks)
    bb = bf16_to_f64(host_bits(bounds))[b.table[0], 0]
    with np.errstate(over="ignore"):
        score = np.abs(q[0].double().cpu().numpy()) @ bb[:, 1].T
        finite = np.isfinite(score.sum(0).astype(np.float32))
        assert 20 < finite[:200].sum() < 180
        for t in range(b.T):
            p = B.select(q[t].double().cpu().numpy(), bb[:, 0], bb[:, 1], np.ones(len(bb), bool), 3200 + t, 16, 40, 1, 1)
            assert blocks[t, 0].tolist() == p.tolist()


@pytest.mark.parametrize("new,past,width", [([2], 900, 0), ([70], 900, 0), ([2], 3000, 0), ([70], 3000, 0),
                                            ([300], 3000, 2100), ([2], 3000, 9000)])
@pytest.mark.parametrize("D", [64, 256])
def test_infinite_bounds_under_any_sign(new, past, width, D):
    """Infinite bounds on either side, under channels whose queries are all positive, all negative, of
    both signs or zero, and infinite queries: a page's score is the formula's, term by term."""
    rng = np.random.default_rng(41)
    b = Batch(rng, new, [past], 16)
    if width:
        b.table = np.concatenate([b.table, np.zeros((1, width - b.table.shape[1]), dtype=b.table.dtype)], axis=1)
        b.dev = (i32(b.table), *b.dev[1:])
    c = filled(rng, b, 2, D)
    v = np.sort(rng.standard_normal((c.num_pages, 2, 2, D)), axis=2)
    for kind, (side, value) in enumerate(((0, -np.inf), (1, np.inf), (0, np.inf), (1, -np.inf), (0, -np.inf))):
        at = rng.random(c.num_pages) < 0.12
        h, ch = rng.integers(0, 2, c.num_pages), rng.integers(0, D, c.num_pages)
        v[at, h[at], side, ch[at]] = value
        if kind >= 2:  # both sides, alike or not
            v[at, h[at], 1 - side, ch[at]] = np.inf if kind == 4 else value
    bounds = dev_bits(round_to_bf16_bits(v)).view(BF16)
    q64, q = queries(rng, b.T, 6, D)
    for ch in range(D):  # a sign for each channel, or none
        sign = ch % 4
        if sign < 2:
            q64[:, :, ch] = np.abs(q64[:, :, ch]) * (1 - 2 * sign)
        elif ch % 16 == 3:
            q64[:, ch % 6, ch] = 0.0
    q64[1, 1, 4], q64[1, 4, 5] = np.inf, -np.inf
    q = torch.from_numpy(q64).cuda().to(BF16)
    bb = bf16_to_f64(host_bits(bounds))
    ok = np.ones(b.table.shape[1], bool)
    for top in (4, 25, 45):
        blocks = torch.empty((b.T, 2, top + 2), dtype=torch.int32, device="cuda")
        M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, b.T, top, blocks=blocks)
        for t in range(b.T):
            for h in range(2):
                p = B.select(q64[t, 3 * h:3 * h + 3], bb[b.table[0], h, 0], bb[b.table[0], h, 1], ok, past + t, 16, top, 1, 1)
                assert blocks[t, h].tolist() == p.tolist() + [-1] * (top + 2 - len(p)), (top, t, h)


@pytest.mark.parametrize("new,past", [([1] * 5, [0, 70, 300, 16, 155]), ([90], [200])])
def test_a_budget_past_the_table(new, past):
    """More pages allowed than the table holds: as many as it holds, and the list ends there."""
    rng = np.random.default_rng(43)
    b = Batch(rng, new, past, 16)
    W = b.table.shape[1]
    c = filled(rng, b, 2, 128)
    bounds = all_bounds(c, b)
    q64, q = queries(rng, b.T, 8, 128)
    lists = [torch.full((b.T, 2, top + 2), -7, dtype=torch.int32, device="cuda") for top in (W - 2, 4000)]
    outs = [M.moe_kv4_sparse_attention(c, bounds, q, *b.dev, b.max_new(), x.shape[2] - 2, blocks=x) for x in lists]
    assert torch.equal(*outs) and torch.equal(lists[1][:, :, :W], lists[0]) and (lists[1][:, :, W:] == -1).all()
    want, tol = K.attention(q64, K.Paged(*host_planes(c), b.table), b.cu, b.len, 128 ** -0.5)
    check(outs[0], want, tol, "everything taken")


@pytest.mark.parametrize("new,past", [
    ([20] * 30, [7 * i % 90 for i in range(30)]),  # tiles of few tokens
    ([175, 334, 200], [40, 7, 100]),               # prompts; a workgroup's tiles before the part, across its border and in it
])
def test_parts_that_end_inside_a_tile(new, past):
    """Parts of 341 rows, a multiple of no tile, out of place and in place (a tile's earlier rows then
    hold results already): the oracle's pages and outputs for every row."""
    rng = np.random.default_rng(44)
    page, D, Hkv, W = 16, 64, 3, 2 ** 16
    b = Batch(rng, new, past, page)
    c = filled(rng, b, Hkv, D)
    bounds = all_bounds(c, b)
    q64, q = queries(rng, b.T, 2 * Hkv, D)
    table = np.concatenate([b.table, np.zeros((b.B, W - b.table.shape[1]), dtype=b.table.dtype)], axis=1)
    dev = (i32(table), *b.dev[1:])
    one, two = (M.moe_kv4_sparse_attention_workspace_bytes(c, T, 2 * Hkv, b.B, W, b.max_new(), 3) for T in (341, 342))
    assert b.T > 341 and one == two  # the 342nd row is another part's
    blocks = torch.empty((b.T, Hkv, 5), dtype=torch.int32, device="cuda")
    out = M.moe_kv4_sparse_attention(c, bounds, q, *dev, b.max_new(), 3, blocks=blocks)
    want, tol, pages, _ = expected(q64, c, bounds, b.table, b.cu, b.len, b.T, 3, 1, 1)
    assert (blocks.cpu().numpy() == pages).all()
    check(out, want, tol, "parts")
    again = torch.empty_like(blocks)
    M.moe_kv4_sparse_attention(c, bounds, q, *dev, b.max_new(), 3, blocks=again, out=q)
    assert torch.equal(again, blocks) and torch.equal(q, out)
