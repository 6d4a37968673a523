"""The norm, the rotary positions and the rotated cache write on the GPU against the fp64 oracle.

fp32 arithmetic is held to bounds counted from its roundings; 8-bit codes and what the rotated write
leaves in the cache are compared bit for bit with what the fp32 results round to."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
from oracle import block_oracle as B
from oracle import kv4_oracle as K
from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits
from parity_util import host_bits, say
from test_gpu_kv4 import Batch, host_planes, i32, make_cache

pytestmark = pytest.mark.gpu

BF16, F32, E4M3, INT8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def values(rng, shape, dtype, scale=1.0):
    """(fp64 values, the same on the GPU)."""
    t = torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dtype)
    return t.double().numpy(), t.cuda()


def padded(t, extra):
    """The same rows further apart, NaN between them."""
    if t is None:
        return None
    w = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert (np.isnan(got) == np.isnan(want)).all(), what
    ok = np.isfinite(want)
    assert (got[~ok & ~np.isnan(want)] == want[~ok & ~np.isnan(want)]).all(), what
    off = np.abs(got - want)[ok]
    if off.size:
        say(f"  {what}: worst {float((off / np.maximum(tol[ok], 1e-300)).max()):.3f} of the bound")
    assert (off <= tol[ok]).all(), what


# ------------------------------------------------------------------ norm

ROWS = [  # rows, channels: every number of threads a row and of steps, vectors or not
    (1, 1), (1, 2048), (3, 7), (5, 64), (2, 100), (300, 512), (2, 513), (65, 2048), (2100, 1000), (2100, 2048),
    (2049, 504), (2050, 1023), (7, 5001), (4, 6144), (3, 8200), (2, 20000), (2, 32768), (1, 32767),
]


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("xt,rt,yt", [(BF16, None, BF16), (F32, F32, BF16), (BF16, BF16, F32), (F32, None, F32),
                                      (BF16, F32, BF16), (F32, BF16, F32)])
def test_norm(T, d, xt, rt, yt):
    rng = np.random.default_rng(T * 7 + d)
    x64, x = values(rng, (T, d), xt)
    r64, r = values(rng, (T, d), rt, 3.0) if rt else (None, None)
    w64, w = values(rng, d, BF16)
    plus = d % 2 == 1
    want, s = B.rmsnorm(x64, w64 + plus, 1e-5, r64)
    tol = np.abs(want) * (B.norm_terms(d) * U + half_step(yt)) + 1e-40
    got = M.moe_rmsnorm(x, w, eps=1e-5, residual=r, plus_one=plus, out_dtype=yt)
    y, h = got if rt else (got, None)
    within(y, want, tol, "y")
    if rt:
        within(h, s, np.abs(s) * (U + half_step(rt)) + 1e-40, "h")
    # rows at other distances, aligned or not: the same bits
    for extra in (8, 3):
        y2 = torch.full((T, d + extra), 7.0, dtype=yt, device="cuda")[:, :d]
        h2 = torch.full((T, d + extra), 7.0, dtype=rt, device="cuda")[:, :d] if rt else None
        M.moe_rmsnorm(padded(x, extra), w, eps=1e-5, residual=padded(r, extra), plus_one=plus, y=y2, h=h2)
        assert torch.equal(y2, y) and (not rt or torch.equal(h2, h))
        assert T == 1 or (y2.as_strided((T - 1, extra), (d + extra, 1), d) == 7.0).all()
    if rt:  # the sum onto the residual itself
        M.moe_rmsnorm(x, w, eps=1e-5, residual=r, h=r, plus_one=plus, y=y2)
        assert torch.equal(r, h) and torch.equal(y2, y)
    if xt == yt:  # the norm onto its input
        x2 = x.clone()
        M.moe_rmsnorm(x2, w, eps=1e-5, residual=None if not rt else values(rng, (T, d), rt)[1] * 0, plus_one=plus, y=x2)
        plain = M.moe_rmsnorm(x, w, eps=1e-5, plus_one=plus, out_dtype=yt)
        assert torch.equal(x2, plain)


@pytest.mark.parametrize("T,d,group", [(5, 64, 0), (5, 64, 64), (3, 128, 128), (70, 2048, 0), (70, 2048, 64),
                                       (777, 5120, 128), (2100, 1024, 128), (2100, 1024, 0), (3, 1001, 0), (2, 20096, 64),
                                       (2, 32768, 0), (1, 1, 0), (4, 192, 64)])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_norm_to_8_bits(T, d, group, kind):
    """Scales and codes are those of the fp32 result, bit for bit."""
    rng = np.random.default_rng(T + d)
    _, x = values(rng, (T, d), BF16)
    _, r = values(rng, (T, d), F32)
    _, w = values(rng, d, BF16)
    x[0] = 0
    r[0] = 0  # a row of zeros
    if T > 4:
        r[1, 0], r[2, d - 1], x[3, d // 2] = float("nan"), float("inf"), -float("inf")
        r[4] *= 1e-30
    y32, h = M.moe_rmsnorm(x, w, residual=r, out_dtype=F32)
    for extra in (0, 8, 5):
        q, scales, h2 = M.moe_rmsnorm(padded(x, extra), w, residual=padded(r, extra), out_dtype=kind, group=group)
        assert torch.equal(h2[torch.isfinite(h2)], h[torch.isfinite(h)]) and scales.shape == (T, d // (group or d))
        y = y32.cpu().numpy().reshape(T, -1, group or d)
        with np.errstate(all="ignore"):
            top = np.abs(y).max(-1)
            want = (top / np.float32(448 if kind == E4M3 else 127)).astype(np.float32)
            want[~np.isfinite(top)] = np.nan
            t = np.where(want[..., None] > 0, y / want[..., None], np.float32(0)).reshape(T, d)
        assert np.array_equal(scales.cpu().numpy(), want, equal_nan=True)
        t = np.clip(np.nan_to_num(t), -448 if kind == E4M3 else -127, 448 if kind == E4M3 else 127)
        if kind == E4M3:
            codes = torch.from_numpy(t.astype(np.float32)).to(E4M3).view(torch.uint8).numpy()
            got = q.view(torch.uint8).cpu().numpy()
        else:
            codes, got = np.rint(t).astype(np.int8), q.cpu().numpy()
        assert (codes == got).all()


def test_norm_special_rows():
    """A NaN or an infinity stays in its row; a row of zeros is zeros; a sum that leaves fp32 gives zeros."""
    x = torch.randn((6, 2048), device="cuda")
    w = torch.ones(2048, dtype=BF16, device="cuda")
    x[1, 5], x[2, 7], x[3], x[4, 0] = float("nan"), float("inf"), 0.0, 1e25
    y = M.moe_rmsnorm(x, w, out_dtype=F32)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 7]) and (y[2, :7] == 0).all() and (y[3] == 0).all()
    assert torch.isfinite(y[[0, 3, 4, 5]]).all() and (y[4] == 0).all()


def test_norm_refusals():
    x, w = torch.zeros((4, 64), device="cuda"), torch.zeros(64, dtype=BF16, device="cuda")
    for bad in (dict(weight=w[:32]), dict(weight=w.float()), dict(residual=x[:3]), dict(residual=x.half()),
                dict(h=x.clone()), dict(y=torch.zeros((4, 63), dtype=BF16, device="cuda")), dict(out_dtype=torch.float16),
                dict(group=64), dict(scales=x), dict(out_dtype=INT8, group=48), dict(out_dtype=INT8, group=32),
                dict(out_dtype=INT8, group=-64), dict(out_dtype=E4M3, scales=torch.zeros(4, device="cuda")),
                dict(residual=x.clone(), h=x), dict(weight=w.cpu()), dict(x=x.t()), dict(x=x[0]), dict(y=w.expand(4, 64)),
                dict(x=x.double()), dict(eps=0.0), dict(out_dtype=BF16, y=x)):
        with pytest.raises(M.MoeError):
            M.moe_rmsnorm(**{**dict(x=x, weight=w), **bad})
    empty = M.moe_rmsnorm(x[:0], w)
    assert empty.shape == (0, 64)


# ------------------------------------------------------------------ rotary positions

HEADS = [  # tokens, heads, channels, channels turned
    (1, 1, 8, 8), (1, 16, 256, 64), (3, 5, 64, 64), (2, 3, 72, 50), (7, 4, 128, 128), (5, 1, 96, 2), (4, 2, 512, 512),
    (130, 9, 128, 90), (4200, 3, 64, 32), (1030, 16, 128, 128), (9, 40, 40, 40), (6, 70, 16, 12), (3, 2, 264, 132),
]


def close_to(rng, x64, x, positions, freqs, w64, w, inter, magnitude, yt, **kw):
    n64 = x64 if w64 is None else B.rmsnorm(x64, w64, 1e-6)[0]
    want, size = B.rope(n64, positions, freqs.double().cpu().numpy(), inter, magnitude)
    # sine and cosine: the turn in fp32 (2 pi 2^-25), 4 ulp of the function, the magnitude's product
    per = 2 * np.pi * 2.0 ** -25 + 5 * U + 3 * U + (0 if w64 is None else B.norm_terms(x64.shape[-1]) * U)
    rest = 0 if w64 is None else np.abs(want) * B.norm_terms(x64.shape[-1]) * U  # channels that pass
    return want, size * per + rest + np.abs(want) * half_step(yt) + 1e-40


@pytest.mark.parametrize("T,H,D,rot", HEADS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xt,yt,norm", [(BF16, BF16, True), (F32, BF16, False), (BF16, F32, False), (F32, F32, True)])
def test_rope(T, H, D, rot, inter, xt, yt, norm):
    rng = np.random.default_rng(T + H + D + rot)
    x64, x = values(rng, (T, H, D), xt)
    w64, w = values(rng, D, BF16) if norm else (None, None)
    positions = rng.integers(0, 1 << 20, T)
    positions[:1] = rng.choice([0, -7, 2 ** 31 - 1, 131071])
    freqs = M.Rope.make(rot, interleaved=inter).freqs
    rope = M.Rope(freqs, inter, 1.25)
    pos = i32(positions)
    want, tol = close_to(rng, x64, x, positions, freqs, w64, w, inter, 1.25, yt)
    y = M.moe_rope(x, rope, pos, weight=w, out_dtype=yt)
    within(y, want, tol, "rope")
    # heads in the middle of wider rows, in and out
    wide = torch.full((T, H + 3, D), float("nan"), dtype=xt, device="cuda")
    wide[:, 1:H + 1] = x
    out = torch.full((T, H + 2, D), 3.0, dtype=yt, device="cuda")
    M.moe_rope(wide[:, 1:H + 1], rope, pos, weight=w, out=out[:, 2:])
    assert torch.equal(out[:, 2:], y) and (out[:, :2] == 3.0).all()
    if xt == yt:
        M.moe_rope(wide[:, 1:H + 1], rope, pos, weight=w, out=wide[:, 1:H + 1])
        assert torch.equal(wide[:, 1:H + 1], y) and torch.isnan(wide[:, 0]).all() and torch.isnan(wide[:, H + 1:]).all()


def test_rope_special_values():
    """Infinities and NaN turn with their partner only; channels past rot pass whatever they hold."""
    x = torch.randn((2, 2, 64), device="cuda")
    x[0, 0, 3], x[0, 1, 40], x[1, 0, 63] = float("inf"), float("nan"), float("inf")
    for inter in (False, True):
        y = M.moe_rope(x, M.Rope.make(32, interleaved=inter), i32([5, 0]))
        assert torch.equal(y[:, :, 32:].nan_to_num(7.0), x[:, :, 32:].nan_to_num(7.0))
        partner = 2 if inter else 19
        bad = ~torch.isfinite(y[0, 0])
        assert bad.nonzero().flatten().tolist() == sorted([3, partner])
        assert torch.equal(y[1, :, :32], x[1, :, :32])  # position 0


def test_rope_refusals():
    x, pos, r = torch.zeros((4, 2, 64), device="cuda"), i32([1, 2, 3, 4]), M.Rope.make(32)
    for bad in (dict(positions=pos[:3]), dict(positions=pos.long()), dict(rope=M.Rope.make(66)), dict(x=x.half()),
                dict(weight=torch.zeros(32, dtype=BF16, device="cuda")), dict(out=x.to(BF16), out_dtype=F32),
                dict(x=torch.zeros((4, 2, 60), device="cuda")), dict(positions=pos.cpu()), dict(x=x[0]),
                dict(rope=M.Rope(torch.ones(16))), dict(out=x.transpose(0, 1)), dict(out_dtype=INT8),
                dict(weight=torch.ones(64, dtype=BF16, device="cuda"), eps=0.0)):
        with pytest.raises(M.MoeError):
            M.moe_rope(**{**dict(x=x, rope=r, positions=pos), **bad})
    assert M.moe_rope(x[:0], r, pos[:0]).shape == (0, 2, 64)


# ------------------------------------------------------------------ the rotated write

WRITES = [  # new tokens, earlier tokens, Hq, Hkv, D, page, rot
    ([1], [0], 1, 1, 64, 16, 64),
    ([1] * 8, [15, 16, 31, 0, 5, 700, 63, 64], 16, 2, 256, 16, 64),
    ([3, 0, 17, 1], [14, 2, 0, 100], 3, 1, 128, 32, 90),
    ([5, 70], [60, 0], 9, 3, 64, 64, 2),
    ([2] * 70, list(range(70)), 4, 4, 64, 16, 48),
    ([1500, 3000], [100, 7], 8, 2, 128, 64, 128),
    ([2], [131070], 64, 8, 128, 128, 128),
]


@pytest.mark.parametrize("new,past,Hq,Hkv,D,page,rot", WRITES)
@pytest.mark.parametrize("dtype,inter,norm", [(BF16, False, True), (F32, True, False), (F32, False, True)])
def test_rope_append(new, past, Hq, Hkv, D, page, rot, dtype, inter, norm):
    rng = np.random.default_rng(len(new) * 1000 + D)
    b = Batch(rng, new, past, page)
    T = b.T + 2  # two rows behind the last sequence
    both64, both = values(rng, (T, Hq + 2 * Hkv, D), dtype)
    q, k, v = both[:, :Hq], both[:, Hq:Hq + Hkv], both[:, Hq + Hkv:]
    w64 = [values(rng, D, BF16) for _ in range(2)] if norm else [(None, None)] * 2
    rope = M.Rope.make(rot, scaling="linear", factor=2.0, interleaved=inter)
    c = make_cache(b.num_pages, Hkv, page, D)
    before = host_planes(c)
    out = torch.full((T, Hq, D), 5.0, dtype=BF16, device="cuda")
    got = M.moe_kv4_rope_append(c, q, k, v, rope, *b.dev, q_weight=w64[0][1], k_weight=w64[1][1], eps=1e-6, q_out=out)
    assert got is out and (out[b.T:] == 5.0).all()
    positions = np.concatenate([np.arange(t - n, t) for n, t in zip(b.new, b.len)])
    want, tol = close_to(rng, both64[:b.T, :Hq], q, positions, rope.freqs, w64[0][0], None, inter, 1.0, BF16)
    within(out[:b.T], want, tol, "queries")
    # the cache holds exactly the quantised turned keys
    turned = M.moe_rope(k[:b.T], rope, i32(positions), weight=w64[1][1], out_dtype=F32)
    alone = M.moe_rope(q[:b.T], rope, i32(positions), weight=w64[0][1], out_dtype=BF16)
    assert torch.equal(alone, out[:b.T])
    _, pg, sl = K.token_slots(b.cu, b.len, b.table, page, b.T)
    for name, x, old, now in zip("kv", (turned, v[:b.T]), before, host_planes(c)):
        for field, a, o, g in zip(("codes", "scales", "biases"), quantised(x), old, now):
            o[pg, :, sl] = a
            assert (o == g).all(), f"{name}.{field}"
    if dtype == BF16:
        M.moe_kv4_rope_append(c, q, k, v, rope, *b.dev, q_weight=w64[0][1], k_weight=w64[1][1], eps=1e-6, q_out=q)
        assert torch.equal(q[:b.T], out[:b.T])


def quantised(x):
    q, s, z = K.quantise(np.ascontiguousarray(x.float().cpu().numpy()))
    return K.pack(q), s, z


def test_rope_append_without_a_place():
    """Positions past the table, pages outside the cache, lengths that do not fit: queries are turned
    at the positions the lengths say, nothing is written elsewhere."""
    rng = np.random.default_rng(4)
    b = Batch(rng, [20, 20, 4, 6], [12, 30, 0, 0], 16)
    table = b.table.copy()
    table[0, 1], table[1, 2] = b.num_pages, -5
    lens = [b.len[0], b.len[1], table.shape[1] * 16 + 2, 3]  # the last sequence has fewer tokens than rows
    dev = (i32(table), i32(b.cu), i32(lens))
    x64, x = values(rng, (b.T, 4, 64), F32)
    c = make_cache(b.num_pages, 1, 16, 64)
    before = host_planes(c)
    rope = M.Rope.make(64)
    out = M.moe_kv4_rope_append(c, x[:, :2], x[:, 2:3], x[:, 3:], rope, *dev)
    positions = np.concatenate([np.arange(t - n, t) for n, t in zip(b.new, lens)])
    assert torch.equal(out, M.moe_rope(x[:, :2], rope, i32(positions), out_dtype=BF16))
    turned = M.moe_rope(x[:, 2:3], rope, i32(positions))
    _, pg, sl = K.token_slots(b.cu, lens, table, 16, b.T)
    placed = (pg >= 0) & (pg < b.num_pages)
    assert 0 < placed.sum() < b.T
    for y, old, now in zip((turned, x[:, 3:]), before, host_planes(c)):
        for a, o, g in zip(quantised(y), old, now):
            o[pg[placed], :, sl[placed]] = a[placed]
            assert (o == g).all()


def test_rope_append_refusals():
    c = make_cache(8, 2, 16, 64)
    dev = (i32([[0, 1]]), i32([0, 4]), i32([4]))
    x = torch.zeros((4, 8, 64), device="cuda")
    r = M.Rope.make(64)
    ok = dict(cache=c, q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], rope=r, page_table=dev[0], cu=dev[1], kv_len=dev[2])
    for bad in (dict(k=x[:, 4:7]), dict(v=x[:3, 6:]), dict(k=x[:, 4:6].to(BF16)), dict(q=x[:, :3]), dict(q=x[0]),
                dict(rope=M.Rope.make(66)), dict(q_out=x[:, :4]), dict(q_weight=torch.ones(32, dtype=BF16, device="cuda")),
                dict(k_weight=torch.ones(64, device="cuda")), dict(kv_len=dev[2].long()), dict(q=x[:, :4].half())):
        with pytest.raises(M.MoeError):
            M.moe_kv4_rope_append(**{**ok, **bad})
    M.moe_kv4_rope_append(**ok)


def test_far_rows():
    """Rows so far apart that their offsets pass 32 bits: the norm and the rotation."""
    wide = torch.empty((1030, 1 << 22), dtype=BF16, device="cuda")
    x = torch.randn((1030, 64), device="cuda").to(BF16)
    wide[:, :64] = x
    w = torch.ones(64, dtype=BF16, device="cuda")
    assert torch.equal(M.moe_rmsnorm(wide[:, :64], w), M.moe_rmsnorm(x, w))
    pos, r = i32(np.arange(1030)), M.Rope.make(32)
    heads = wide[:, :64].unflatten(1, (2, 32))
    want = M.moe_rope(x.view(1030, 2, 32), r, pos)
    assert torch.equal(M.moe_rope(heads, r, pos), want)
    M.moe_rope(heads, r, pos, out=heads)
    assert torch.equal(heads, want)


def test_rope_against_differences():
    """A score of two turned vectors depends on their distance alone, near and far."""
    rng = np.random.default_rng(3)
    _, x = values(rng, (2, 1, 128), F32)
    for inter in (False, True):
        r = M.Rope.make(128, interleaved=inter)
        dots = []
        for p in (0, 1000, 130000, 1 << 24):
            y = M.moe_rope(x, r, i32([p + 77, p]))
            dots.append(float((y[0].double() * y[1].double()).sum()))
        # the frequencies' products with positions are exact, so the angles' distance is
        assert max(abs(d - dots[0]) for d in dots) <= 128 * 8 * 5 * U * 4


def test_stream_argument():
    """Work on a stream given as argument, outputs and workspaces allocated for it."""
    s = torch.cuda.Stream()
    x, w = torch.randn((4096, 2048), device="cuda"), torch.ones(2048, dtype=BF16, device="cuda")
    want = M.moe_rmsnorm(x, w, residual=x)
    heads = x.view(4096, 16, 128)
    pos, r = i32(np.arange(4096)), M.Rope.make(128)
    turned = M.moe_rope(heads, r, pos)
    torch.cuda.synchronize()
    for _ in range(5):
        a = M.moe_rmsnorm(x, w, residual=x, stream=s)
        b = M.moe_rope(heads, r, pos, stream=s)
        s.synchronize()
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1]) and torch.equal(b, turned)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("first", [0, 100000, 2 ** 28])
def test_products_are_rounded_apart(inter, first):
    """fp32 results are the sum of two rounded products, bit for bit, with the cosines and sines that
    (1, 0) is turned to; those are the ones in 64 bits, rounded, but where that is next to a tie."""
    T, D = 300, 128
    r, pos = M.Rope.make(D, interleaved=inter), i32(np.arange(first, first + T))
    unit = torch.zeros((T, 1, D), device="cuda")
    lo, hi = (slice(0, None, 2), slice(1, None, 2)) if inter else (slice(0, D // 2), slice(D // 2, None))
    unit[..., lo] = 1
    u = M.moe_rope(unit, r, pos)
    c, s = u[..., lo], u[..., hi]
    angle = pos.double()[:, None] * r.freqs.double()
    for got, want in ((c[:, 0], torch.cos(angle)), (s[:, 0], torch.sin(angle))):
        # off by half a step at the most, and what 2^-44 is of it (of the smallest sine, 2^-24 or so, more)
        step = torch.nextafter(got.abs(), torch.full_like(got, 2.0)).double() - got.abs().double()
        assert ((got.double() - want).abs() <= step / 2 + 2.0 ** -44).all()
    _, x = values(np.random.default_rng(5), (T, 6, D), F32)
    y = M.moe_rope(x, r, pos)
    a, b = x[..., lo], x[..., hi]
    assert torch.equal(y[..., lo], a * c - b * s) and torch.equal(y[..., hi], a * s + b * c)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("first", [2 ** 29 - 150, 2 ** 30 + 12345, 2 ** 31 - 300, -2 ** 31])
def test_angles_of_the_farthest_positions(inter, first):
    """Position times frequency has up to 55 bits; cosine and sine are those of the whole product,
    rounded to fp32 but where that is next to a tie."""
    T, D = 300, 128
    r, pos = M.Rope.make(D, interleaved=inter), np.arange(first, first + T)
    unit = torch.zeros((T, 1, D), device="cuda")
    lo, hi = (slice(0, None, 2), slice(1, None, 2)) if inter else (slice(0, D // 2), slice(D // 2, None))
    unit[..., lo] = 1
    u = M.moe_rope(unit, r, i32(pos))
    f = r.freqs.double().cpu().numpy()
    angle = pos.astype(np.float64)[:, None] * f
    # what fp64 rounds off the product, in whole numbers of 2^-60 (a frequency is at most 1 and at least 10000^-1)
    whole = lambda v: int(v * 2.0 ** 60) if abs(v) < 2 else int(v) * 2 ** 60 + int((v - int(v)) * 2.0 ** 60)
    off = np.array([[(int(p) * whole(float(g)) - whole(float(a))) * 2.0 ** -60 for g, a in zip(f, row)]
                    for p, row in zip(pos, angle)])
    assert (np.abs(off) <= 2.0 ** -23).all() and ((off != 0).any() or abs(first) < 2 ** 30)
    cos, sin = np.cos(angle), np.sin(angle)
    cos, sin = cos - off * sin - off ** 2 / 2 * cos, sin + off * cos - off ** 2 / 2 * sin  # off^3 is below 2^-69
    for got, want in ((u[:, 0, lo], cos), (u[:, 0, hi], sin)):
        got = got.cpu().numpy()
        # half a step, and 2^-44 as in test_products_are_rounded_apart
        assert (np.abs(got.astype(np.float64) - want) <= np.spacing(np.abs(got)).astype(np.float64) / 2 + 2.0 ** -44).all()
