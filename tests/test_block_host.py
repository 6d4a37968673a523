"""Norms, rotary positions, page bounds and attention over selected pages without a GPU: the C
ABI's argument validation (every call returns before any HIP call), the binding's refusals, the
frequencies, and the oracle against brute force."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
from oracle import block_oracle as B

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
A, X, Y, H, S, W = (0x100000 * (i + 1) for i in range(6))  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        from bit_quantized_grouped_router_amd import build
        build.build()
    return M.lib()


def norm(L, T=3, d=128, x=X, xs=128, xd=0, r=None, rs=128, h=None, hs=128, hd=0, w=W, plus=0, eps=1e-6, y=Y, ys=128,
         yd=0, scales=None, group=0):
    return L.moe_rmsnorm(T, d, x, xs, xd, r, rs, h, hs, hd, w, plus, eps, y, ys, yd, scales, group, None)


def test_rmsnorm_refusals(L):
    for bad, st in [(dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769, xs=40000, ys=40000), UNSUPPORTED),
                    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                    (dict(eps=float("inf")), INVALID), (dict(xd=2), INVALID), (dict(yd=4), INVALID),
                    (dict(yd=-1), INVALID), (dict(r=A, hd=2), INVALID), (dict(h=H), INVALID), (dict(xs=127), INVALID),
                    (dict(ys=127), INVALID), (dict(r=A, rs=127), INVALID), (dict(r=A, h=H, hs=1), INVALID),
                    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(x=X + 2), ALIGN),
                    (dict(y=Y + 8), ALIGN), (dict(r=A + 4), ALIGN), (dict(w=W + 2), ALIGN),
                    (dict(yd=2, scales=S, group=0), INVALID), (dict(yd=2, scales=S, group=100), INVALID),
                    (dict(yd=2, scales=S, group=32), UNSUPPORTED), (dict(yd=3, scales=None, group=64), INVALID),
                    (dict(yd=3, scales=S + 4, group=64), ALIGN),
                    (dict(y=X, yd=1), INVALID), (dict(y=X, ys=136), INVALID), (dict(y=W), INVALID),
                    (dict(r=A, y=A), INVALID), (dict(r=A, h=A, hs=136), INVALID), (dict(r=A, h=X), INVALID),
                    (dict(r=A, h=Y), INVALID), (dict(yd=2, scales=X, group=64), INVALID),
                    (dict(yd=2, scales=Y, group=64), INVALID)]:
        assert norm(L, **bad) == st, bad
    assert norm(L, T=0, x=None, w=None, y=None) == OK


def spec(freqs=A, rot=64, interleaved=0, magnitude=1.0):
    return M.MoeRopeSpec(freqs, rot, interleaved, magnitude)


def rope(L, T=3, heads=4, D=128, x=X, xs=512, xd=0, pos=S, r=None, n=None, out=Y, os_=512, od=0):
    return L.moe_rope(T, heads, D, x, xs, xd, pos, spec() if r is None else r, n, out, os_, od, None)


BAD_ROPE = [(spec(rot=0), INVALID), (spec(rot=63), INVALID), (spec(rot=130), INVALID), (spec(freqs=None), INVALID),
            (spec(freqs=A + 4), ALIGN)]
BAD_NORM = [(M.MoeHeadNorm(None, 1e-6, 0), INVALID), (M.MoeHeadNorm(W + 2, 1e-6, 0), ALIGN),
            (M.MoeHeadNorm(W, 0.0, 0), INVALID), (M.MoeHeadNorm(W, float("nan"), 0), INVALID)]


def test_rope_refusals(L):
    for bad, st in [(dict(T=-1), INVALID), (dict(heads=0), INVALID), (dict(D=0), INVALID), (dict(D=100), UNSUPPORTED),
                    (dict(D=520), UNSUPPORTED), (dict(T=2 ** 30, heads=8, xs=1024, os_=1024), UNSUPPORTED),
                    (dict(xd=2), INVALID), (dict(od=3), INVALID), (dict(xs=504), INVALID), (dict(xs=516), UNSUPPORTED),
                    (dict(os_=500), INVALID), (dict(x=None), INVALID), (dict(pos=None), INVALID),
                    (dict(out=None), INVALID), (dict(x=X + 8), ALIGN), (dict(pos=S + 4), ALIGN),
                    (dict(out=X, od=1), INVALID), (dict(out=X, os_=520), INVALID), (dict(out=S), INVALID),
                    (dict(out=A), INVALID)]:
        assert rope(L, **bad) == st, bad
    for r, st in BAD_ROPE:
        assert rope(L, r=r) == st
    for n, st in BAD_NORM:
        assert rope(L, n=n) == st
    assert L.moe_rope(3, 4, 128, X, 512, 0, S, None, None, Y, 512, 0, None) == INVALID
    assert rope(L, T=0, x=None, pos=None, out=None) == OK


def dims(B=2, Hq=16, Hkv=2, D=128, page=16, num_pages=9, max_pages=4):
    return M.MoeKv4Dims(B, Hq, Hkv, D, page, num_pages, max_pages)


CACHE, BATCH = M.MoeKv4Cache(*[A] * 6), M.MoeKv4Batch(A, A, A)
BAD_DIMS = [(dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
            (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(B=65536), UNSUPPORTED),
            (dict(page=65536, max_pages=32768), UNSUPPORTED)]


def write(L, dm=None, c=CACHE, T=3, q=X, qs=2048, k=H, ks=256, v=W, vs=256, dtype=0, r=None, qn=None, kn=None, out=Y,
          os_=2048, b=BATCH):
    return L.moe_kv4_rope_append(dims() if dm is None else dm, c, T, q, qs, k, ks, v, vs, dtype,
                                 spec() if r is None else r, qn, kn, out, os_, b, None)


def test_rope_append_refusals(L):
    for bad, st in BAD_DIMS + [(dict(Hq=15), INVALID), (dict(Hq=0), INVALID)]:
        assert write(L, dm=dims(**bad)) == st, bad
    for bad, st in [(dict(T=-1), INVALID), (dict(dtype=2), INVALID), (dict(qs=2040), INVALID),
                    (dict(ks=252), INVALID), (dict(vs=260), UNSUPPORTED), (dict(os_=2052), UNSUPPORTED),
                    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=W + 2), ALIGN), (dict(out=Y + 4), ALIGN),
                    (dict(out=X, dtype=1), INVALID), (dict(out=X, os_=2056), INVALID), (dict(out=H), INVALID),
                    (dict(out=W), INVALID), (dict(c=M.MoeKv4Cache(*[0] * 6)), INVALID),
                    (dict(b=M.MoeKv4Batch(A, A + 4, A)), ALIGN), (dict(T=2 ** 27), UNSUPPORTED)]:
        assert write(L, **bad) == st, bad
    for r, st in BAD_ROPE:
        assert write(L, r=r) == st
    for n, st in BAD_NORM:
        assert write(L, qn=n) == st and write(L, kn=n) == st
    assert write(L, T=0, q=None, k=None, v=None, out=None) == OK


def test_bounds_refusals(L):
    call = lambda dm=None, c=CACHE, T=3, bounds=Y, b=BATCH: L.moe_kv4_bounds(dims() if dm is None else dm, c, T, bounds,
                                                                             b, None)
    for bad, st in BAD_DIMS:
        assert call(dm=dims(**bad)) == st, bad
    assert call(T=-1) == INVALID and call(bounds=None) == INVALID and call(bounds=Y + 8) == ALIGN
    assert call(b=M.MoeKv4Batch(0, 0, 0)) == INVALID and call(T=0, bounds=None) == OK


def sparse(L, dm=None, c=CACHE, bounds=S, T=3, new=3, q=X, qs=2048, out=Y, os_=2048, b=BATCH, pages=(5, 1, 2), scale=0.1,
           blocks=None, ws=A, ws_bytes=None):
    dm, pg = dims() if dm is None else dm, None if pages is None else M.MoeKv4Pages(*pages)
    if ws_bytes is None:
        ws_bytes = L.moe_kv4_sparse_attention_workspace_bytes(dm, T, new, pg)
    return L.moe_kv4_sparse_attention(dm, c, bounds, T, new, q, qs, out, os_, b, pg, scale, blocks, ws, ws_bytes, None)


def test_sparse_refusals(L):
    for bad, st in BAD_DIMS + [(dict(Hq=15), INVALID), (dict(Hq=65, Hkv=1), UNSUPPORTED),
                               (dict(max_pages=2 ** 20 + 1), UNSUPPORTED)]:
        assert sparse(L, dm=dims(**bad)) == st, bad
    for bad, st in [(dict(T=-1), INVALID), (dict(new=0), INVALID), (dict(new=-1), INVALID),
                    (dict(pages=None), INVALID), (dict(pages=(-1, 1, 1)), INVALID), (dict(pages=(1, -1, 1)), INVALID),
                    (dict(pages=(1, 1, 0)), INVALID), (dict(pages=(4094, 2, 1)), UNSUPPORTED),
                    (dict(pages=(2 ** 31 - 1, 2 ** 31 - 1, 1)), UNSUPPORTED), (dict(scale=0.0), INVALID),
                    (dict(scale=float("nan")), INVALID), (dict(scale=2.0 ** 65), INVALID), (dict(qs=2047), INVALID),
                    (dict(os_=2049), UNSUPPORTED), (dict(q=None), INVALID), (dict(out=Y + 4), ALIGN),
                    (dict(bounds=None), INVALID), (dict(bounds=S + 2), ALIGN), (dict(blocks=W + 4), ALIGN),
                    (dict(out=X, os_=2056), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 8), ALIGN),
                    (dict(ws_bytes=0), WORKSPACE), (dict(c=None), INVALID)]:
        assert sparse(L, **bad) == st, bad
    need = L.moe_kv4_sparse_attention_workspace_bytes(dims(), 3, 3, M.MoeKv4Pages(5, 1, 2))
    assert need > 0 and sparse(L, ws_bytes=need - 1) == WORKSPACE
    assert sparse(L, T=0, q=None, out=None, ws=None) == OK
    for bad in (dict(D=100), dict(Hq=130)):
        assert L.moe_kv4_sparse_attention_workspace_bytes(dims(**bad), 3, 3, M.MoeKv4Pages(5, 1, 2)) == 0
    assert L.moe_kv4_sparse_attention_workspace_bytes(dims(), 0, 0, M.MoeKv4Pages(5, 1, 2)) == 0


PLANES = M.MoeKv4Cache(*(0x2000000 + 0x100000 * i for i in range(6)))
ARRAYS = M.MoeKv4Batch(*(0x3000000 + 0x100000 * i for i in range(3)))
FREQS, QW, KW, WS = (0x4000000 + 0x100000 * i for i in range(4))
HELD = [getattr(c, f) for c in (PLANES, ARRAYS) for f, _ in c._fields_]


def test_outputs_at_inputs_addresses(L):
    """What a call writes lies nowhere that its other workgroups read or write."""
    for at in HELD + [FREQS, QW, KW, H, W]:
        assert write(L, c=PLANES, b=ARRAYS, r=spec(freqs=FREQS), qn=M.MoeHeadNorm(QW, 1e-6, 0),
                     kn=M.MoeHeadNorm(KW, 1e-6, 0), out=at) == INVALID, hex(at)
    for at in HELD:
        assert L.moe_kv4_bounds(dims(), PLANES, 3, at, ARRAYS, None) == INVALID, hex(at)
    own = dict(c=PLANES, b=ARRAYS, ws=WS, blocks=H)
    for at in HELD + [S, WS]:
        assert sparse(L, **{**own, "out": at}) == INVALID, hex(at)
    for at in HELD + [S, WS, X, Y]:
        assert sparse(L, **{**own, "blocks": at}) == INVALID, hex(at)
    for at in HELD + [S, X, Y, H]:
        assert sparse(L, **{**own, "ws": at}) == INVALID, hex(at)


def test_sparse_workspace_is_bounded(L):
    """Score keys are held for a part of a long call's rows: 256 MB and what the rows' lists take."""
    dm = dims(B=1, Hq=64, Hkv=8, page=16, max_pages=8192, num_pages=8192)
    one = L.moe_kv4_sparse_attention_workspace_bytes(dm, 1, 1, M.MoeKv4Pages(60, 2, 2))
    assert 8 * 8192 * 4 <= one <= 16 << 20
    most = L.moe_kv4_sparse_attention_workspace_bytes(dm, 131072, 131072, M.MoeKv4Pages(60, 2, 2))
    assert 256 << 20 <= most <= 300 << 20


def test_sparse_workspace_of_a_budget_past_the_table(L):
    """Lists are as wide as the page table at the most, whatever a token may take."""
    for T, new, Hq, Hkv, width in ((32768, 32768, 64, 8, 64), (1, 1, 16, 2, 40), (64, 1, 16, 2, 512)):
        dm = dims(B=1 if new == T else T, Hq=Hq, Hkv=Hkv, max_pages=width, num_pages=4096)
        need = lambda top: L.moe_kv4_sparse_attention_workspace_bytes(dm, T, new, M.MoeKv4Pages(top, 1, 1))
        assert need(width - 2) == need(width - 1) == need(4094) > need(1), (T, width)
    most = L.moe_kv4_sparse_attention_workspace_bytes(dims(B=1, Hq=64, Hkv=8, max_pages=4096, num_pages=4096), 2 ** 20,
                                                      2 ** 20, M.MoeKv4Pages(4094, 1, 1))
    assert 512 << 20 <= most <= 700 << 20  # keys and lists


def test_binding_refusals():
    """Shapes, types and devices that the binding itself refuses (nothing reaches the library)."""
    x = torch.zeros(2, 8)
    with pytest.raises((M.MoeError, RuntimeError, AssertionError)):
        M.moe_rmsnorm(x, torch.zeros(8, dtype=torch.bfloat16))  # not in GPU memory, or no GPU
    with pytest.raises(M.MoeError):
        M.moe_rmsnorm(torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(M.MoeError):
        M.moe_rope(x, None, None)
    for bad in (torch.zeros(2, 2), torch.zeros(4, dtype=torch.float64), torch.zeros(8)[::2]):
        with pytest.raises(M.MoeError):
            M.Rope(bad)


def test_sizes_past_32_bits():
    """Sizes that the C interface's integers would cut to others are refused."""
    x = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="meta")
    w, many = x(8), 2 ** 32 + 3
    for bad in (x(many, 8), x(1, many)):
        with pytest.raises(M.MoeError, match="32 bits"):
            M.moe_rmsnorm(bad, w)
    r = M.Rope(torch.ones(4))
    for bad in (x(many, 1, 8), x(1, many, 8), x(1, 1, many)):
        with pytest.raises(M.MoeError, match="32 bits"):
            M.moe_rope(bad, r, w)
    g = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t)
    plane = lambda: M.W4Matrix(g(9, 2, 16, 32, t=torch.uint8), g(9, 2, 16, 1), g(9, 2, 16, 1))
    c, i = M.KV4Cache(plane(), plane()), lambda *s: torch.zeros(s, dtype=torch.int32)
    for T in (many, -1):
        with pytest.raises(M.MoeError, match="T "):
            M.moe_kv4_bounds(c, g(9, 2, 2, 64), i(1, 4), i(2), i(1), T)
    ok = dict(cache=c, T=4, Hq=4, B=1, max_pages=4, max_new=4, top=2)
    assert M.moe_kv4_sparse_attention_workspace_bytes(**ok) > 0
    for k in ("T", "Hq", "B", "max_pages", "top", "first", "recent"):
        assert M.moe_kv4_sparse_attention_workspace_bytes(**{**ok, k: 2 ** 32 + 4}) == 0, k


def test_frequencies():
    """Each scaling at both ends: the fastest pair, the slowest, and no scaling at factor 1."""
    f = lambda **k: M.Rope.make(device="cpu", **k)
    plain = f(rot=64, base=1e6)
    assert plain.magnitude == 1.0 and plain.freqs.shape == (32,)
    want = np.array([1e6 ** (-2 * i / 64) for i in range(32)], dtype=np.float32)
    assert (plain.freqs.numpy() == want).all()
    assert (f(rot=64, base=1e6, scaling="linear", factor=4.0).freqs == plain.freqs / 4).all()
    raised = f(rot=64, base=1e6, scaling="base", factor=4.0).freqs
    assert raised[0] == 1.0 and abs(raised[-1] / plain.freqs[-1] * 4 - 1) < 1e-6
    assert (raised[1:] < plain.freqs[1:]).all()
    ramp = f(rot=64, base=1e4, scaling="ramp", factor=8.0, trained=4096)
    base = f(rot=64, base=1e4).freqs
    turns = 4096 * base.double() / (2 * math.pi)
    assert torch.equal(ramp.freqs[turns >= 32 * 1.4], base[turns >= 32 * 1.4])
    assert torch.equal(ramp.freqs[turns <= 1 / 1.4], base[turns <= 1 / 1.4] / 8)
    assert (ramp.freqs[1:] < ramp.freqs[:-1]).all() and abs(ramp.magnitude - (0.1 * math.log(8) + 1)) < 1e-12
    for s in ("none", "linear", "base"):
        assert torch.equal(f(rot=64, base=1e6, scaling=s).freqs, plain.freqs)
    assert f(rot=2, scaling="base", factor=2.0).freqs.tolist() == [0.5]
    for bad in (dict(rot=3), dict(rot=0), dict(rot=64, base=1.0), dict(rot=64, factor=0.5), dict(rot=64, scaling="x"),
                dict(rot=64, scaling="ramp", factor=2.0), dict(rot=64, scaling="ramp", factor=2.0, trained=9, fast=1.0)):
        with pytest.raises(M.MoeError):
            f(**bad)


@pytest.mark.parametrize("trained", [1, 6, 7, 40, 128, 300, 4096, 10 ** 6])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (64.0, 32.0), (2.0, 1.5), (1e-3, 1e-4)])
def test_ramp_keeps_and_divides_what_it_says(trained, fast, slow):
    """Pairs of at least `fast` turns stay and those of at most `slow` are divided, also where every
    pair is one or the other; what lies between falls from one to the other."""
    base = M.Rope.make(64, base=1e4, device="cpu").freqs.double()
    ramp = M.Rope.make(64, base=1e4, scaling="ramp", factor=8.0, trained=trained, fast=fast, slow=slow, device="cpu").freqs
    turns = trained * base / (2 * math.pi)
    # the turns of fp32 frequencies, at a border, decide to 2^-20 of it
    few, many = turns <= slow * (1 - 2.0 ** -20), turns >= fast * (1 + 2.0 ** -20)
    assert torch.equal(ramp[few], (base[few] / 8).float()) and torch.equal(ramp[many], base[many].float())
    assert (ramp <= base * (1 + 2.0 ** -24)).all() and (ramp >= base / 8 * (1 - 2.0 ** -24)).all()
    assert ((ramp / base)[1:] <= (ramp / base)[:-1] * (1 + 2.0 ** -22)).all()


# ------------------------------------------------------------------ the oracle

def test_oracle_rope_keeps_products():
    """A turn keeps each pair's length, and a score only depends on the distance of positions."""
    rng = np.random.default_rng(1)
    f = np.array([1.0, 0.3, 0.01])
    for inter in (False, True):
        q, k = rng.standard_normal((2, 1, 1, 8))
        at = lambda x, p: B.rope(x, np.array([p]), f, inter)[0]
        assert np.allclose(np.linalg.norm(at(q, 977)), np.linalg.norm(q))
        assert np.allclose((at(q, 1000) * at(k, 990)).sum(), (at(q, 13) * at(k, 3)).sum())
        assert (at(q, 5)[..., 6:] == q[..., 6:]).all() and (at(q, 0) == q).all()
    a, b = B.pairs(6, True)
    assert list(a) == [0, 2, 4] and list(b) == [1, 3, 5]
    one = np.zeros((1, 1, 4))
    one[0, 0, 0] = 1.0
    y = B.rope(one, np.array([1]), np.array([math.pi / 2, 0.1]))[0]
    assert np.allclose(y[0, 0], [0, 0, 1, 0])  # channel 0's partner is rot / 2


def test_oracle_norm():
    y, s = B.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.5, np.array([[0.0, 0.0]]))
    assert np.allclose(y, np.array([[3.0, 8.0]]) / math.sqrt(13.0)) and (s == [[3.0, 4.0]]).all()


def test_oracle_select():
    """By hand: always-taken pages, ties, pages that do not exist, NaN, and the bound itself."""
    rng = np.random.default_rng(2)
    lo, hi = np.sort(rng.standard_normal((2, 10, 4)), axis=0)
    q = rng.standard_normal((3, 4))
    # the score bounds the sum of any keys' scores inside the page
    s = np.maximum(q[:, None] * lo, q[:, None] * hi).sum((0, 2))
    for _ in range(50):
        keys = lo + rng.random((10, 4)) * (hi - lo)
        assert ((q @ keys.T).sum(0) <= s + 1e-12).all()
    both = np.minimum(q, 0).sum(0) @ lo.T + np.maximum(q, 0).sum(0) @ hi.T
    assert np.allclose(s, both)
    ones = np.ones((1, 1))
    sel = lambda score, exists=None, pos=159, **k: list(B.select(
        ones, np.array(score, dtype=float)[:, None], np.array(score, dtype=float)[:, None],
        np.ones(10, bool) if exists is None else np.array(exists, bool), pos, 16, **k))
    score = [9, 1, 5, 5, 2, 5, 8, 0, 9, 9]
    assert sel(score, top=2, first=1, recent=2) == [0, 2, 6, 8, 9]
    assert sel(score, top=3, first=1, recent=2) == [0, 2, 3, 6, 8, 9]
    assert sel(score, top=0, first=1, recent=1) == [0, 9]
    assert sel(score, top=99, first=0, recent=1) == list(range(10))
    assert sel(score, pos=20, top=1, first=1, recent=1) == [0, 1]
    assert sel(score, pos=-3, top=1, first=1, recent=1) == []
    assert sel(score, pos=10 ** 6, top=1, first=0, recent=1) == [0, 9]
    assert sel(score, exists=[0, 1, 1, 1, 1, 1, 0, 1, 1, 0], top=2, first=1, recent=2) == [2, 3, 8]
    score[6] = float("nan")
    assert sel(score, top=1, first=1, recent=2) == [0, 2, 8, 9]
    assert sel(score, top=7, first=1, recent=2) == list(range(10))


def test_oracle_bounds():
    v = np.array([[[1.0, -0.0], [2.0, 0.0]], [[-3.0, 5.0], [np.nan, 7.0]]])
    b = B.bounds(v, 4)
    assert (b[0] == [[1, 0], [2, 0]]).all() and not np.signbit(b[0]).any()
    assert np.isnan(b[1, :, 0]).all() and (b[1, :, 1] == [5, 7]).all()
    assert (B.bounds(v, 3)[1] == [[-3, 5], [-3, 5]]).all() and (B.bounds(v, 2)[1] == 0).all()


def test_index_arithmetic_on_hostile_positions(tmp_path):
    """kv4_scored and the spans of rows, compiled for the host: what is scored lies before the token's
    own page and inside the table, whatever the position."""
    src, so = tmp_path / "scored.cpp", tmp_path / "scored.so"
    src.write_text('''
#include "moe_kv4_sparse.h"
using namespace moe;
extern "C" void scored(int page_shift, int max_pages, long long pos, int first, int recent, int *out) {
  Kv4Dims dm{1, 1, 1, 64, 1 << page_shift, page_shift, 1, max_pages};
  const Kv4Scored s = kv4_scored(dm, pos, first, recent);
  out[0] = s.lo, out[1] = s.hi, out[2] = s.own;
}
extern "C" void row_span(int row, int len, long long *out) {
  const Kv4Span s = kv4_row_span(row, len);
  out[0] = s.begin, out[1] = s.n, out[2] = s.first, out[3] = s.len;
}
''')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    import subprocess
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-static-libubsan", "-shared", "-fPIC", "-I",
                    os.path.join(root, "bit_quantized_grouped_router_amd", "csrc"), str(src), "-o", str(so)], check=True)
    h = ctypes.CDLL(str(so))
    h.scored.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    out = (ctypes.c_int * 3)()
    for shift, pages in ((4, 1), (4, 100), (16, 32767), (10, 1 << 20)):
        cap = pages << shift
        for pos in (-2 ** 31, -1, 0, 1, (1 << shift) - 1, 1 << shift, cap - 1, cap, cap + 1, 2 ** 31 - 1):
            for first in (0, 1, 3, 4095):
                for recent in (1, 2, 4096):
                    h.scored(shift, pages, pos, first, recent, out)
                    lo, hi, own = out
                    assert own == (-1 if pos < 0 else min(pos, cap - 1) >> shift)
                    assert lo == first and hi == own - recent and hi < own < pages
    span = (ctypes.c_longlong * 4)()
    for row, n in ((0, -1), (5, -2 ** 31), (7, 0), (9, 12)):
        h.row_span(row, n, span)
        assert list(span) == ([row, 0, 0, 0] if n < 0 else [row, 1, n - 1, n])
