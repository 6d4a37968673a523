"""The 4-bit cache and the int4-g64 projection without a GPU: argument validation of the C
ABI (every call returns before any HIP call), and the index arithmetic the kernels share
with the host, compiled for the CPU and tried on hostile lengths and page numbers."""
import ctypes
import os
import subprocess

import pytest

import bit_quantized_grouped_router_amd as M

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
FAKE = 0x100000  # never dereferenced
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        from bit_quantized_grouped_router_amd import build
        build.build()
    return M.lib()


def plane(p=FAKE):
    return M.MoeW4Matrix(p, p, p)


def dims(B=2, Hq=16, Hkv=2, D=128, page=16, num_pages=9, max_pages=4):
    return M.MoeKv4Dims(B, Hq, Hkv, D, page, num_pages, max_pages)


def cache(p=FAKE):
    return M.MoeKv4Cache(p, p, p, p, p, p)


def batch(p=FAKE):
    return M.MoeKv4Batch(p, p, p)


def move(L, name, dm=None, c=None, T=3, k=FAKE, ks=256, v=FAKE, vs=256, dtype=0, b=None):
    R = ctypes.byref
    return getattr(L, name)(R(dims() if dm is None else dm), R(cache() if c is None else c), T, k, ks, v,
                            vs, dtype, R(batch() if b is None else b), None)


BAD_DIMS = [(dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID), (dict(page=0), INVALID),
            (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(D=96), UNSUPPORTED),
            (dict(D=512), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
            (dict(page=131072), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
            (dict(page=65536, max_pages=32768), UNSUPPORTED)]


@pytest.mark.parametrize("name", ["moe_kv4_append", "moe_kv4_read"])
def test_append_and_read_refusals(L, name):
    for bad, st in BAD_DIMS:
        assert move(L, name, dm=dims(**bad)) == st, bad
    assert move(L, name, T=-1) == INVALID
    assert move(L, name, dtype=2) == INVALID
    assert move(L, name, ks=255) == INVALID          # rows would overlap
    assert move(L, name, vs=260) == UNSUPPORTED      # rows lose their alignment
    assert move(L, name, k=None) == INVALID
    assert move(L, name, v=FAKE + 2) == ALIGN
    assert move(L, name, c=cache(FAKE + 8)) == ALIGN
    assert move(L, name, b=batch(0)) == INVALID
    assert move(L, name, T=0, k=None, v=None) == OK  # nothing to do


def attend(L, dm=None, T=3, max_new=3, q=FAKE, qs=2048, out=FAKE, os_=2048, scale=0.1, window=0,
           ws=FAKE, ws_bytes=None, c=None, b=None):
    R = ctypes.byref
    dm = dims() if dm is None else dm
    if ws_bytes is None:
        ws_bytes = L.moe_kv4_attention_workspace_bytes(R(dm), T, max_new, window)
    return L.moe_kv4_attention(R(dm), R(cache() if c is None else c), T, max_new, q, qs, out, os_,
                               R(batch() if b is None else b), scale, 1, window, ws, ws_bytes, None)


def test_attention_refusals(L):
    for bad, st in BAD_DIMS + [(dict(Hq=15), INVALID), (dict(Hq=0), INVALID)]:
        assert attend(L, dm=dims(**bad)) == st, bad
    assert attend(L, T=-1) == INVALID
    assert attend(L, max_new=0) == INVALID
    assert attend(L, window=-1) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attend(L, scale=scale) == INVALID
    assert attend(L, qs=2047) == INVALID
    assert attend(L, os_=2049) == UNSUPPORTED
    assert attend(L, q=None) == INVALID
    assert attend(L, out=FAKE + 4) == ALIGN
    assert attend(L, c=cache(0)) == INVALID
    assert attend(L, b=batch(FAKE + 4)) == ALIGN
    assert attend(L, T=0, q=None, out=None, ws=None) == OK


def test_attention_workspace(L):
    long = dims(B=1, page=128, max_pages=1024, num_pages=1024)
    need = L.moe_kv4_attention_workspace_bytes(ctypes.byref(long), 1, 1, 0)
    assert need > 0
    assert attend(L, dm=long, T=1, max_new=1, ws_bytes=need - 1) == WORKSPACE
    assert attend(L, dm=long, T=1, max_new=1, ws=None) == INVALID
    assert attend(L, dm=long, T=1, max_new=1, ws=FAKE + 8) == ALIGN
    # max_new past the rows there are changes nothing
    assert L.moe_kv4_attention_workspace_bytes(ctypes.byref(long), 1, 999, 0) == need
    # a window bounds what has to be split
    assert L.moe_kv4_attention_workspace_bytes(ctypes.byref(long), 1, 1, 64) <= need
    assert L.moe_kv4_attention_workspace_bytes(ctypes.byref(dims(D=100)), 1, 1, 0) == 0
    assert L.moe_kv4_attention_workspace_bytes(None, 1, 1, 0) == 0


def test_attention_limits(L):
    """The largest scale and row counts, and the prompts' workspace: none where their rows fill
    the card, and no more than a part for every row and split."""
    assert attend(L, scale=2.0 ** 65) == INVALID
    wide = dims(B=1, Hq=4, Hkv=1, D=64, page=128, max_pages=512, num_pages=512)
    ws = lambda dm, T, new: L.moe_kv4_attention_workspace_bytes(ctypes.byref(dm), T, new, 0)
    assert attend(L, dm=wide, T=2 ** 28, max_new=2 ** 28) == UNSUPPORTED   # 2^30 rows of a head
    assert attend(L, dm=wide, T=2 ** 29, max_new=1) == UNSUPPORTED         # 2^31 rows in all
    assert ws(wide, 2 ** 28, 2 ** 28) == 0
    assert ws(wide, 2 ** 20, 2 ** 20) == 0
    some = ws(wide, 2048, 2048)
    part = 2048 * 4 * (64 + 2) * 4
    assert some > part and some % part == 0 and some // part <= 8


def project(L, T=3, rows=5, cols=128, x=FAKE, xs=128, w=None, bias=None, act=0, res=None, rs=0, y=FAKE,
            ys=5, dtype=0):
    return L.moe_linear_w4(T, rows, cols, x, xs, ctypes.byref(plane() if w is None else w), bias, act, res,
                           rs, y, ys, dtype, None)


def test_linear_refusals(L):
    assert project(L, T=-1) == INVALID
    assert project(L, rows=0) == INVALID
    assert project(L, cols=0) == INVALID
    assert project(L, cols=100, xs=104) == UNSUPPORTED
    assert project(L, act=4) == INVALID
    assert project(L, act=-1) == INVALID
    assert project(L, dtype=2) == INVALID
    assert project(L, xs=120) == INVALID
    assert project(L, xs=130) == UNSUPPORTED
    assert project(L, ys=4) == INVALID
    assert project(L, res=FAKE * 2, rs=4) == INVALID
    assert project(L, res=FAKE, rs=6, ys=5) == INVALID   # y itself with another stride
    assert project(L, x=None) == INVALID
    assert project(L, y=FAKE + 2) == ALIGN
    assert project(L, bias=FAKE + 2) == ALIGN
    assert project(L, res=FAKE + 8, rs=5) == ALIGN
    assert project(L, w=plane(FAKE + 4)) == ALIGN
    assert project(L, rows=1 << 20, cols=1 << 14, xs=1 << 14, ys=1 << 20) == UNSUPPORTED
    assert project(L, T=0, x=None, y=None) == OK


SHIM = r"""
#include <cstdint>
#include "moe_kv4.h"
using namespace moe;
extern "C" void span(int c0, int c1, int len, int T, long long *o) {
  const Kv4Span s = kv4_span(c0, c1, len, T);
  o[0] = s.begin, o[1] = s.n, o[2] = s.first, o[3] = s.len;
}
static Kv4Dims dims(int page_shift, int num_pages, int max_pages) {
  return Kv4Dims{1, 1, 2, 64, 1 << page_shift, page_shift, num_pages, max_pages};
}
extern "C" void range(int page_shift, int max_pages, long long p0, long long p1, long long len, int causal,
                      int window, long long *o) {
  const Kv4Range r = kv4_range(dims(page_shift, 1, max_pages), p0, p1, len, causal, window);
  o[0] = r.lo, o[1] = r.hi;
}
extern "C" void share(long long lo, long long hi, int per, int splits, int split, int *o) {
  const Kv4Share s = kv4_share(Kv4Range{lo, hi}, per, splits, split);
  o[0] = s.begin, o[1] = s.end, o[2] = s.used;
}
extern "C" int page_ok(int num_pages, int page) { return kv4_page_ok(dims(4, num_pages, 1), page); }
extern "C" long long row(int page_shift, int page, int head, int slot) {
  return kv4_row(dims(page_shift, 1 << 30, 1), page, head, slot);
}
"""


@pytest.fixture(scope="module")
def H(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-static-libubsan", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "bit_quantized_grouped_router_amd", "csrc"), str(src), "-o", str(so)],
                   check=True)
    h = ctypes.CDLL(str(so))
    ll = ctypes.c_longlong
    h.range.argtypes = [ctypes.c_int, ctypes.c_int, ll, ll, ll, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    h.share.argtypes = [ll, ll, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    h.row.restype = ll
    return h


BIG = 2 ** 31 - 1
HOSTILE = [-BIG - 1, -7, -1, 0, 1, 5, 16, 17, 100, BIG]


def test_spans_stay_inside_the_rows(H):
    o = (ctypes.c_longlong * 4)()
    for T in (1, 16, 100):
        for c0 in HOSTILE:
            for c1 in HOSTILE:
                for ln in HOSTILE:
                    H.span(c0, c1, ln, T, o)
                    begin, n, first, length = o
                    assert 0 <= begin <= T and 0 <= n and begin + n <= T
                    assert first == length - n and length == max(ln, 0)
    H.span(3, 7, 20, 50, o)
    assert list(o) == [3, 4, 16, 20]


def test_ranges_stay_inside_the_table(H):
    o = (ctypes.c_longlong * 2)()
    for shift, width in ((4, 1), (4, 7), (6, 3), (16, 32767)):
        cap = width << shift
        for p0 in (-BIG, -1, 0, 3, 40, 111, cap, BIG):
            for p1 in (p0, p0 + 1, p0 + 50):
                for ln in (0, 1, 33, cap, BIG):
                    for causal in (0, 1):
                        for window in (0, 1, 16, BIG):
                            H.range(shift, width, p0, p1, ln, causal, window, o)
                            seen = [p for p in range(0, min(cap, ln, 300))
                                    if any((not causal or p <= i) and (not window or p > i - window)
                                           for i in {p0, p1})]
                            assert 0 <= o[0] and o[1] <= min(cap, ln)
                            for p in seen:
                                assert o[0] <= p < o[1]


def test_shares_cover_every_tile_once(H):
    o = (ctypes.c_int * 3)()
    for lo, hi in ((0, 0), (5, 5), (9, 3), (0, 1), (0, 32), (31, 33), (100, 100000), (0, BIG), (BIG - 40, BIG)):
        for splits, per in ((1, 1), (1, 16), (2, 0), (7, 16), (7, BIG), (512, 1), (512, 40)):
            tiles, used = [], None
            for s in range(splits):
                H.share(lo, hi, per, splits, s, o)
                used = o[2] if used is None else used
                assert o[2] == used and 1 <= used <= splits
                if s >= used:
                    assert o[0] >= o[1]
                if o[0] < o[1]:
                    tiles.append((o[0], o[1]))
            want = (lo // 32, -(-hi // 32)) if hi > lo else None
            if want is None:
                assert not tiles and used == 1
            else:
                assert tiles[0][0] == want[0] and tiles[-1][1] == want[1] and len(tiles) == used
                assert all(a[1] == b[0] for a, b in zip(tiles, tiles[1:]))


def test_pages(H):
    for page in HOSTILE:
        assert bool(H.page_ok(17, page)) == (0 <= page < 17)
    assert H.row(4, 3, 1, 5) == (3 * 2 + 1) * 16 + 5
    assert H.row(16, 2 ** 20, 1, 65535) == (2 ** 21 + 1) * 65536 + 65535  # past 32 bits


def test_binding_refuses_shapes_and_types():
    import torch
    t = torch.zeros
    bf = torch.bfloat16
    w = M.W4Matrix(t(1, 5, 32, dtype=torch.uint8), t(1, 5, 1, dtype=bf), t(1, 5, 1, dtype=bf))
    with pytest.raises(M.MoeError):
        M.moe_linear_w4(t(3, 128, dtype=bf), w)                # another width
    with pytest.raises(M.MoeError):
        M.moe_linear_w4(t(3, 64, dtype=bf), w, act="tanh")
    with pytest.raises(M.MoeError):
        M.moe_linear_w4(t(64, dtype=bf), w)
    g = t(4, 2, 16, 1, dtype=bf)
    codes = t(4, 2, 16, 32, dtype=torch.uint8)
    good = M.W4Matrix(codes, g, g)
    M.KV4Cache(good, good)
    for bad in (M.W4Matrix(codes, t(4, 2, 16, 2, dtype=bf), g), M.W4Matrix(codes, g.float(), g),
                M.W4Matrix(codes.float(), g, g), M.W4Matrix(codes[:3], g, g)):
        with pytest.raises(M.MoeError):
            M.KV4Cache(good, bad)
    assert M._rows(t(3, 2, 64), (3, 2, 64), "k", (torch.float32,)) == 128
    assert M._rows(t(3, 8, 64)[:, 2:4], (3, 2, 64), "k", (torch.float32,)) == 512
    assert M._rows(t(1, 5), (1, 5), "y", (torch.float32,)) == 8
    for bad in (t(3, 64, 2).transpose(1, 2), t(2, 64).expand(3, 2, 64), t(3, 2, 128)[..., ::2],
                t(3, 2, 32), t(3, 2, 64, dtype=bf)):
        with pytest.raises(M.MoeError):
            M._rows(bad, (3, 2, 64), "k", (torch.float32,))


PLACE_SHIM = r"""
#include "moe_kv4.h"
using namespace moe;
// how many (tile, head) of n x heads are not taken exactly once
extern "C" long long lost(int n, long long heads, int causal, int pair, unsigned char *seen) {
  for (long long i = 0; i < n * heads; ++i) seen[i] = 0;
  long long bad = 0;
  for (long long hs = 0; hs < heads; ++hs)
    for (int x = 0; x < n; ++x) {
      const Kv4Place p = kv4_prompt_place(x, hs, n, heads, causal, pair);
      if (p.tile < 0 || p.tile >= n || p.hs < 0 || p.hs >= heads) return -1;
      seen[p.hs * n + p.tile]++;
    }
  for (long long i = 0; i < n * heads; ++i) bad += seen[i] != 1;
  return bad;
}
// the tile that shares a CU with workgroup 0's, of one head
extern "C" int tile_of(int x, int n, int pair) { return kv4_prompt_place(x, 0, n, 1, true, pair).tile; }
"""


def test_prompt_tiles_are_taken_exactly_once(tmp_path):
    """Every row tile of every head by one workgroup, for all shapes of up to 512 tiles and
    heads, with and without a mask, in pairs and not; and past the sizes that pair."""
    src, so = tmp_path / "place.cpp", tmp_path / "place.so"
    src.write_text(PLACE_SHIM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    "-static-libubsan", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "bit_quantized_grouped_router_amd", "csrc"), str(src), "-o", str(so)],
                   check=True)
    h = ctypes.CDLL(str(so))
    h.lost.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    h.lost.restype = ctypes.c_longlong
    seen = ctypes.create_string_buffer(1 << 20)
    shapes = [(n, k) for n in range(1, 513) for k in range(1, 513) if n * k <= 600]
    shapes += [(513, 1), (512, 2), (700, 3), (3, 700), (512, 512), (1000, 1), (1, 1000)]
    for n, heads in shapes:
        for causal in (0, 1):
            for pair in (0, 1):
                assert h.lost(n, heads, causal, pair, seen) == 0, (n, heads, causal, pair)
    # the longest tile is beside the shortest, and they come longest first
    assert [h.tile_of(x, 512, 1) for x in (0, 1, 255, 256, 257, 511)] == [511, 510, 256, 0, 1, 255]
    assert [h.tile_of(x, 300, 1) for x in (0, 43, 256, 299)] == [299, 256, 0, 43]
    assert [h.tile_of(x, 300, 0) for x in (0, 299)] == [299, 0]


def test_replaced_cache_planes_are_checked_by_every_call():
    """The sizes a call passes on are those of the tensors it passes on."""
    import torch

    def plane(pages, heads, page, D):
        g = torch.zeros(pages, heads, page, D // 64, dtype=torch.bfloat16)
        return M.W4Matrix(torch.zeros(pages, heads, page, D // 2, dtype=torch.uint8), g, g.clone())

    dev = [torch.zeros(s, dtype=torch.int32) for s in ((1, 2), (2,), (1,))]
    kv = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    calls = (lambda c: M.moe_kv4_append(c, kv, kv, *dev), lambda c: M.moe_kv4_read(c, *dev, 1),
             lambda c: M.moe_kv4_attention(c, q, *dev, max_new=1))

    def changed():
        for part in ("k", "v"):
            for pages, heads, page, D in ((3, 2, 16, 64), (4, 1, 16, 64), (4, 2, 32, 64), (4, 2, 16, 128)):
                c = M.KV4Cache(plane(4, 2, 16, 64), plane(4, 2, 16, 64))
                setattr(c, part, plane(pages, heads, page, D))
                yield c
            for field, t in (("codes", torch.zeros(3, 2, 16, 32, dtype=torch.uint8)),
                             ("scales", torch.zeros(4, 2, 16, 1)), ("biases", torch.zeros(1, dtype=torch.bfloat16))):
                c = M.KV4Cache(plane(4, 2, 16, 64), plane(4, 2, 16, 64))
                setattr(getattr(c, part), field, t)
                yield c
        c = M.KV4Cache(plane(4, 2, 16, 64), plane(4, 2, 16, 64))
        c.v.codes.resize_(2, 2, 16, 32)
        yield c

    for c in changed():
        for call in calls:
            with pytest.raises(M.MoeError, match="cache"):
                call(c)
    # both planes replaced: their sizes count
    c = M.KV4Cache(plane(4, 2, 16, 64), plane(4, 2, 16, 64))
    c.k, c.v = plane(2, 1, 32, 128), plane(2, 1, 32, 128)
    assert (c.num_pages, c.Hkv, c.page, c.D) == (2, 1, 32, 128) == tuple(c.sizes())
    with pytest.raises(AttributeError):
        c.num_pages = 100


def test_attention_onto_its_queries_keeps_their_stride(L):
    assert attend(L, q=FAKE, out=FAKE, qs=2048, os_=4096) == INVALID
    assert attend(L, q=FAKE, out=FAKE, qs=2056, os_=2048) == INVALID
    assert attend(L, q=FAKE, out=FAKE, qs=4096, os_=4096, ws=FAKE + 8,
                  dm=dims(B=1, page=128, max_pages=1024, num_pages=1024), T=1, max_new=1) == ALIGN  # past that check
    assert attend(L, q=FAKE, out=FAKE, qs=2048, os_=4096, ws=FAKE + 8,
                  dm=dims(B=1, page=128, max_pages=1024, num_pages=1024), T=1, max_new=1) == ALIGN  # one row has no stride


def test_linear_launch_limits(L):
    """Sizes just past the limits that a launch dimension sets."""
    def status(T, rows, xs=64):
        return project(L, T=T, rows=rows, cols=64, xs=xs, ys=rows)

    assert status(16, 2 ** 27 - 143) == UNSUPPORTED               # 2^23 - 8 blocks of 16 rows
    assert status(1, 2 ** 27 - 143) == UNSUPPORTED
    assert status(2 ** 31 - 2175, 16) == UNSUPPORTED
    assert status(32 * 1024, 16 * 8192 - 15, xs=1 << 23) == UNSUPPORTED  # 2^23 blocks
    assert status(2 ** 20, 2 ** 16) == UNSUPPORTED                # T * rows


def test_workspace_of_a_prompt_beside_single_tokens(L):
    """The parts of the few rows are kept for those sequences, not for every row of the prompt."""
    for T, Hq, Hkv, D, B in ((8193, 16, 2, 128, 2), (100001, 16, 2, 128, 2), (32769, 64, 8, 128, 2),
                             (32776, 16, 2, 256, 9), (20300, 32, 1, 64, 300)):
        dm = dims(B=B, Hq=Hq, Hkv=Hkv, D=D, page=128, max_pages=1024, num_pages=1 << 20)
        need = L.moe_kv4_attention_workspace_bytes(ctypes.byref(dm), T, T, 0)
        few = 64 // (Hq // Hkv)   # tokens of a sequence that has few rows
        slots = 2 * 5 * 256       # twice the workgroups that the card holds
        assert need <= B * few * Hq * (D + 2) * 4 * max(1, slots // (B * Hkv * (few * Hq // Hkv // 16))), (T, need)
        assert need < 1 << 28


def test_outputs_onto_what_is_still_read_or_written(L):
    assert project(L, rows=128, ys=128, y=FAKE) == INVALID           # y onto x
    assert project(L, T=1, rows=128, ys=128, y=FAKE, dtype=1) == INVALID
    assert move(L, "moe_kv4_read", k=FAKE, v=FAKE) == INVALID        # keys and values in one place
