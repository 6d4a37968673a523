"""The steps of a decoder layer together, as a server uses them: the residual's addition and norm,
the projection, rotated write, page bounds, attention over selected pages, projection onto the
residual stream, norm, experts. Each step is held to the fp64 oracle on the inputs the step before
it produced; then the same steps captured in graphs, on other streams and at once."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
import moe_inputs as G
from oracle import block_oracle as B
from oracle import kv4_oracle as K
from oracle import moe_oracle as O
from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits
from parity_util import host_bits
from test_gpu_attention_block import i32, linear_tol, matrix, planes, within
from test_gpu_sparse import expected

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


class Layer:
    """Weights of a small layer's attention half, its cache and its pages' bounds."""
    d, Hq, Hkv, D, page, rot = 256, 8, 2, 64, 16, 32
    pages = dict(top=4, first=1, recent=2)

    def __init__(self, seed, batch, width):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.wqkv, self.qkv64 = matrix(rng, (self.Hq + 2 * self.Hkv) * self.D, self.d)
        self.wo, self.o64 = matrix(rng, self.d, self.Hq * self.D)
        norm = lambda n: torch.from_numpy(1 + 0.2 * rng.standard_normal(n)).cuda().to(BF16)
        self.w1, self.w2, self.qw, self.kw = norm(self.d), norm(self.d), norm(self.D), norm(self.D)
        n = batch * width + 2
        self.cache = M.KV4Cache.empty(n, self.Hkv, self.page, self.D)
        self.bounds = torch.full((n, self.Hkv, 2, self.D), float("nan"), dtype=BF16, device="cuda")
        self.host_table = rng.permutation(n)[:batch * width].reshape(batch, width)
        self.table = i32(self.host_table)
        self.rope = M.Rope.make(self.rot, scaling="ramp", factor=4.0, trained=512)

    def run(self, y, h, cu, lens, max_new, stream=None):
        """(x, h, qkv as projected, q, attention, h after it, x after it) for the step before's output y
        and the residual stream h."""
        T, n = y.shape[0], self.Hq * self.D
        m = n + self.Hkv * self.D
        heads = lambda t: t.unflatten(1, (-1, self.D))
        kw = dict(stream=stream)
        x, h = M.moe_rmsnorm(y, self.w1, residual=h, **kw)
        qkv = M.moe_linear_w4(x, self.wqkv, **kw)
        batch = (self.table, cu, lens)
        q = M.moe_kv4_rope_append(self.cache, heads(qkv[:, :n]), heads(qkv[:, n:m]), heads(qkv[:, m:]), self.rope, *batch,
                                  q_weight=self.qw, k_weight=self.kw, **kw)
        M.moe_kv4_bounds(self.cache, self.bounds, *batch, T, **kw)
        o = M.moe_kv4_sparse_attention(self.cache, self.bounds, q, *batch, max_new, **self.pages, **kw)
        h2 = M.moe_linear_w4(o.view(T, n), self.wo, residual=h, **kw)
        return x, h, qkv, q, o, h2, M.moe_rmsnorm(h2, self.w2, plus_one=True, **kw)

    def fill(self, past):
        n = sum(past)
        x = torch.from_numpy(self.rng.standard_normal((n, self.Hq + 2 * self.Hkv, self.D))).cuda().to(BF16)
        batch = (self.table, i32([0] + list(np.cumsum(past))), i32(past))
        M.moe_kv4_rope_append(self.cache, x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:],
                              self.rope, *batch, k_weight=self.kw)
        M.moe_kv4_bounds(self.cache, self.bounds, *batch, n)


def f64(t):
    return t.double().cpu().numpy()


def normed(got, x64, w64, what, residual=None):
    want, s = B.rmsnorm(x64, w64, 1e-6, residual)
    within(got, want, np.abs(want) * (B.norm_terms(x64.shape[1]) * U + 2.0 ** -8), what)
    return s


def test_prompt_then_decode_and_drafts():
    lay = Layer(1, 3, 24)
    cfg = G.small_config("layer", T=1, d=256, f=128, E=16, k=4, seed=5)
    wr = torch.from_numpy(G.make_router(cfg).view(np.int16)).cuda()
    wts_np = G.make_weights(cfg)
    wts = M.W4Weights.from_numpy(wts_np)
    lens = np.zeros(3, dtype=int)
    # prompts, single tokens, then three drafts of which two are rejected and others take their place
    for new, back in [([70, 0, 130], 0), ([1, 33, 1], 0), ([1, 1, 1], 0), ([3, 3, 3], 0), ([1, 1, 1], 2), ([0, 2, 1], 0)]:
        lens = lens - back + new
        cu = [0] + list(np.cumsum(new))
        T = cu[-1]
        y = torch.from_numpy(lay.rng.standard_normal((T, 256)).astype(np.float32)).cuda()
        h0 = torch.from_numpy(3 * lay.rng.standard_normal((T, 256)).astype(np.float32)).cuda()
        x, h, qkv, q, o, h2, x2 = lay.run(y, h0, i32(cu), i32(lens), max(new))
        s = normed(x, f64(y), f64(lay.w1), "input norm", f64(h0))
        within(h, s, np.abs(s) * U, "residual")
        want = K.linear(f64(x), lay.qkv64)
        within(qkv, want, linear_tol(f64(x), lay.qkv64, want, BF16), "qkv")
        # rotated queries, and keys as the cache holds them: exactly those of the turned heads in fp32
        heads = qkv.unflatten(1, (-1, 64))
        at = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)])
        assert torch.equal(q, M.moe_rope(heads[:, :8], lay.rope, i32(at), weight=lay.qw))
        keys = M.moe_rope(heads[:, 8:10], lay.rope, i32(at), weight=lay.kw, out_dtype=F32)
        k64, size = B.rope(B.rmsnorm(f64(heads[:, 8:10]), f64(lay.kw), 1e-6)[0], at, f64(lay.rope.freqs), False,
                           lay.rope.magnitude)
        within(keys, k64, 80 * U * (size + np.abs(k64)), "keys")
        _, pg, sl = K.token_slots(cu, lens, lay.host_table, 16, T)
        host = planes(lay.cache)
        for t, (codes, sc, bi) in zip((keys, heads[:, 10:].float()), host):
            cq, ws, wb = K.quantise(np.ascontiguousarray(t.cpu().numpy()))
            assert (codes[pg, :, sl] == K.pack(cq)).all() and (sc[pg, :, sl] == ws).all() and (bi[pg, :, sl] == wb).all()
        # bounds of every page that attention may read, then attention over the oracle's own selection
        with np.errstate(over="ignore", invalid="ignore"):  # pages that nothing was written to hold anything
            kv = bf16_to_f64(round_to_bf16_bits(K.values(*host[0]).astype(np.float32).astype(np.float64)))
        bb = bf16_to_f64(host_bits(lay.bounds))
        for b in range(3):
            if new[b]:
                for c in range((lens[b] - 1) // 16 + 1):
                    p = lay.host_table[b, c]
                    for hd in range(2):
                        assert (bb[p, hd] == B.bounds(kv[p:p + 1, hd], lens[b] - 16 * c)[0]).all()
        want, tol, _, done = expected(f64(q), lay.cache, lay.bounds, lay.host_table, cu, lens, T, **lay.pages)
        assert done.all()
        within(o, want, tol, "attention")
        o64 = f64(o).reshape(T, 512)
        want = K.linear(o64, lay.o64, residual=f64(h))
        within(h2, want, linear_tol(o64, lay.o64, want, F32) + 2.0 ** -23 * np.abs(f64(h)), "output projection")
        normed(x2, f64(h2), f64(lay.w2) + 1, "norm after attention")
        dm = M.dims(T, 256, 128, 16, 4)
        z = M.moe_layer_forward_hidden(dm, x2, wr, wts)
        ref = O.layer_forward(host_bits(x2), M.moe_router_logits(x2, wr).cpu().numpy(), wts_np, 4, BM=M.moe_block_m())["y"]
        err, rms = np.abs(f64(z) - ref), np.sqrt((ref ** 2).mean())
        assert err.max() <= 2e-2 * rms and err.mean() <= 2e-3 * rms
        # and onto the residual stream, in place, for the next layer
        hh = h2.clone()
        xn, back_h = M.moe_rmsnorm(z, lay.w1, residual=hh, h=hh)
        assert back_h is hh
        s = normed(xn, f64(z), f64(lay.w1), "next norm", f64(h2))
        within(hh, s, np.abs(s) * U, "next residual")


def steps(past, new):
    return [0] + list(np.cumsum(new)), np.array(past) + new


@pytest.mark.parametrize("new,past", [([1, 1, 1], [500, 30, 2100]), ([200, 1, 160], [20, 400, 700])])
def test_captured_and_replayed(new, past):
    """A step captured once and replayed with other inputs and lengths, two graphs taking turns,
    eager work and synchronizations in between: every replay as the eager call."""
    cu, lens = steps(past, new)
    T = cu[-1]
    rng = np.random.default_rng(4)
    layers, graphs = [Layer(s, 3, 160) for s in (2, 3)], []
    cu = i32(cu)
    for lay in layers:
        lay.fill(past)
        st = dict(y=torch.zeros((T, 256), device="cuda"), h=torch.zeros((T, 256), device="cuda"), lens=i32(lens))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                lay.run(st["y"], st["h"], cu, st["lens"], max(new))
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st["out"] = lay.run(st["y"], st["h"], cu, st["lens"], max(new))
        graphs.append((g, st))
    for step in range(4):
        got = []
        for (g, st), lay in zip(graphs, layers):
            st["y"].copy_(torch.from_numpy(rng.standard_normal((T, 256))))
            st["h"].copy_(torch.from_numpy(rng.standard_normal((T, 256))))
            st["lens"].copy_(i32(lens - np.array([0, step, 3 * step])))
            g.replay()
            if step == 1:
                torch.cuda.synchronize()
            got.append([t.clone() for t in st["out"]])
        torch.randn(1 << 20, device="cuda").sort()
        if step == 2:
            torch.cuda.synchronize()
        for (g, st), lay, a in zip(graphs, layers, got):
            b = lay.run(st["y"], st["h"], cu, st["lens"], max(new))
            assert all(torch.equal(s, t) for s, t in zip(a, b)), step
            assert torch.isfinite(a[-1]).all()


def test_two_calls_at_once_on_other_streams():
    """Two layers on two streams, given as argument and as current stream, each call with its own
    workspace, against the same calls one after the other."""
    past, new = [3000, 900, 40, 1500], [1, 1, 2, 1]
    cu, lens = steps(past, new)
    layers = [Layer(s, 4, 200) for s in (6, 7)]
    rng = np.random.default_rng(8)
    args = []
    for lay in layers:
        lay.fill(past)
        y, h = (torch.from_numpy(rng.standard_normal((5, 256)).astype(np.float32)).cuda() for _ in range(2))
        args.append((y, h, i32(cu), i32(lens), 2))
    want = [lay.run(*a) for lay, a in zip(layers, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        got[0].append(layers[0].run(*args[0], stream=streams[0]))
        with torch.cuda.stream(streams[1]):
            got[1].append(layers[1].run(*args[1]))
    for s in streams:
        s.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_own_workspace_is_enough_and_checked():
    lay = Layer(9, 2, 260)
    past = [3000, 1700]
    lay.fill(past)
    for new in ([1, 1], [300, 200]):
        T = sum(new)
        q = torch.from_numpy(lay.rng.standard_normal((T, 8, 64))).cuda().to(BF16)
        args = (lay.cache, lay.bounds, q, lay.table, i32([0, new[0], T]), i32(past), max(new))
        need = M.moe_kv4_sparse_attention_workspace_bytes(lay.cache, T, 8, 2, 260, max(new), **lay.pages)
        want = M.moe_kv4_sparse_attention(*args, **lay.pages)
        for fill in (0xA5, 0xFF, 0):
            ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
            got = M.moe_kv4_sparse_attention(*args, **lay.pages, ws=ws[:need])
            assert torch.equal(got, want) and (ws[need:] == fill).all()
        with pytest.raises(M.MoeError):
            M.moe_kv4_sparse_attention(*args, **lay.pages, ws=ws[:need - 1])
