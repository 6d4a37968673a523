"""The int4-g64 operators of an attention block together, as a decoder uses them: projection,
cache write, attention, projection onto the fp32 residual stream, then the expert layer. Each
step is held to the fp64 oracle on the inputs the step before it produced; then the same steps
captured in graphs, on other streams and at once."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
import moe_inputs as G
from oracle import kv4_oracle as K
from oracle import moe_oracle as O
from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits
from parity_util import host_bits, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def matrix(rng, rows, cols):
    x = (rng.standard_normal((rows, cols)) * cols ** -0.5).astype(np.float32)
    q, s, b = K.quantise(x)
    dev = lambda a: torch.from_numpy(a.view(np.int16)).cuda().view(BF16)[None]
    return (M.W4Matrix(torch.from_numpy(K.pack(q)).cuda()[None], dev(s), dev(b)), K.weights(K.pack(q), s, b))


class Block:
    """Weights of a small attention block and its cache."""
    d, Hq, Hkv, D, page = 256, 8, 2, 64, 16

    def __init__(self, seed, B, width):
        rng = np.random.default_rng(seed)
        self.rng, self.B = rng, B
        self.wqkv, self.qkv64 = matrix(rng, (self.Hq + 2 * self.Hkv) * self.D, self.d)
        self.wo, self.o64 = matrix(rng, self.d, self.Hq * self.D)
        self.bias = torch.from_numpy(rng.standard_normal(self.qkv64.shape[0])).cuda().to(BF16)
        pages = B * width + 2
        self.cache = M.KV4Cache.empty(pages, self.Hkv, self.page, self.D)
        self.host_table = rng.permutation(pages)[:B * width].reshape(B, width)
        self.table = i32(self.host_table)

    def run(self, x, h, cu, lens, max_new, stream=None, window=0, out=None):
        """(qkv, attention, h + projection) for hidden rows x (bf16) and the residual stream h."""
        qkv = M.moe_linear_w4(x, self.wqkv, bias=self.bias, stream=stream)
        T, n = x.shape[0], self.Hq * self.D
        m = n + self.Hkv * self.D
        heads = lambda t: t.unflatten(1, (-1, self.D))
        M.moe_kv4_append(self.cache, heads(qkv[:, n:m]), heads(qkv[:, m:]), self.table, cu, lens, stream=stream)
        o = M.moe_kv4_attention(self.cache, heads(qkv[:, :n]), self.table, cu, lens, max_new, window=window,
                                stream=stream)
        return qkv, o, M.moe_linear_w4(o.view(T, n), self.wo, residual=h, y=out, stream=stream)


def planes(c):
    return [(m.codes.cpu().numpy(), host_bits(m.scales), host_bits(m.biases)) for m in (c.k, c.v)]


def within(got, want, tol, what):
    off = np.abs(got.double().cpu().numpy() - want)
    say(f"  {what}: worst {float((off / np.maximum(tol, 1e-30)).max()):.3f} of the bound")
    assert (off <= tol).all(), what


def linear_tol(x, w, y, dtype):
    """fp32 sums of x's columns, and the result's rounding."""
    return (x.shape[1] + 8) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T + 4) + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * np.abs(y)


def test_prompt_then_decode_steps():
    blk = Block(1, 3, 24)
    rng, cfg = blk.rng, G.small_config("block", T=1, d=256, f=128, E=16, k=4, seed=5)
    wr = torch.from_numpy(G.make_router(cfg).view(np.int16)).cuda()
    wts_np = G.make_weights(cfg)
    wts = M.W4Weights.from_numpy(wts_np)
    lens = np.zeros(3, dtype=int)
    bias = blk.bias.double().cpu().numpy()
    for new in ([70, 0, 130], [1, 33, 1], [1, 1, 1], [1, 1, 1], [0, 2, 1]):
        lens = lens + new
        cu = [0] + list(np.cumsum(new))
        T = cu[-1]
        h = torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)).cuda()
        x = h.to(BF16)
        qkv, o, y = blk.run(x, h, i32(cu), i32(lens), max(new))
        x64, h64 = x.double().cpu().numpy(), h.double().cpu().numpy()
        want = K.linear(x64, blk.qkv64, bias)
        within(qkv, want, linear_tol(x64, blk.qkv64, want, BF16), "qkv")
        # the cache holds exactly the quantised keys and values
        kv = qkv.float().cpu().numpy()[:, 512:].reshape(T, 2, 2, 64)
        _, pg, sl = K.token_slots(cu, lens, blk.host_table, 16, T)
        host = planes(blk.cache)
        for i, (codes, s, b) in enumerate(host):
            q, ws, wb = K.quantise(np.ascontiguousarray(kv[:, i]))
            assert (codes[pg, :, sl] == K.pack(q)).all() and (s[pg, :, sl] == ws).all() and (b[pg, :, sl] == wb).all()
        q64 = qkv.double().cpu().numpy()[:, :512].reshape(T, 8, 64)
        want, tol = K.attention(q64, K.Paged(*host, blk.host_table), cu, lens, 0.125)
        within(o, want, tol, "attention")
        o64 = o.double().cpu().numpy().reshape(T, 512)
        want = K.linear(o64, blk.o64, residual=h64)
        within(y, want, linear_tol(o64, blk.o64, want, F32) + 2.0 ** -23 * np.abs(h64), "output projection")
        # and on into the expert layer, routed on the GPU's own scores
        xb = y.to(BF16)
        dm = M.dims(T, 256, 128, 16, 4)
        z = M.moe_layer_forward_hidden(dm, xb, wr, wts)
        logits = M.moe_router_logits(xb, wr).cpu().numpy()
        ref = O.layer_forward(host_bits(xb), logits, wts_np, 4, BM=M.moe_block_m())["y"]
        err, rms = np.abs(z.double().cpu().numpy() - ref), np.sqrt((ref ** 2).mean())
        assert err.max() <= 2e-2 * rms and err.mean() <= 2e-3 * rms


@pytest.mark.parametrize("new,past", [([1, 1, 1], [500, 30, 2100]), ([300, 1, 260], [20, 400, 700])])
def test_captured_and_replayed(new, past):
    """A step captured once and replayed with other inputs and lengths, two graphs taking turns,
    eager work and synchronizations in between: every replay as the eager call."""
    width = 200 if max(new) == 1 else 520  # positions enough for the prompts' kernel
    blocks = [Block(s, 3, width) for s in (2, 3)]
    cu = i32([0] + list(np.cumsum(new)))
    T = sum(new)
    rng = np.random.default_rng(4)
    filled = [int(p) for p in past]
    graphs = []
    for blk in blocks:
        n = sum(filled)
        kv = [torch.from_numpy(rng.standard_normal((n, 2, 64))).cuda().to(BF16) for _ in range(2)]
        M.moe_kv4_append(blk.cache, *kv, blk.table, i32([0] + list(np.cumsum(filled))), i32(filled))
        st = dict(x=torch.zeros((T, 256), dtype=BF16, device="cuda"), h=torch.zeros((T, 256), device="cuda"),
                  lens=i32(np.array(past) + new))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                blk.run(st["x"], st["h"], cu, st["lens"], max(new))
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st["out"] = blk.run(st["x"], st["h"], cu, st["lens"], max(new))
        graphs.append((g, st))
    for step in range(4):
        got = []
        for (g, st), blk in zip(graphs, blocks):
            st["x"].copy_(torch.from_numpy(rng.standard_normal((T, 256))))
            st["h"].copy_(torch.from_numpy(rng.standard_normal((T, 256))))
            st["lens"].copy_(i32(np.array(past) + new - np.array([0, step, 3 * step])))
            g.replay()
            if step == 1:
                torch.cuda.synchronize()
            got.append([t.clone() for t in st["out"]])
        torch.randn(1 << 20, device="cuda").sort()
        if step == 2:
            torch.cuda.synchronize()
        for (g, st), blk, a in zip(graphs, blocks, got):
            b = blk.run(st["x"], st["h"], cu, st["lens"], max(new))
            assert all(torch.equal(s, t) for s, t in zip(a, b)), step
            assert torch.isfinite(a[2]).all()


def test_two_calls_at_once_on_other_streams():
    """Two blocks on two streams, given as argument and as current stream, with split keys (each
    call its own workspace), against the same calls one after the other."""
    blocks = [Block(s, 4, 200) for s in (6, 7)]
    rng = np.random.default_rng(8)
    new, past = [1, 1, 2, 1], [3100, 900, 40, 2500]
    cu, lens = i32([0] + list(np.cumsum(new))), i32(np.array(past) + new)
    args = []
    for blk in blocks:
        kv = [torch.from_numpy(rng.standard_normal((sum(past), 2, 64))).cuda().to(BF16) for _ in range(2)]
        M.moe_kv4_append(blk.cache, *kv, blk.table, i32([0] + list(np.cumsum(past))), i32(past))
        h = torch.from_numpy(rng.standard_normal((5, 256)).astype(np.float32)).cuda()
        args.append((h.to(BF16), h, cu, lens, 2))
    want = [blk.run(*a) for blk, a in zip(blocks, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            if i == 0:
                got[i].append(blocks[i].run(*args[i], stream=streams[i]))
            else:
                with torch.cuda.stream(streams[i]):
                    got[i].append(blocks[i].run(*args[i]))
    for s in streams:
        s.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_own_workspace_is_enough_and_checked():
    blk = Block(9, 2, 260)
    rng = np.random.default_rng(10)
    past = [3000, 1700]
    kv = [torch.from_numpy(rng.standard_normal((sum(past), 2, 64))).cuda().to(BF16) for _ in range(2)]
    M.moe_kv4_append(blk.cache, *kv, blk.table, i32([0, 3000, 4700]), i32(past))
    for new in ([1, 1], [600, 500]):
        T = sum(new)
        q = torch.from_numpy(rng.standard_normal((T, 8, 64))).cuda().to(BF16)
        cu = i32([0, new[0], T])
        need = M.moe_kv4_attention_workspace_bytes(blk.cache, T, 8, 2, 260, max(new))
        want = M.moe_kv4_attention(blk.cache, q, blk.table, cu, i32(past), max(new))
        ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        got = M.moe_kv4_attention(blk.cache, q, blk.table, cu, i32(past), max(new), ws=ws[:need])
        assert torch.equal(got, want) and (ws[need:] == 0xA5).all()
        assert need > 0
        with pytest.raises(M.MoeError):
            M.moe_kv4_attention(blk.cache, q, blk.table, cu, i32(past), max(new), ws=ws[:need - 1])
