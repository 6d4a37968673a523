"""What a decoder layer needs around the int4-g64 operators it already has: what is measured.

Five operators:
  norm    root-mean-square norm of hidden rows, with the residual's addition before it, to bf16, fp32 or
          8 bits (e4m3 or int8) with a scale for each row or group of a row;
  rope    rotary positions on the heads of a projection, both layouts, part of a head, with the heads' own
          norm, frequencies scaled for long contexts;
  write   the same on queries and keys, the keys quantised into the paged int4-g64 cache in the same pass
          and the values beside them, then the cache's rows read back;
  bounds  per page and cache head the smallest and largest key of each channel, brought up to date for the
          pages that new tokens lie in;
  sparse  attention of each new token over the cache pages that a score from those bounds selects for it.

A case names one operator and its sizes. With ``own`` false, run() computes it with elementary torch
operations in 32 bits (64 for angles and for the scores that a selection goes by); with ``own`` true it
calls the framework. exact() is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the expert layer's output of one decode token, added to the fp32 residual stream, for the next block
        dict(name="norm, 1 token", op="norm", T=1, d=2048, x="f32", r="f32", out="bf16", group=0, plus_one=True),
        # rows sent on in 8 bits with a scale for each 128 channels, odd number of tokens
        dict(name="norm, 777 tokens, e4m3", op="norm", T=777, d=5120, x="bf16", r="bf16", out="e4m3", group=128,
             plus_one=False),
        # a prompt's rows between attention and the expert layer
        dict(name="norm, 8192 tokens", op="norm", T=8192, d=2048, x="f32", r="f32", out="bf16", group=0,
             plus_one=False),
        # query heads of a decode batch: a quarter of each head rotated, heads normed first
        dict(name="rope, 64 tokens, part", op="rope", T=64, H=16, D=256, rot=64, interleaved=False, norm=True,
             scaled=False, x="bf16", out="bf16"),
        # query heads of a long prompt, neighbouring channels paired, scaled frequencies
        dict(name="rope, 8192 tokens", op="rope", T=8192, H=16, D=128, rot=128, interleaved=True, norm=False,
             scaled=True, x="bf16", out="bf16"),
        # one new token for each of 8 sequences, from the fused projection
        dict(name="rotated write, 8 tokens", op="write", B=8, new=1, past=700, spread=0, Hq=16, Hkv=2, D=256,
             page=64, rot=64, interleaved=False, norm=True, x="bf16"),
        # several requests' prompts, fp32 projections, whole heads rotated
        dict(name="rotated write, prompts", op="write", B=7, new=1500, past=100, spread=3, Hq=32, Hkv=8, D=128,
             page=16, rot=128, interleaved=False, norm=False, x="f32"),
        # decode step of 64 sequences: one page each to bring up to date
        dict(name="bounds, 64 tokens", op="bounds", B=64, new=1, past=8100, spread=5, Hkv=2, D=256, page=64),
        # after a long prompt: every page of it
        dict(name="bounds, prompt", op="bounds", B=1, new=60000, past=1003, spread=0, Hkv=2, D=128, page=64),
        # one very long context at batch 1, 2048 of its keys
        dict(name="sparse, 1 x 128K", op="sparse", B=1, new=1, past=131149, spread=0, Hq=16, Hkv=2, D=128,
             page=64, top=29, first=1, recent=2),
        # a serving batch of long mixed contexts
        dict(name="sparse, 64 mixed", op="sparse", B=64, new=1, past=32000, spread=5, Hq=16, Hkv=2, D=256,
             page=64, top=20, first=1, recent=3),
        # a prompt chunk behind a long context, each token with its own pages
        dict(name="sparse, prompt of 1500", op="sparse", B=1, new=1500, past=60000, spread=0, Hq=16, Hkv=2,
             D=128, page=32, top=28, first=1, recent=3),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(max(w["bytes"], w["flops"] / 50) for w in map(work, listed()))
    while True:
        op = rng.choice(["norm", "rope", "write", "bounds", "sparse", "sparse"])
        if op == "norm":
            c = dict(op=op, T=log_int(rng, 1, 8192), x=rng.choice(["bf16", "f32"]),
                     r=rng.choice(["", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32", "e4m3", "int8"]),
                     group=0, plus_one=rng.random() < 0.5)
            c["d"] = 64 * log_int(rng, 1, 100) if rng.random() < 0.7 else log_int(rng, 33, 6001)
            if c["out"] in ("e4m3", "int8") and c["d"] % 128 == 0:
                c["group"] = rng.choice([0, 64, 128])
        elif op == "rope":
            c = dict(op=op, T=log_int(rng, 1, 8192), H=log_int(rng, 1, 64), D=8 * log_int(rng, 4, 32),
                     interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, scaled=rng.random() < 0.5,
                     x=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
            c["rot"] = c["D"] if rng.random() < 0.5 else 2 * rng.randint(1, c["D"] // 2)
        else:
            c = dict(op=op, B=log_int(rng, 1, 64), new=1, past=log_int(rng, 1, 5000), spread=rng.randint(0, 50),
                     Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]),
                     page=rng.choice([16, 32, 64, 128]))
            if op == "write":
                c.update(new=log_int(rng, 1, 3000), Hq=c["Hkv"] * rng.choice([1, 2, 3, 4, 8]),
                         interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, x=rng.choice(["bf16", "f32"]))
                c["rot"] = c["D"] if rng.random() < 0.5 else 2 * rng.randint(1, c["D"] // 2)
            elif op == "bounds":
                c.update(new=log_int(rng, 1, 9000))
            else:
                c.update(Hq=c["Hkv"] * rng.choice([1, 2, 3, 4, 8, 12]), past=log_int(rng, 100, 120000),
                         new=rng.choice([1, 1, 2, 5, log_int(rng, 8, 1500)]), top=rng.randint(0, 40),
                         first=rng.randint(0, 3), recent=rng.randint(1, 4))
                if keys_read(c) * c["Hkv"] * c["D"] > 900_000_000:
                    continue  # the plain form's keys
                if c["B"] * c["new"] * c["Hkv"] * (c["new"] + c["past"]) / c["page"] > 30_000_000:
                    continue  # the plain form's scores
        if op in ("write", "bounds", "sparse") and c["B"] * (c["new"] + c["past"]) * c["Hkv"] * c["D"] > 600_000_000:
            continue  # the cache, when it is made
        w = work(c)
        if max(w["bytes"], w["flops"] / 50) <= top:
            return c


def lengths(case):
    """(new tokens, all tokens) of each sequence; ragged where spread is not 0."""
    B, new, past = case["B"], case["new"], case["past"]
    if not case["spread"]:
        return [new] * B, [new + past] * B
    r = random.Random(case["spread"])
    some = [new if new == 1 or i == 0 else r.randint(new // 4, new) for i in range(B)]
    old = [past if i == 0 else int(past * math.exp(-r.uniform(0.0, 2.7))) for i in range(B)]
    return some, [n + o for n, o in zip(some, old)]


def pages_taken(case, pos):
    """Pages that a token at each of positions pos attends to."""
    own_page = pos // case["page"]
    free = np.maximum(own_page - case["recent"] + 1 - case["first"], 0)  # pages that are scored
    return own_page + 1 - free + np.minimum(free, case["top"])


def keys_read(case):
    """Keys in the pages of all tokens of a case, summed (of one cache head)."""
    return sum(int(pages_taken(case, np.arange(t - n, t)).sum()) for n, t in zip(*lengths(case))) * case["page"]


SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "int8": 1}


def work(case):
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        n = T * d * (SIZE[case["x"]] + SIZE[case["out"]] + (2 * SIZE[case["r"]] if case["r"] else 0)) + 2 * d
        if case["out"] in ("e4m3", "int8"):
            n += T * (d // case["group"] if case["group"] else 1) * 4
        return {"bytes": n, "flops": 6.0 * T * d}
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["out"]]) + 4 * case["T"] + 2 * case["rot"],
                "flops": 3.0 * n}
    new, total = lengths(case)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if case["op"] == "write":  # read the projection, write queries and cache, read the cache, write its values
        q, kv = sum(new) * case["Hq"] * D, sum(new) * Hkv * D * 2
        return {"bytes": q * (SIZE[case["x"]] + 2) + kv * (SIZE[case["x"]] + 2 * 0.5625 + 2),
                "flops": 3.0 * q + 8.0 * kv}
    if case["op"] == "bounds":  # the pages' keys and the two bounds of each channel
        keys = sum(t - (t - n) // page * page for n, t in zip(new, total) if n)
        pages = sum((t - 1) // page - (t - n) // page + 1 for n, t in zip(new, total) if n)
        return {"bytes": keys * Hkv * D * 0.5625 + pages * Hkv * D * 4, "flops": 4.0 * keys * Hkv * D}
    byt = flo = 0.0
    for n, t in zip(new, total):
        pos = np.arange(t - n, t)
        scored = np.maximum(pos // page - case["recent"] + 1 - case["first"], 0)
        taken = pages_taken(case, pos)
        # a sequence's bounds and pages once, however many of its tokens read them
        byt += int(scored.max(initial=0)) * Hkv * D * 4 + min(int(taken.sum()), (t - 1) // page + 1) * page * Hkv * D * 2 * 0.5625
        byt += n * case["Hq"] * D * 4 + n * Hkv * (case["top"] + case["first"] + case["recent"]) * 4
        flo += int(scored.sum()) * Hkv * D * 4.0 + int(taken.sum()) * page * case["Hq"] * D * 4.0
    return {"bytes": byt, "flops": flo}


# ------------------------------------------------------------------ inputs

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def quantise(x):
    """Codes (one value each), scales and biases of groups of 64 along the last axis."""
    x = x.float()
    g = x.view(*x.shape[:-1], -1, GROUP)
    lo, hi = g.amin(-1), g.amax(-1)
    b = lo.to(torch.bfloat16)
    span = hi - b.float()
    s = (span * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).to(torch.bfloat16)
    s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
    t = (g - b.float()[..., None]).double()
    d = s.double()[..., None]
    q = torch.where(d > 0, torch.round(t / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(t))
    return q.clamp(0, 15).to(torch.uint8).view(x.shape), s, b


def packed(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def unpacked(codes, scales, biases):
    """scale * code + bias in 32 bits along the last axis."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).float().view(*codes.shape[:-1], -1, GROUP)
    return (scales.float()[..., None] * q + biases.float()[..., None]).view(*codes.shape[:-1], -1)


def plane(pages, Hkv, page, D, gen, drift):
    """Keys or values of whole pages, quantised from seeded values, some pages at a time. drift: how far a
    page's values lie from the others', as neighbouring tokens' keys do."""
    c = {"codes": torch.empty((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda"),
         "scales": torch.empty((pages, Hkv, page, D // GROUP), dtype=torch.bfloat16, device="cuda"),
         "biases": torch.empty((pages, Hkv, page, D // GROUP), dtype=torch.bfloat16, device="cuda")}
    step = max(1, (1 << 25) // (Hkv * page * D))
    for i in range(0, pages, step):
        m = min(step, pages - i)
        x = torch.randn((m, Hkv, page, D), generator=gen, device="cuda")
        if drift:
            x += drift * torch.randn((m, Hkv, 1, D), generator=gen, device="cuda")
        q, c["scales"][i:i + m], c["biases"][i:i + m] = quantise(x.to(torch.bfloat16))
        c["codes"][i:i + m] = packed(q)
    return c


def all_bounds(c):
    """The smallest and largest key of every channel, [pages, Hkv, 2, D], of pages that are full."""
    pages, Hkv, page, half = c["codes"].shape
    out = torch.empty((pages, Hkv, 2, 2 * half), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 25) // (Hkv * page * half))
    for i in range(0, pages, step):
        x = unpacked(*(c[f][i:i + step] for f in ("codes", "scales", "biases"))).to(torch.bfloat16)
        out[i:i + step, :, 0], out[i:i + step, :, 1] = x.amin(2), x.amax(2)
    return out


def frequencies(rot, scaled):
    """Radians a position for each pair; scaled: the slow ones stretched by 8, the fast ones left, between
    them a ramp over the turns that a pair makes in 8192 positions."""
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaled:
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
        f = f * keep + f / 8.0 * (1.0 - keep)
    return torch.tensor(f, dtype=torch.float32, device="cuda"), (0.1 * math.log(8.0) + 1.0 if scaled else 1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    weight = lambda n: (1.0 + 0.1 * normal(n)).to(torch.bfloat16)
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        st["x_"] = normal(T, d).to(TYPES[case["x"]])
        st["r_"] = (4.0 * normal(T, d)).to(TYPES[case["r"]]) if case["r"] else None
        st["w"] = (0.1 * normal(d)).to(torch.bfloat16) if case["plus_one"] else weight(d)
        return st
    if "rot" in case:
        st["freqs"], st["magnitude"] = frequencies(case["rot"], case.get("scaled", False))
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        st["x_"] = normal(T, H, D).to(TYPES[case["x"]])
        st["pos"] = torch.randint(0, 131072, (T,), generator=gen, device="cuda", dtype=torch.int32)
        st["w"] = weight(D) if case["norm"] else None
        return st
    new, total = lengths(case)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    T = sum(new)
    width = max(-(-t // page) for t in total)
    pages = B * width + 3
    st["table"] = torch.randperm(pages, generator=gen, device="cuda")[:B * width].view(B, width).int()
    st["cu"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()
    st["len"] = torch.tensor(total, dtype=torch.int32).cuda()
    st["T"], st["max_new"] = T, max(new)
    if case["op"] == "write":
        for name in ("k", "v"):
            st[name + "_cache"] = {
                "codes": torch.zeros((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda"),
                "scales": torch.zeros((pages, Hkv, page, D // GROUP), dtype=torch.bfloat16, device="cuda"),
                "biases": torch.zeros((pages, Hkv, page, D // GROUP), dtype=torch.bfloat16, device="cuda")}
        st["qkv"] = normal(T, case["Hq"] + 2 * Hkv, D).to(TYPES[case["x"]])  # as one projection leaves them
        st["qw"], st["kw"] = (weight(D), weight(D)) if case["norm"] else (None, None)
        return st
    st["k_cache"] = plane(pages, Hkv, page, D, gen, drift=0.7)
    if case["op"] == "bounds":
        st["v_cache"] = st["k_cache"]  # not read
        st["bounds"] = normal(pages, Hkv, 2, D).to(torch.bfloat16)
        return st
    st["v_cache"] = plane(pages, Hkv, page, D, gen, drift=0.0)
    st["bounds"] = all_bounds(st["k_cache"])
    st["q"] = normal(T, case["Hq"], D).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return run_own(st)
    return {"norm": plain_norm, "rope": plain_rope, "write": plain_write, "bounds": plain_bounds,
            "sparse": plain_sparse}[st["op"]](st)


def run_own(st):
    import bit_quantized_grouped_router_amd as M
    if st["op"] == "norm":
        got = M.moe_rmsnorm(st["x_"], st["w"], eps=EPS, residual=st["r_"], plus_one=st["plus_one"],
                            out_dtype=TYPES[st["out"]], group=st["group"])
        return in_bf16(st, got) if st["out"] in LARGEST else got
    if "rot" in st:
        rope = M.Rope(st["freqs"], interleaved=st["interleaved"], magnitude=st["magnitude"])
    if st["op"] == "rope":
        return M.moe_rope(st["x_"], rope, st["pos"], weight=st["w"], eps=EPS, out_dtype=TYPES[st["out"]])
    k, v = st["k_cache"], st["v_cache"]
    cache = M.KV4Cache(M.W4Matrix(k["codes"], k["scales"], k["biases"]),
                       M.W4Matrix(v["codes"], v["scales"], v["biases"]))
    batch = (st["table"], st["cu"], st["len"])
    if st["op"] == "write":
        Hq, m, qkv = st["Hq"], st["Hq"] + st["Hkv"], st["qkv"]
        q = M.moe_kv4_rope_append(cache, qkv[:, :Hq], qkv[:, Hq:m], qkv[:, m:], rope, *batch, q_weight=st["qw"],
                                  k_weight=st["kw"], eps=EPS)
        return (q, *M.moe_kv4_read(cache, *batch, st["T"]))
    if st["op"] == "bounds":
        M.moe_kv4_bounds(cache, st["bounds"], *batch, st["T"])
        return st["bounds"]
    blocks = torch.empty((st["T"], st["Hkv"], st["top"] + st["first"] + st["recent"]), dtype=torch.int32, device="cuda")
    out = M.moe_kv4_sparse_attention(cache, st["bounds"], st["q"], *batch, max_new=st["max_new"], top=st["top"],
                                     first=st["first"], recent=st["recent"], blocks=blocks)
    return out, blocks


def in_bf16(st, got):
    """The values that an 8-bit result stands for, in bf16, its scales, and the sum that was normed."""
    q, scales = got[0].float(), got[1]
    v = (q.view(st["T"], scales.shape[1], -1) * scales[..., None]).view(st["T"], st["d"]).to(torch.bfloat16)
    return (v, scales, *got[2:])


def plain_norm(st):
    s = st["x_"].float()
    if st["r_"] is not None:
        s = s + st["r_"].float()
    w = st["w"].float() + 1.0 if st["plus_one"] else st["w"].float()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * w
    h = () if st["r_"] is None else (s.to(TYPES[st["r"]]),)
    if st["out"] not in LARGEST:
        y = y.to(TYPES[st["out"]])
        return (y, *h) if h else y
    g = y.view(st["T"], -1, st["group"] or st["d"])
    scales = g.abs().amax(-1) / LARGEST[st["out"]]
    t = (g / scales[..., None]).clamp(-LARGEST[st["out"]], LARGEST[st["out"]]).view(y.shape)
    return in_bf16(st, ((torch.round(t) if st["out"] == "int8" else t).to(TYPES[st["out"]]), scales, *h))


def normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def rotated(st, x, pos):
    """x [T, H, D] in 32 bits, its first rot channels turned."""
    rot = st["rot"]
    angle = pos.double()[:, None] * st["freqs"].double()
    c = (torch.cos(angle) * st["magnitude"]).float()[:, None]
    s = (torch.sin(angle) * st["magnitude"]).float()[:, None]
    p = x[..., :rot]
    a, b = (p[..., 0::2], p[..., 1::2]) if st["interleaved"] else (p[..., :rot // 2], p[..., rot // 2:])
    a, b = a * c - b * s, a * s + b * c
    p = torch.stack([a, b], dim=-1).flatten(-2) if st["interleaved"] else torch.cat([a, b], dim=-1)
    return torch.cat([p, x[..., rot:]], dim=-1)


def plain_rope(st):
    return rotated(st, normed(st["x_"], st["w"]), st["pos"]).to(TYPES[st["out"]])


def places(st):
    """Sequence and position of every new token."""
    tok = torch.arange(st["T"], device="cuda")
    cu, length = st["cu"].long(), st["len"].long()
    b = torch.searchsorted(cu[1:], tok, right=True)
    return b, length[b] - cu[b + 1] + tok


def plain_write(st):
    b, pos = places(st)
    page, slot = st["table"].long()[b, pos // st["page"]], pos % st["page"]
    Hq, m = st["Hq"], st["Hq"] + st["Hkv"]
    q = rotated(st, normed(st["qkv"][:, :Hq], st["qw"]), pos).to(torch.bfloat16)
    k = rotated(st, normed(st["qkv"][:, Hq:m], st["kw"]), pos)
    out = [q]
    for c, x in ((st["k_cache"], k), (st["v_cache"], st["qkv"][:, m:].float())):
        codes, s, bias = quantise(x.contiguous())
        c["codes"][page, :, slot], c["scales"][page, :, slot], c["biases"][page, :, slot] = packed(codes), s, bias
        out.append(unpacked(*(c[f][page, :, slot] for f in ("codes", "scales", "biases"))).to(torch.bfloat16))
    return tuple(out)


def plain_bounds(st):
    b, pos = places(st)
    page = st["page"]
    lead = (pos % page == 0) | (pos == (st["len"].long() - st["cu"][1:].long() + st["cu"][:-1].long())[b])
    b, block = b[lead], pos[lead] // page
    at = st["table"].long()[b, block]
    c = st["k_cache"]
    x = unpacked(*(c[f][at] for f in ("codes", "scales", "biases"))).to(torch.bfloat16)  # [n, Hkv, page, D]
    there = (block[:, None] * page + torch.arange(page, device="cuda") < st["len"].long()[b][:, None])[:, None, :, None]
    inf = torch.tensor(float("inf"), dtype=torch.bfloat16, device="cuda")
    st["bounds"][at, :, 0] = torch.where(there, x, inf).amin(2)
    st["bounds"][at, :, 1] = torch.where(there, x, -inf).amax(2)
    return st["bounds"]


def plain_sparse(st):
    B, Hq, Hkv, D, page, n = st["B"], st["Hq"], st["Hkv"], st["D"], st["page"], st["max_new"]
    G, W, T = Hq // Hkv, st["table"].shape[1], st["T"]
    cu, length = st["cu"].long(), st["len"].long()
    # scores of every page for queries padded to n a sequence, in 64 bits: they decide a selection
    i = torch.arange(n, device="cuda")
    real = i[None] < (cu[1:] - cu[:-1])[:, None]
    row = (cu[:-1, None] + i[None]).clamp(max=T - 1)
    q = st["q"].double()[row].view(B, n, Hkv, G, D)
    q = torch.cat([q.clamp(max=0).sum(3), q.clamp(min=0).sum(3)], dim=-1).permute(0, 2, 1, 3).contiguous()
    bound = st["bounds"][st["table"].long()].double()  # [B, W, Hkv, 2, D]
    score = torch.matmul(q, bound.permute(0, 2, 3, 4, 1).reshape(B, Hkv, 2 * D, W).contiguous())
    score = score.permute(0, 2, 1, 3)[real].float()  # [T, Hkv, W]
    b, pos = places(st)
    c = torch.arange(W, device="cuda")
    mine = (pos // page)[:, None]
    scored = (c >= st["first"]) & (c <= mine - st["recent"])
    score = score.masked_fill(~scored[:, None], float("-inf"))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :st["top"]]
    taken = torch.zeros_like(score, dtype=torch.bool).scatter(-1, best, True) & scored[:, None]
    taken = taken | ((c <= mine) & ~scored)[:, None]
    # their numbers in ascending order, -1 behind them
    blocks = torch.sort(torch.where(taken, c, W), dim=-1).values
    size = st["top"] + st["first"] + st["recent"]
    blocks = torch.cat([blocks, torch.full((T, Hkv, size), W, device="cuda")], dim=-1)[..., :size]
    blocks = torch.where(blocks < W, blocks, -1)
    # attention over those pages
    at = st["table"].long()[b[:, None, None], blocks.clamp(min=0)]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    k, v = (unpacked(*(st[name][f][at, head] for f in ("codes", "scales", "biases"))).view(T, Hkv, -1, D)
            for name in ("k_cache", "v_cache"))
    key = (blocks[..., None] * page + torch.arange(page, device="cuda")).view(T, Hkv, -1)
    seen = (blocks >= 0)[..., None].expand(-1, -1, -1, page).reshape(T, Hkv, -1) & (key <= pos[:, None, None])
    s = torch.matmul(st["q"].float().view(T, Hkv, G, D), k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(D))
    s = s.masked_fill(~seen[:, :, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p / p.sum(-1, keepdim=True), v)
    return o.view(T, Hq, D).to(torch.bfloat16), blocks.int()


# ------------------------------------------------------------------ the definitions in 64 bits

def exact_norm(case, st):
    s = st["x_"].double() + (st["r_"].double() if case["r"] else 0.0)
    w = st["w"].double() + (1.0 if case["plus_one"] else 0.0)
    y = s / torch.sqrt(s.pow(2).sum(1, keepdim=True) / case["d"] + EPS) * w
    h = [s] if case["r"] else []
    if case["out"] not in LARGEST:
        return tuple([y] + h) if h else y
    group = case["group"] or case["d"]
    scales = torch.stack([p.abs().max(1).values for p in y.split(group, dim=1)], dim=1) / LARGEST[case["out"]]
    t = y / scales.repeat_interleave(group, dim=1)
    if case["out"] == "int8":
        t = t.round()
    else:  # three bits behind the leading one, none below 2^-9
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        t = torch.round(t / step) * step
    return tuple([t * scales.repeat_interleave(group, dim=1), scales] + h)


def exact_heads(x, w, freqs, magnitude, interleaved, pos):
    """Norm and rotation of heads [T, H, D] in 64 bits, as products of complex numbers."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
    n = freqs.numel()
    order = torch.arange(2 * n, device="cuda")
    order = order.view(n, 2) if interleaved else order.view(2, n).t()
    z = torch.view_as_complex(x[..., order].contiguous())
    angle = pos.double()[:, None, None] * freqs.double()
    z = z * torch.polar(torch.full_like(angle, magnitude), angle)
    y = x.clone()
    y[..., order.reshape(-1)] = torch.view_as_real(z).flatten(-2)
    return y


def exact_groups(x):
    """What 64 values x (float64, last axis) are read back as: scale * code + bias."""
    lo, hi = x.amin(-1), x.amax(-1)
    b = lo.to(torch.bfloat16).double()
    s = ((hi - b) / 15.0).to(torch.bfloat16).double()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)[..., None]
    q = torch.where(s > 0, torch.round((x - b[..., None]) / s), torch.zeros_like(x)).clamp(0, 15)
    return s * q + b[..., None]


def exact_values(c, pages, h):
    """Rows [pages * page, D] of one head in 64 bits."""
    at = pages.long()
    codes = c["codes"][at, h].int().flatten(0, 1)
    v = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device="cuda")
    v[:, 0::2] = (codes % 16).double()
    v[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    s = c["scales"][at, h].flatten(0, 1).double().repeat_interleave(GROUP, dim=1)
    return v * s + c["biases"][at, h].flatten(0, 1).double().repeat_interleave(GROUP, dim=1)


def exact_sparse(case, st):
    new, total = lengths(case)
    page, D, G = case["page"], case["D"], case["Hq"] // case["Hkv"]
    out = torch.zeros((st["T"], case["Hq"], D), dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, t) in enumerate(zip(new, total)):
        pages = st["table"][b][:-(-t // page)]
        W = pages.numel()
        c = torch.arange(W, device="cuda")
        step = max(1, min(n, 100_000_000 // (G * W * max(page, D))))
        for h in range(case["Hkv"]):
            k, v = exact_values(st["k_cache"], pages, h), exact_values(st["v_cache"], pages, h)
            lo, hi = st["bounds"][pages.long(), h].double().unbind(1)
            for i in range(0, n, step):
                rows = torch.arange(i, min(i + step, n), device="cuda")
                q = st["q"][start + rows, h * G:(h + 1) * G].double()  # [m, G, D]
                pos = (t - n + rows)[:, None]
                most = torch.maximum(q[:, :, None] * lo, q[:, :, None] * hi).sum((1, 3)).float()
                free = (c >= case["first"]) & (c <= pos // page - case["recent"])
                rank = torch.argsort(torch.where(free, -most, math.inf), dim=1, stable=True).argsort(1)
                keep = torch.where(free, rank < case["top"], c <= pos // page)
                keep = keep.repeat_interleave(page, dim=1) & (torch.arange(W * page, device="cuda") <= pos)
                z = torch.matmul(q, k.t()) / math.sqrt(D)
                z = torch.softmax(z.masked_fill(~keep[:, None], -math.inf), dim=-1)
                out[start + rows, h * G:(h + 1) * G] = torch.matmul(z, v)
        start += n
    return out, None


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(case, st)
    if case["op"] == "rope":
        return exact_heads(st["x_"], st["w"], st["freqs"], st["magnitude"], case["interleaved"], st["pos"])
    if case["op"] == "sparse":
        return exact_sparse(case, st)
    new, total = lengths(case)
    if case["op"] == "write":
        pos = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)])
        Hq, m = case["Hq"], case["Hq"] + case["Hkv"]
        turn = lambda x, w: exact_heads(x, w, st["freqs"], st["magnitude"], case["interleaved"], pos)
        held = lambda x: exact_groups(x.reshape(*x.shape[:2], -1, GROUP)).view(x.shape)
        return (turn(st["qkv"][:, :Hq], st["qw"]), held(turn(st["qkv"][:, Hq:m], st["kw"])),
                held(st["qkv"][:, m:].double()))
    out = st["bounds"].double()
    for b, (n, t) in enumerate(zip(new, total)):
        if n == 0:
            continue
        blocks = torch.arange((t - n) // case["page"], (t - 1) // case["page"] + 1, device="cuda")
        pages = st["table"][b][blocks]
        for h in range(case["Hkv"]):
            x = exact_values(st["k_cache"], pages, h).view(blocks.numel(), case["page"], -1)
            gone = (blocks[:, None] * case["page"] + torch.arange(case["page"], device="cuda") >= t)[..., None]
            out[pages.long(), h, 0] = x.masked_fill(gone, math.inf).amin(1)
            out[pages.long(), h, 1] = x.masked_fill(gone, -math.inf).amax(1)
    return out
