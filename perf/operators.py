"""The operators of the int4-g64 attention half of a decoder layer: what is measured.

Three operators, in the framework's int4-g64 format (unsigned 4-bit codes, one bf16 scale and one
bf16 bias per 64 values, value = scale * code + bias):
  cache      new keys and values quantised into a paged cache, and cache rows read back;
  attention  queries over the paged 4-bit cache (one, a few or many new tokens a sequence);
  linear     y = act(x W^T + bias) + residual with int4-g64 weights.

A case names one operator and its sizes. With ``own`` false, run() computes it with elementary torch
operations in 32 bits; with ``own`` true it calls the framework. exact() is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token for each of 8 sequences: the cache write of a small decode step
        dict(name="cache write, 8 tokens", op="append", B=8, new=1, past=700, spread=0, Hkv=2, D=256,
             page=64, dtype="bf16"),
        # the prompt chunk of several requests, written while prefilling, from fp32 projections
        dict(name="cache write, prompts", op="append", B=7, new=1500, past=100, spread=3, Hkv=8, D=128,
             page=16, dtype="f32"),
        # whole sequences rebuilt to bf16, as before a re-ordering or an export of the cache
        dict(name="cache read, whole sequences", op="read", B=16, new=8191, past=0, spread=4, Hkv=4,
             D=128, page=128, dtype="bf16"),
        # a single short conversation at batch 1: latency
        dict(name="attention, 1 x 500", op="attention", B=1, new=1, past=499, spread=0, Hq=16, Hkv=2,
             D=256, page=16, causal=True, window=0),
        # a serving batch of mixed lengths
        dict(name="attention, 64 mixed", op="attention", B=64, new=1, past=8100, spread=5, Hq=16, Hkv=2,
             D=256, page=64, causal=True, window=0),
        # one very long context at batch 1: the whole card on one sequence
        dict(name="attention, 1 x 128K", op="attention", B=1, new=1, past=131149, spread=0, Hq=16, Hkv=2,
             D=128, page=128, causal=True, window=0),
        # every head its own keys, small heads, a sliding window, three draft tokens checked at once
        dict(name="attention, drafts in a window", op="attention", B=5, new=3, past=2900, spread=6, Hq=8,
             Hkv=8, D=64, page=32, causal=True, window=1000),
        # a prompt chunk behind an earlier context
        dict(name="attention, prefill 4096", op="attention", B=1, new=4096, past=1003, spread=0, Hq=16,
             Hkv=2, D=128, page=64, causal=True, window=0),
        # the fused q, k, v projection of one decode token
        dict(name="linear, 1 token", op="linear", T=1, rows=5120, cols=2048, bias=True, act="none",
             residual=False, dtype="bf16"),
        # the output projection of a small batch, added to the fp32 residual stream
        dict(name="linear, 37 tokens, residual", op="linear", T=37, rows=2048, cols=4096, bias=False,
             act="none", residual=True, dtype="f32"),
        # a dense feed-forward projection with its activation, odd number of outputs
        dict(name="linear, 777 tokens, silu", op="linear", T=777, rows=1001, cols=2048, bias=True,
             act="silu", residual=False, dtype="bf16"),
        # the fused projection of a long prompt
        dict(name="linear, 8192 tokens", op="linear", T=8192, rows=5120, cols=2048, bias=True, act="none",
             residual=False, dtype="bf16"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(max(w["bytes"], w["flops"] / 50) for w in map(work, listed()))
    while True:
        op = rng.choice(["append", "read", "attention", "attention", "linear"])
        if op == "linear":
            c = dict(op=op, T=log_int(rng, 1, 8192), rows=log_int(rng, 60, 6000),
                     cols=64 * log_int(rng, 2, 96), bias=rng.random() < 0.5,
                     act=rng.choice(["none", "relu", "silu", "gelu"]), residual=rng.random() < 0.5,
                     dtype=rng.choice(["bf16", "f32"]))
        else:
            c = dict(op=op, B=log_int(rng, 1, 64), new=1, past=0, spread=rng.randint(0, 50),
                     Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]),
                     page=rng.choice([16, 32, 64, 128, 256]))
            if op == "append":
                c.update(new=log_int(rng, 1, 3000), past=log_int(rng, 1, 5000),
                         dtype=rng.choice(["bf16", "f32"]))
            elif op == "read":
                c.update(new=log_int(rng, 1, 9000), dtype=rng.choice(["bf16", "f32"]))
            else:
                c.update(Hq=c["Hkv"] * rng.choice([1, 2, 3, 4, 8, 12]),
                         new=rng.choice([1, 1, 2, 5, log_int(rng, 8, 3000)]),
                         past=log_int(rng, 1, 120000), causal=rng.random() < 0.8,
                         window=rng.choice([0, 0, 0, log_int(rng, 16, 4000)]))
                if c["Hq"] * c["B"] * c["new"] * (c["new"] + c["past"]) > 700_000_000:
                    continue  # the plain form's scores
        w = work(c)
        if op != "linear" and c["B"] * (c["new"] + c["past"]) * c["Hkv"] * c["D"] > 600_000_000:
            continue  # the plain form's keys
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


def keys_seen(case):
    """Keys that all the new tokens of a case attend to, summed."""
    n = 0
    for new, total in zip(*lengths(case)):
        pos = np.arange(total - new, total, dtype=np.int64)
        first = np.maximum(pos - case["window"] + 1, 0) if case["window"] else np.zeros_like(pos)
        last = pos if case["causal"] else np.full_like(pos, total - 1)
        n += int((last - first + 1).sum())
    return n


def work(case):
    if case["op"] == "linear":
        T, n, k = case["T"], case["rows"], case["cols"]
        out = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * k * 0.5625 + T * k * 2 + T * n * out * (2 if case["residual"] else 1)
                + (2 * n if case["bias"] else 0), "flops": 2.0 * T * n * k}
    new, total = lengths(case)
    row = case["Hkv"] * case["D"] * 2  # key and value elements of a token
    if case["op"] == "attention":
        kept = sum(min(t, n + case["window"] - 1) if case["window"] else t for n, t in zip(new, total))
        return {"bytes": kept * row * 0.5625 + sum(new) * case["Hq"] * case["D"] * 4,
                "flops": 4.0 * keys_seen(case) * case["Hq"] * case["D"]}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":  # read the inputs, write the cache, read it, write the values
        return {"bytes": sum(new) * row * (2 * size + 2 * 0.5625), "flops": sum(new) * row * 8.0}
    return {"bytes": sum(new) * row * (size + 0.5625), "flops": sum(new) * row * 2.0}


# ------------------------------------------------------------------ inputs

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def plane(n, shape, gen, outliers):
    """n int4-g64 matrices of shape (rows, cols), quantised from seeded values, a part at a time."""
    rows, cols = shape
    codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, rows, cols // GROUP), dtype=torch.bfloat16, device="cuda")
    biases = torch.empty_like(scales)
    heavy = torch.ones(cols, device="cuda")
    if outliers:  # a few channels of the keys are large, as in trained models
        heavy[torch.randperm(cols, generator=gen, device="cuda")[:4]] = 5.0
    step = max(1, (1 << 24) // (rows * cols))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn((m, rows, cols), generator=gen, device="cuda") * heavy
        q, scales[i:i + m], biases[i:i + m] = quantise(x.to(torch.bfloat16))
        codes[i:i + m] = packed(q)
    return {"codes": codes, "scales": scales, "biases": biases}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["op"] == "linear":
        T, n, k = case["T"], case["rows"], case["cols"]
        st["x"] = torch.randn((T, k), generator=gen, device="cuda").to(torch.bfloat16)
        w = torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5
        q, s, b = quantise(w.to(torch.bfloat16))
        st["w"] = {"codes": packed(q)[None], "scales": s[None], "biases": b[None]}
        st["b"] = (torch.randn(n, generator=gen, device="cuda").to(torch.bfloat16) if case["bias"] else None)
        st["r"] = (torch.randn((T, n), generator=gen, device="cuda").to(TYPES[case["dtype"]])
                   if case["residual"] else None)
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
    if case["op"] == "append":
        empty = dict(device="cuda")
        for name in ("k", "v"):
            st[name + "_cache"] = {
                "codes": torch.zeros((pages, Hkv, page, D // 2), dtype=torch.uint8, **empty),
                "scales": torch.zeros((pages, Hkv, page, D // GROUP), dtype=torch.bfloat16, **empty),
                "biases": torch.zeros((pages, Hkv, page, D // GROUP), dtype=torch.bfloat16, **empty)}
        kv = torch.randn((T, 2 * Hkv, D), generator=gen, device="cuda")
        kv[:, :Hkv, :4] *= 5.0
        st["kv"] = kv.to(TYPES[case["dtype"]])  # keys then values of a token, as one projection leaves them
        return st
    for name in ("k", "v"):
        c = plane(pages * Hkv, (page, D), gen, outliers=name == "k")
        st[name + "_cache"] = {f: a.view(pages, Hkv, page, -1) for f, a in c.items()}
    if case["op"] == "attention":
        st["q"] = torch.randn((T, case["Hq"], D), generator=gen, device="cuda").to(torch.bfloat16)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return run_own(st)
    if st["op"] == "linear":
        return plain_linear(st)
    if st["op"] == "attention":
        return plain_attention(st)
    return plain_cache(st)


def run_own(st):
    import bit_quantized_grouped_router_amd as M
    if st["op"] == "linear":
        w = st["w"]
        return M.moe_linear_w4(st["x"], M.W4Matrix(w["codes"], w["scales"], w["biases"]), bias=st["b"],
                               act=st["act"], residual=st["r"], out_dtype=TYPES[st["dtype"]])
    k, v = st["k_cache"], st["v_cache"]
    cache = M.KV4Cache(M.W4Matrix(k["codes"], k["scales"], k["biases"]),
                       M.W4Matrix(v["codes"], v["scales"], v["biases"]))
    table, cu, length = st["table"], st["cu"], st["len"]
    if st["op"] == "attention":
        return M.moe_kv4_attention(cache, st["q"], table, cu, length, max_new=st["max_new"],
                                   causal=st["causal"], window=st["window"])
    if st["op"] == "append":
        H = st["Hkv"]
        M.moe_kv4_append(cache, st["kv"][:, :H], st["kv"][:, H:], table, cu, length)
    return M.moe_kv4_read(cache, table, cu, length, st["T"], dtype=TYPES[st["dtype"]])


def rows_of(st):
    """Page and slot of every new token."""
    tok = torch.arange(st["T"], device="cuda")
    cu, length = st["cu"].long(), st["len"].long()
    b = torch.searchsorted(cu[1:], tok, right=True)
    pos = length[b] - cu[b + 1] + tok
    return st["table"].long()[b, pos // st["page"]], pos % st["page"]


def values_of(cache, page, slot):
    """Cache values scale * code + bias in 32 bits, [..., Hkv, D], at (page, slot)."""
    c = cache["codes"][page, :, slot]
    q = torch.stack([c & 15, c >> 4], dim=-1).float()
    q = q.view(*c.shape[:-1], -1, GROUP)
    s, b = cache["scales"][page, :, slot].float(), cache["biases"][page, :, slot].float()
    return (s[..., None] * q + b[..., None]).view(*c.shape[:-1], -1)


def plain_cache(st):
    page, slot = rows_of(st)
    out = []
    H = st["Hkv"]
    if st["op"] == "append":
        both = st["kv"].view(st["T"], 2, H, st["D"])
        q, s, b = quantise(both)
        q = packed(q)
        k, v = st["k_cache"], st["v_cache"]
        k["codes"][page, :, slot], v["codes"][page, :, slot] = q[:, 0], q[:, 1]
        k["scales"][page, :, slot], v["scales"][page, :, slot] = s[:, 0], s[:, 1]
        k["biases"][page, :, slot], v["biases"][page, :, slot] = b[:, 0], b[:, 1]
    out = [values_of(st[n], page, slot).to(TYPES[st["dtype"]]) for n in ("k_cache", "v_cache")]
    return tuple(out)


def plain_attention(st):
    B, Hq, Hkv, D, n = st["B"], st["Hq"], st["Hkv"], st["D"], st["max_new"]
    cu, length = st["cu"].long(), st["len"].long()
    L = st["table"].shape[1] * st["page"]
    t = torch.arange(L, device="cuda")
    page = st["table"].long()[:, t // st["page"]]
    slot = (t % st["page"]).expand(B, L)
    k = values_of(st["k_cache"], page, slot)  # [B, L, Hkv, D]
    v = values_of(st["v_cache"], page, slot)
    # queries padded to n a sequence
    i = torch.arange(n, device="cuda")
    new = cu[1:] - cu[:-1]
    real = i[None] < new[:, None]
    row = (cu[:-1, None] + i[None]).clamp(max=st["T"] - 1)
    q = st["q"].float()[row].view(B, n, Hkv, Hq // Hkv, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * (Hq // Hkv), D).contiguous()
    s = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * (1.0 / math.sqrt(D))
    pos = (length - new)[:, None] + i[None]
    seen = t[None, None] < length[:, None, None]
    if st["causal"]:
        seen = seen & (t[None, None] <= pos[..., None])
    if st["window"]:
        seen = seen & (t[None, None] > pos[..., None] - st["window"])
    s = s.view(B, Hkv, n, Hq // Hkv, L).masked_fill(~seen[:, None, :, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, L), v.permute(0, 2, 1, 3).contiguous())
    o = o.view(B, Hkv, n, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    return o[real].to(torch.bfloat16)


def plain_linear(st):
    w = st["w"]
    c = w["codes"][0]
    q = torch.stack([c & 15, c >> 4], dim=-1).float().view(c.shape[0], -1, GROUP)
    m = (w["scales"][0].float()[..., None] * q + w["biases"][0].float()[..., None]).to(torch.bfloat16)
    y = torch.matmul(st["x"].float(), m.view(c.shape[0], -1).float().t())
    if st["b"] is not None:
        y = y + st["b"].float()
    if st["act"] == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif st["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif st["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if st["r"] is not None:
        y = y + st["r"].float()
    return y.to(TYPES[st["dtype"]])


# ------------------------------------------------------------------ the definitions in 64 bits

def to_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def exact_groups(x):
    """What 64 values x (float32, last axis) are read back as: scale * code + bias."""
    lo, hi = x.min(-1), x.max(-1)
    b = to_bf16(lo)
    s = to_bf16((hi - b) * np.float32(1.0 / 15.0))
    s = np.where(s < 2.0 ** -126, np.float32(0), s)
    t = (x - b[..., None]).astype(np.float64)  # the difference is rounded to 32 bits by definition
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, np.rint(t / s[..., None].astype(np.float64)), 0.0)
    return s[..., None].astype(np.float64) * np.clip(q, 0, 15) + b[..., None]


def exact_cache(cache, pages, total, page, h):
    """Keys or values [total, D] of one sequence and head in 64 bits."""
    t = torch.arange(total, device="cuda")
    at = (pages[t // page].long(), h, t % page)
    c = cache["codes"][at].int()
    v = torch.empty((total, 2 * c.shape[1]), dtype=torch.float64, device="cuda")
    v[:, 0::2] = (c % 16).double()
    v[:, 1::2] = torch.div(c, 16, rounding_mode="floor").double()
    s = cache["scales"][at].double().repeat_interleave(GROUP, dim=1)
    return v * s + cache["biases"][at].double().repeat_interleave(GROUP, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        w = st["w"]
        c = w["codes"][0].int()
        m = torch.empty((case["rows"], case["cols"]), dtype=torch.float64, device="cuda")
        m[:, 0::2], m[:, 1::2] = (c % 16).double(), torch.div(c, 16, rounding_mode="floor").double()
        m = m * w["scales"][0].double().repeat_interleave(GROUP, dim=1)
        m = m + w["biases"][0].double().repeat_interleave(GROUP, dim=1)
        m = m.float().to(torch.bfloat16).double()  # weights are rebuilt to bf16, by definition
        z = st["x"].double() @ m.t()
        if case["bias"]:
            z = z + st["b"].double()
        if case["act"] == "relu":
            z = z.clamp(min=0)
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        return z + st["r"].double() if case["residual"] else z
    if case["op"] == "append":
        kv = st["kv"].float().cpu().numpy()
        v = exact_groups(kv.reshape(*kv.shape[:2], -1, GROUP)).reshape(kv.shape)
        return v[:, :case["Hkv"]].copy(), v[:, case["Hkv"]:].copy()
    new, total = lengths(case)
    Hkv, page = case["Hkv"], case["page"]
    if case["op"] == "read":
        return tuple(torch.cat([torch.stack([exact_cache(st[n], st["table"][b], total[b], page, h)
                                             for h in range(Hkv)], dim=1)
                                for b in range(case["B"])]) for n in ("k_cache", "v_cache"))
    G, row = case["Hq"] // Hkv, 0
    out = torch.zeros((st["T"], case["Hq"], case["D"]), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        t = torch.arange(total[b], device="cuda")
        pos = torch.arange(total[b] - new[b], total[b], device="cuda")[:, None]
        hidden = (t > pos) if case["causal"] else torch.zeros_like(t > pos)
        if case["window"]:
            hidden = hidden | (t <= pos - case["window"])
        for h in range(Hkv):
            k = exact_cache(st["k_cache"], st["table"][b], total[b], page, h)
            v = exact_cache(st["v_cache"], st["table"][b], total[b], page, h)
            for g in range(h * G, (h + 1) * G):
                z = st["q"][row:row + new[b], g].double() @ k.t() / math.sqrt(case["D"])
                out[row:row + new[b], g] = torch.softmax(z.masked_fill(hidden, -math.inf), dim=-1) @ v
        row += new[b]
    return out
