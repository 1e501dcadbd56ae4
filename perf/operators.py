"""Measured cases of the operators around the KV cache: rotary positions (alone and fused with the append),
attention with capped or biased scores and per-row key ranges (documents, prefixes) with its gradients and its form
for one token, the attention weight each cached key receives, and eviction of the lightest keys.

Every case runs in two forms. With ``own`` false, ``run`` computes it from elementary torch operations in 32 bits
(angles in 64); with ``own`` true it makes the calls a user of the library makes. ``exact`` computes the same
results in 64 bits, written apart from both. Sizes follow the library's workloads (32 query and 8 KV heads of 128,
8192 cached positions for decode, 4096-token prompts, histories of 32768).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _rope(name=None, *, B, h, S, d, rot, offset=0, interleaved=False, inverse=False, fused=0, start=0,
          yarn=1.0, dtype="bf16"):
    c = dict(op="rope", B=B, h=h, S=S, d=d, rot=rot, offset=offset, interleaved=interleaved, inverse=inverse,
             fused=fused, start=start, yarn=yarn, dtype=dtype)
    return dict(c, name=name) if name else c


def _append(name=None, *, B, h_q, h_kv, S, T, d, rot, interleaved=False, page=0, yarn=1.0, dtype="bf16"):
    c = dict(op="append", B=B, h_q=h_q, h_kv=h_kv, S=S, T=T, d=d, rot=rot, interleaved=interleaved, page=page,
             yarn=yarn, dtype=dtype)
    return dict(c, name=name) if name else c


def _weights(name=None, *, B, h_q, h_kv, S, T, d, shortest=0, window=0, page=0, accumulate=False, dtype="bf16"):
    c = dict(op="weights", B=B, h_q=h_q, h_kv=h_kv, S=S, T=T, d=d, shortest=shortest or T, window=window, page=page,
             accumulate=accumulate, dtype=dtype)
    return dict(c, name=name) if name else c


def _evict(name=None, *, B, h_kv, T, budget, d, shortest=0, sink=0, recent=0, page=0, dtype="bf16"):
    c = dict(op="evict", B=B, h_kv=h_kv, T=T, budget=budget, d=d, shortest=shortest or T, sink=sink, recent=recent,
             page=page, dtype=dtype)
    return dict(c, name=name) if name else c


def _attend(name=None, *, B, h_q, h_kv, S, T, d, cap=0.0, alibi=False, docs=0, prefix=0, causal=True, window=0,
            grad=False, page=0, shortest=0, dtype="bf16"):
    c = dict(op="attend", B=B, h_q=h_q, h_kv=h_kv, S=S, T=T, d=d, cap=cap, alibi=alibi, docs=docs, prefix=prefix,
             causal=causal, window=window, grad=grad, page=page, shortest=shortest or T, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of eight sequences: its q and k rotated, k and v appended (every decode step)
        _append("append_one_token", B=8, h_q=32, h_kv=8, S=1, T=1024, d=128, rot=128),
        # a 512-token prompt chunk of four sequences into 16-token pages, interleaved pairs, stretched context
        _append("append_chunk_paged", B=4, h_q=32, h_kv=8, S=512, T=2048, d=128, rot=128, interleaved=True, page=16,
                yarn=8.0),
        # the gradient of the rotation for long prompts, read in place from a fused q/k/v buffer (B, S, 48 heads, 128)
        _rope("rope_gradient_long", B=2, h=32, S=8192, d=128, rot=128, fused=16, inverse=True),
        # a 4096-token prompt whose scores are capped, causal
        _attend("prefill_capped", B=1, h_q=32, h_kv=8, S=4096, T=4096, d=128, cap=50.0),
        # a training step over twelve documents packed into one 4096-token row, distance bias: outputs and gradients
        _attend("train_documents_biased", B=1, h_q=32, h_kv=8, S=4096, T=4096, d=128, alibi=True, docs=12, grad=True),
        # one token of eight ragged sequences over 16-token pages, capped and biased
        _attend("decode_capped_biased", B=8, h_q=32, h_kv=8, S=1, T=8192, d=128, cap=30.0, alibi=True, page=16,
                shortest=2001),
        # check mode: a small fp32 training step with a bidirectional prefix, capped, odd sizes
        _attend("train_prefix_fp32", B=2, h_q=6, h_kv=2, S=67, T=67, d=96, cap=20.0, prefix=13, causal=False,
                grad=True, dtype="fp32"),
        # the weight one decoded token gives every cached key, added to the running totals
        _weights("weights_one_token", B=8, h_q=32, h_kv=8, S=1, T=8192, d=128, accumulate=True),
        # the last 33 queries of prompts score long ragged histories in 16-token pages, NaN behind each sequence
        _weights("weights_last_queries", B=2, h_q=32, h_kv=8, S=33, T=32768, d=128, shortest=21001, page=16),
        # every query of a 4096-token prompt, causal
        _weights("weights_whole_prompt", B=1, h_q=32, h_kv=8, S=4096, T=4096, d=128),
        # eight sequences of 8192 keys cut to a quarter, into a smaller cache
        _evict("evict_to_quarter", B=8, h_kv=8, T=8192, budget=2048, d=128, sink=4, recent=256),
        # long ragged histories in 16-token pages, into fresh pages of the same pool
        _evict("evict_long_paged", B=4, h_kv=8, T=32768, budget=4096, d=128, shortest=3001, sink=4, recent=512, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope", "attend", "attend", "decode", "weights", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128]) if dtype == "bf16" and op in ("weights", "attend", "decode") else rng.choice([64, 72, 80, 96, 128, 128, 192, 256])
    h_kv = rng.choice([1, 2, 3, 4, 8])
    r = rng.choice([1, 2, 3, 4, 7, 8, 16]) if h_kv < 8 else rng.choice([1, 2, 4])
    page = rng.choice([0, 0, 16, 64, 48])
    up = lambda t: -(-t // page) * page if page else t  # noqa: E731
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        offset = rng.choice([0, d - rot, rng.randint(0, d - rot)])
        B, S = rng.randint(1, 8), _log(rng, 1, 8192)
        h = max(1, min(h_kv * r, 67108864 // (B * S * d)))
        return _rope(B=B, h=h, S=S, d=d, rot=rot, offset=offset, interleaved=rng.random() < 0.5,
                     inverse=rng.random() < 0.5, fused=rng.choice([0, 0, 1, 8]), start=_log(rng, 1, 1000000) - 1,
                     yarn=rng.choice([1.0, 4.0, 32.0]), dtype=dtype)
    if op == "append":
        B, S = rng.randint(1, 16), _log(rng, 1, 2048)
        T = up(S + _log(rng, 1, 1024))
        h_q = h_kv * r
        B = max(1, min(B, 33554432 // (h_kv * T * d), 67108864 // (S * (h_q + 2 * h_kv) * d)))
        return _append(B=B, h_q=h_q, h_kv=h_kv, S=S, T=T, d=d, rot=rng.choice([d, d // 2]),
                       interleaved=rng.random() < 0.5, page=page, yarn=rng.choice([1.0, 8.0]), dtype=dtype)
    if op == "weights":
        T = up(_log(rng, 1, 32768 if dtype == "bf16" else 4096))
        S = min(T, rng.choice([1, 1, 1, _log(rng, 2, 128), _log(rng, 2, 2048)]))
        if dtype == "fp32":
            S = min(S, 64)
        room = (100000000 if dtype == "bf16" else 6000000) // (h_kv * r * S * T) if S > 1 else 60000000 // (h_kv * T * d)
        while S > 1 and room < 1:
            S //= 2
            room = (100000000 if dtype == "bf16" else 6000000) // (h_kv * r * S * T)
        B = max(1, min(rng.randint(1, 16), room, 67108864 // (h_kv * T * d)))
        return _weights(B=B, h_q=h_kv * r, h_kv=h_kv, S=S, T=T, d=d, shortest=rng.randint(S, T),
                        window=rng.choice([0, 0, 0, _log(rng, 1, T)]), page=page, accumulate=rng.random() < 0.5,
                        dtype=dtype)
    if op in ("attend", "decode"):
        cap, alibi = rng.choice([(0.0, True), (0.0, False), (20.0, False), (50.0, False), (30.0, True)])
        if op == "decode":
            T = up(_log(rng, 1, 32768 if dtype == "bf16" else 4096))
            B = max(1, min(rng.randint(1, 16), 60000000 // (h_kv * T * d)))
            return _attend(B=B, h_q=h_kv * r, h_kv=h_kv, S=1, T=T, d=d, cap=cap, alibi=alibi,
                           window=rng.choice([0, 0, _log(rng, 1, T)]), page=page, shortest=rng.randint(1, T), dtype=dtype)
        T = _log(rng, 2, 4096 if dtype == "bf16" else 512)
        S = T if rng.random() < 0.7 else rng.randint(2, T)
        mask = rng.choice(["none", "docs", "prefix", "window"]) if S == T else "none"
        room = (500000000 if dtype == "bf16" else 10000000) // (h_kv * r * S * T)
        h_kv = h_kv if room else 1
        B = max(1, min(rng.randint(1, 8), room))
        return _attend(B=B, h_q=h_kv * r, h_kv=h_kv, S=S, T=T, d=d, cap=cap, alibi=alibi,
                       docs=rng.randint(1, min(T, 16)) if mask == "docs" else 0,
                       prefix=rng.randint(1, T) if mask == "prefix" else 0, causal=mask != "prefix",
                       window=_log(rng, 1, T) if mask == "window" else 0, grad=rng.random() < 0.5, dtype=dtype)
    T = up(_log(rng, 2, 32768))
    budget = _log(rng, 1, T)
    sink = rng.choice([0, 0, min(4, budget)])
    recent = rng.choice([0, rng.randint(0, budget - sink)])
    B = max(1, min(rng.randint(1, 16), 67108864 // (h_kv * T * d)))
    return _evict(B=B, h_kv=h_kv, T=T, budget=budget, d=d, shortest=rng.randint(1, T), sink=sink, recent=recent,
                  page=page, dtype=dtype)


def _lengths(c):
    """The cached length of each sequence: evenly spread from the full history to the shortest."""
    return [c["T"] - (c["T"] - c["shortest"]) * b // max(1, c["B"] - 1) for b in range(c["B"])]


def _documents(c):
    """First and last-but-one positions of the documents packed into a row: shorter ones first."""
    if not c["docs"]:
        return [(0, c["T"])]
    cut = [int(c["T"] * (i / c["docs"]) ** 1.4) for i in range(c["docs"] + 1)]
    return [(lo, hi) for lo, hi in zip(cut, cut[1:]) if hi > lo]


def _ranges(c):
    """(S, 2): the keys lo <= j < hi that each row's document and prefix let it see (S = T rows)."""
    out = []
    for lo, hi in _documents(c):
        out += [(lo, min(hi, max(p + 1, lo + c["prefix"]))) for p in range(lo, hi)]
    return out


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        n = c["B"] * c["h"] * c["S"] * c["d"]
        return {"bytes": 2 * e * n, "flops": 3 * c["B"] * c["h"] * c["S"] * c["rot"]}
    if c["op"] == "append":
        rows = c["B"] * c["S"] * (c["h_q"] + 2 * c["h_kv"])
        return {"bytes": 2 * e * rows * c["d"], "flops": 3 * c["B"] * c["S"] * (c["h_q"] + c["h_kv"]) * c["rot"]}
    lens = _lengths(c)
    if c["op"] == "attend":
        pairs, keys = 0, 0
        for n in lens:
            see = _ranges(c) if c["docs"] or c["prefix"] else [(0, n)] * c["S"]
            at = [n - c["S"] + i for i in range(c["S"])]
            see = [(max(lo, p - c["window"] + 1) if c["window"] else lo, min(hi, p + 1) if c["causal"] else hi)
                   for (lo, hi), p in zip(see, at)]
            pairs += sum(max(0, hi - lo) for lo, hi in see)
            keys += max(hi for _, hi in see) - min(lo for lo, _ in see)
        qo, kv = c["B"] * c["h_q"] * c["S"], keys * c["h_kv"]
        nbytes = (2 * qo + 2 * kv) * c["d"] * e + 4 * qo
        if not c["grad"]:
            return {"bytes": nbytes, "flops": 4 * pairs * c["h_q"] * c["d"]}
        return {"bytes": nbytes + (2 * qo + 2 * c["B"] * c["T"] * c["h_kv"]) * c["d"] * e,
                "flops": 14 * pairs * c["h_q"] * c["d"]}
    if c["op"] == "weights":
        pairs, keys = 0, 0
        for n in lens:
            lo = max(0, n - c["S"] - c["window"] + 1) if c["window"] else 0
            keys += n - lo
            for p in range(n - c["S"], n):
                pairs += min(p + 1, c["window"]) if c["window"] else p + 1
        q = c["B"] * c["h_q"] * c["S"] * (c["d"] * e + 4)
        out = c["h_kv"] * 4 * (2 * keys if c["accumulate"] else c["B"] * c["T"])
        return {"bytes": keys * c["h_kv"] * c["d"] * e + q + out, "flops": 2 * pairs * c["h_q"] * c["d"]}
    kept = sum(min(n, c["budget"]) for n in lens) * c["h_kv"]
    return {"bytes": sum(lens) * c["h_kv"] * 4 + kept * (4 * c["d"] * e + 8), "flops": sum(lens) * c["h_kv"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _inv_freq(rot, yarn):
    """Angle per position of each pair: base 10000, stretched by parts over a context `yarn` times 4096 long."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if yarn == 1.0:
        return f.cuda(), 1.0
    turns = 4096 * f / (2 * math.pi)
    fast = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (f * (fast + (1.0 - fast) / yarn)).cuda(), 0.1 * math.log(yarn) + 1.0


def _pool(dense, page, g):
    """A cache (B, h, T, d) as a pool of pages in random order, with spare pages, and its block table."""
    B, h, T, d = dense.shape
    n = T // page
    order = torch.randperm(B * n, generator=g, device="cuda")
    pages = torch.empty((B * n, h, page, d), dtype=dense.dtype, device="cuda")
    pages[order] = dense.view(B, h, n, page, d).permute(0, 2, 1, 3, 4).reshape(B * n, h, page, d)
    return pages, order.view(B, n).to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    s = dict(c=c)
    B, d = c["B"], c["d"]
    if c["op"] == "rope":
        f = c["fused"]
        qkv = normal(B, c["S"], c["h"] + f, d)
        s["x"] = qkv[:, :, : c["h"]].transpose(1, 2) if f else normal(B, c["h"], c["S"], d)
        s["inv_freq"], s["scale"] = _inv_freq(c["rot"], c["yarn"])
        s["positions"] = torch.randint(0, c["start"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        return s
    if c["op"] == "append":
        qkv = normal(B, c["S"], c["h_q"] + 2 * c["h_kv"], d)
        s["q"], s["k"], s["v"] = (t.transpose(1, 2) for t in qkv.split([c["h_q"], c["h_kv"], c["h_kv"]], dim=2))
        s["inv_freq"], s["scale"] = _inv_freq(c["rot"], c["yarn"])
        s["pos"] = torch.randint(0, c["T"] - c["S"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["kc"], s["vc"] = normal(B, c["h_kv"], c["T"], d), normal(B, c["h_kv"], c["T"], d)
        if c["page"]:
            s["kc"], s["table"] = _pool(s["kc"], c["page"], g)
            s["vc"] = torch.randn(s["kc"].shape, generator=g, device="cuda").to(dt)
        return s
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    s["lens"] = lens
    if c["op"] == "attend":
        # peaked scores (standard deviation 3), so that the cap and the bias matter
        s["q"] = (3.0 * torch.randn((B, c["h_q"], c["S"], d), generator=g, device="cuda")).to(dt)
        s["k"], s["v"] = normal(B, c["h_kv"], c["T"], d), normal(B, c["h_kv"], c["T"], d)
        s["slopes"] = 2.0 ** (-8.0 * (1 + torch.arange(c["h_q"], device="cuda")) / c["h_q"]) if c["alibi"] else None
        s["range"] = None
        if c["docs"] or c["prefix"]:
            s["range"] = torch.tensor(_ranges(c), dtype=torch.int32, device="cuda").expand(B, -1, -1).contiguous()
        if c["grad"]:
            s["do"] = normal(B, c["h_q"], c["S"], d)
        if c["page"]:
            s["k"], s["table"] = _pool(s["k"], c["page"], g)
            s["v"] = torch.randn(s["k"].shape, generator=g, device="cuda").to(dt)
        if c["S"] == 1 and not c["grad"]:
            s["q"] = s["q"][:, :, 0].contiguous()
        return s
    behind = torch.arange(c["T"], device="cuda")[None, :] >= lens[:, None]  # rows that hold nothing yet
    if c["op"] == "weights":
        k = normal(B, c["h_kv"], c["T"], d)
        s["q"] = normal(B, c["h_q"], c["S"], d)
        s["lse"] = torch.logsumexp(_scores(s["q"], k, lens, c["window"]), -1).reshape(B, c["h_q"], c["S"])
        k.masked_fill_(behind[:, None, :, None], float("nan"))
        s["w"] = torch.rand((B, c["h_kv"], c["T"]), generator=g, device="cuda")
        s["k"] = k
        if c["page"]:
            s["k"], s["table"] = _pool(k, c["page"], g)
        if c["S"] == 1:
            s["q"], s["lse"] = s["q"][:, :, 0], s["lse"][:, :, 0]
        return s
    s["k"], s["v"] = normal(B, c["h_kv"], c["T"], d), normal(B, c["h_kv"], c["T"], d)
    # summed attention weights: a heavy tail, and keys that no query looked at
    w = torch.exp(2.0 * torch.randn((B, c["h_kv"], c["T"]), generator=g, device="cuda")) / c["T"]
    s["w"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
    s["w_out"] = torch.zeros((B, c["h_kv"], c["budget"]), device="cuda")
    if c["page"]:
        p, m = c["page"], -(-c["budget"] // c["page"])
        s["k"], s["table"] = _pool(s["k"], p, g)
        s["v"] = torch.randn(s["k"].shape, generator=g, device="cuda").to(dt)
        n = s["k"].shape[0]
        for name in ("k", "v"):
            s[name] = torch.cat([s[name], normal(B * m, c["h_kv"], p, d)])
        s["table_out"] = (n + torch.randperm(B * m, generator=g, device="cuda")).view(B, m).to(torch.int32)
        s["w_out"] = torch.zeros((B, c["h_kv"], m * p), device="cuda")
    else:
        s["k_out"], s["v_out"] = normal(B, c["h_kv"], c["budget"], d), normal(B, c["h_kv"], c["budget"], d)
    return s


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _visible(lens, S, T, window):
    """(B, S, T): query i sits at cache row lens - S + i and sees the keys at and before it, within the window."""
    at = lens[:, None] - S + torch.arange(S, device="cuda")[None, :]
    key = torch.arange(T, device="cuda")
    seen = key[None, None, :] <= at[:, :, None]
    return seen & (key[None, None, :] > at[:, :, None] - window) if window else seen


def _scores(q, k, lens, window):
    """(B, h_kv, r, S, T) fp32 scores, -inf where a query does not see a key."""
    B, h_kv, T, d = k.shape
    S = q.shape[2]
    s = q.float().reshape(B, h_kv, -1, d) @ k.float().transpose(2, 3)
    s = (s / math.sqrt(d)).view(B, h_kv, -1, S, T)
    return s.masked_fill(~_visible(lens, S, T, window)[:, None, None], float("-inf"))


def _turned(x, inv_freq, at, scale, offset, interleaved, inverse):
    """x (B, h, S, d) rotated by the angles of the positions at (B, S)."""
    angle = at.double()[:, None, :, None] * inv_freq
    cos, sin = (scale * angle.cos()).float(), (scale * angle.sin()).float()
    sin = -sin if inverse else sin
    rot = 2 * inv_freq.numel()
    y = x.float()
    part = y[..., offset:offset + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else part.split(rot // 2, dim=-1)
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y[..., :offset], part, y[..., offset + rot:]], -1).to(x.dtype)


def _dense(pages, table):
    B, n = table.shape
    _, h, p, d = pages.shape
    return pages[table.long()].transpose(1, 2).reshape(B, h, n * p, d)


def _attended(s):
    """Capped and biased attention over the keys each row sees, and its gradients."""
    c = s["c"]
    k, v = (_dense(s[n], s["table"]) if c["page"] else s[n] for n in ("k", "v"))
    q = s["q"].float().reshape(c["B"], c["h_kv"], -1, c["d"])
    k, v, scale = k.float()[:, :, :c["T"]], v.float(), 1 / math.sqrt(c["d"])
    shape = (c["B"], c["h_kv"], c["h_q"] // c["h_kv"], c["S"], c["T"])
    score = (q @ k.transpose(2, 3) * scale).view(shape)
    if c["cap"]:
        turn = torch.tanh(score / c["cap"])
        score = c["cap"] * turn
    at = (s["lens"][:, None] - c["S"] + torch.arange(c["S"], device="cuda"))[:, :, None]
    key = torch.arange(c["T"], device="cuda")
    if c["alibi"]:
        away = (at - key).abs()[:, None, None]
        score = score - s["slopes"].view(1, c["h_kv"], -1, 1, 1) * away
    seen = key < s["lens"][:, None, None]
    if c["causal"]:
        seen = seen & (key <= at)
    if c["window"]:
        seen = seen & (key > at - c["window"])
    if s["range"] is not None:
        seen = seen & (key >= s["range"][..., :1]) & (key < s["range"][..., 1:])
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    lse = torch.logsumexp(score, -1)
    p = (score - lse[..., None]).exp_()
    flat = (c["B"], c["h_kv"], -1, c["T"])
    o = p.reshape(flat) @ v
    out = {"o": o.to(s["q"].dtype).view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}
    if not c["grad"]:
        return out
    do = s["do"].float().reshape(q.shape)
    dp = (do @ v.transpose(2, 3) - (do * o).sum(-1, keepdim=True)).view(shape)
    ds = p * dp
    if c["cap"]:
        ds = ds * (1 - turn * turn)
    ds = ds.reshape(flat) * scale
    out["dq"] = (ds @ k).to(s["q"].dtype).view(s["q"].shape)
    out["dk"] = (ds.transpose(2, 3) @ q).to(s["q"].dtype)
    out["dv"] = (p.reshape(flat).transpose(2, 3) @ do).to(s["q"].dtype)
    return out


def _plain(s):
    c = s["c"]
    if c["op"] == "rope":
        at = s["positions"][:, None] + torch.arange(c["S"], device="cuda")
        return _turned(s["x"], s["inv_freq"], at, s["scale"], c["offset"], c["interleaved"], c["inverse"])
    if c["op"] == "append":
        at = s["pos"].long()[:, None] + torch.arange(c["S"], device="cuda")
        q = _turned(s["q"], s["inv_freq"], at, s["scale"], 0, c["interleaved"], False)
        k = _turned(s["k"], s["inv_freq"], at, s["scale"], 0, c["interleaved"], False).transpose(1, 2)
        v = s["v"].transpose(1, 2)
        if c["page"]:
            page, slot = s["table"].long().gather(1, at // c["page"]), at % c["page"]
        else:
            page, slot = torch.arange(c["B"], device="cuda")[:, None].expand_as(at), at
        s["kc"][page, :, slot] = k
        s["vc"][page, :, slot] = v
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if c["op"] == "attend":
        return _attended(s)
    lens, T = s["lens"], c["T"]
    inside = torch.arange(T, device="cuda")[None, :] < lens[:, None]
    if c["op"] == "weights":
        k = _dense(s["k"], s["table"]) if c["page"] else s["k"]
        q, lse = (s["q"][:, :, None], s["lse"][:, :, None]) if c["S"] == 1 else (s["q"], s["lse"])
        p = _scores(q, k, lens, c["window"])
        p = (p - lse.view(c["B"], c["h_kv"], -1, c["S"], 1)).exp_()
        w = p.sum((2, 3))
        if not c["accumulate"]:
            return w * inside[:, None]
        s["w"] += w * inside[:, None]
        return s["w"]
    # the order of keeping: protected keys, then by weight, the lower index first among equals
    n, key = lens[:, None], torch.arange(T, device="cuda")[None, :]
    safe = inside & ((key < c["sink"]) | (key >= n - c["recent"]))
    rank = s["w"].masked_fill(safe[:, None], float("inf")).masked_fill(~inside[:, None], float("-inf"))
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    new_len = lens.clamp(max=c["budget"])
    there = torch.arange(c["budget"], device="cuda")[None, None, :] < new_len[:, None, None]
    kept = order.masked_fill(~there, T).sort(dim=-1).values
    at = kept.clamp(max=T - 1)
    kept = kept.masked_fill(~there, -1).to(torch.int32)
    w_out = torch.zeros_like(s["w_out"])
    w_out[..., :c["budget"]] = s["w"].gather(2, at) * there
    rows = at[..., None].expand(-1, -1, -1, c["d"])
    if c["page"]:
        pos = torch.arange(c["budget"], device="cuda")
        page = s["table_out"].long()[:, pos // c["page"]]
        dst = (page[:, None, :], torch.arange(c["h_kv"], device="cuda")[None, :, None], (pos % c["page"])[None, None, :])
        for name in ("k", "v"):
            new = _dense(s[name], s["table"]).gather(2, rows)
            s[name][dst] = torch.where(there[..., None], new, s[name][dst])
        return {"k": s["k"], "v": s["v"], "w": w_out, "kept": kept, "len": new_len}
    for name in ("k", "v"):
        s[name + "_out"].copy_(torch.where(there[..., None], s[name].gather(2, rows), s[name + "_out"]))
    return {"k": s["k_out"], "v": s["v_out"], "w": w_out, "kept": kept, "len": new_len}


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------
def _called(s):
    import kv_cache_attention_gqa_b200 as gqa

    c = s["c"]
    if c["op"] == "rope":
        return gqa.rope(s["x"], s["inv_freq"], s["positions"], offset=c["offset"], interleaved=c["interleaved"],
                        inverse=c["inverse"], scale=s["scale"])
    if c["op"] == "append":
        how = dict(interleaved=c["interleaved"], scale=s["scale"])
        if c["page"]:
            q = gqa.kv_rope_append_paged(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], s["table"], s["inv_freq"],
                                         **how)
        else:
            q = gqa.kv_rope_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], s["inv_freq"], **how)
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if c["op"] == "attend":
        how = dict(kv_len=s["lens"], softcap=c["cap"], alibi_slopes=s["slopes"], key_range=s["range"],
                   window=c["window"])
        if s["q"].dim() == 3:
            o, lse = (gqa.decode_paged(s["q"], s["k"], s["v"], s["table"], return_lse=True, **how) if c["page"]
                      else gqa.decode(s["q"], s["k"], s["v"], return_lse=True, **how))
            return {"o": o, "lse": lse}
        how.update(q_start=s["lens"] - c["S"], causal=c["causal"])
        o, lse = gqa.prefill(s["q"], s["k"], s["v"], return_lse=True, **how)
        if not c["grad"]:
            return {"o": o, "lse": lse}
        dq, dk, dv = gqa.prefill_backward(s["q"], s["k"], s["v"], o, s["do"], lse, **how)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if c["op"] == "weights":
        how = dict(kv_len=s["lens"], window=c["window"], weights=s["w"] if c["accumulate"] else None)
        if c["page"]:
            return gqa.kv_weights_paged(s["q"], s["k"], s["table"], s["lse"], **how)
        return gqa.kv_weights(s["q"], s["k"], s["lse"], **how)
    how = dict(kv_len=s["lens"], sink=c["sink"], recent=c["recent"], weights_out=s["w_out"])
    if c["page"]:
        kept, new_len = gqa.kv_evict_paged(s["k"], s["v"], s["table"], s["w"], c["budget"],
                                           block_table_out=s["table_out"], **how)
        return {"k": s["k"], "v": s["v"], "w": s["w_out"], "kept": kept, "len": new_len}
    kept, new_len = gqa.kv_evict(s["k"], s["v"], s["w"], c["budget"], k_out=s["k_out"], v_out=s["v_out"], **how)
    return {"k": s["k_out"], "v": s["v_out"], "w": s["w_out"], "kept": kept, "len": new_len}


def run(s):
    return _called(s) if own else _plain(s)


# ------------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ------------------------------------------------------------------------------------------------
def _rotate64(x, inv_freq, at, scale, offset, interleaved, sign):
    """One sequence x (h, S, d) as complex pairs times scale e^{i sign angle}."""
    m = inv_freq.numel()
    i = torch.arange(m, device="cuda")
    first, second = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + m + i)
    y = x.double().clone()
    z = torch.complex(y[..., first], y[..., second])
    z = z * torch.polar(torch.full((at.numel(), m), scale, dtype=torch.float64, device="cuda"),
                        sign * at.double()[:, None] * inv_freq[None, :])
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    B, S = c["B"], c.get("S", 0)
    if c["op"] == "rope":
        i = torch.arange(S, device="cuda")
        return torch.stack([_rotate64(s["x"][b], s["inv_freq"], int(s["positions"][b]) + i, s["scale"], c["offset"],
                                      c["interleaved"], -1.0 if c["inverse"] else 1.0) for b in range(B)])
    if c["op"] == "append":
        i = torch.arange(S, device="cuda")
        kc, vc, q = s["kc"].double(), s["vc"].double(), []
        for b in range(B):
            p = int(s["pos"][b])
            how = (s["inv_freq"], p + i, s["scale"], 0, c["interleaved"], 1.0)
            q.append(_rotate64(s["q"][b], *how))
            k = _rotate64(s["k"][b], *how)
            if not c["page"]:
                kc[b, :, p:p + S], vc[b, :, p:p + S] = k, s["v"][b].double()
                continue
            for t0 in range(-(p % c["page"]), S, c["page"]):  # page by page
                lo, hi = max(t0, 0), min(t0 + c["page"], S)
                at, to = int(s["table"][b, (p + lo) // c["page"]]), (p + lo) % c["page"]
                kc[at, :, to:to + hi - lo], vc[at, :, to:to + hi - lo] = k[:, lo:hi], s["v"][b, :, lo:hi].double()
        return {"q": torch.stack(q), "k": kc, "v": vc}
    if c["op"] == "attend":
        names = ("q", "k", "v") if c["grad"] else ()
        outs = {n: [] for n in ("o", "lse", *("d" + n for n in names))}
        for b, n in enumerate(_lengths(c)):
            at = torch.arange(n - c["S"], n, device="cuda")[:, None]
            key = torch.arange(c["T"], device="cuda")[None, :]
            hidden = key >= n
            if c["causal"]:
                hidden = hidden | (key > at)
            if c["window"]:
                hidden = hidden | (at - key >= c["window"])
            if s["range"] is not None:
                hidden = hidden | (key < s["range"][b, :, :1]) | (key >= s["range"][b, :, 1:])
            group = {m: [] for m in outs}
            for g in range(c["h_kv"]):
                k, v = (s[m][s["table"][b].long(), g].reshape(-1, c["d"]) if c["page"] else s[m][b, g] for m in ("k", "v"))
                k, v = k.double(), v.double()
                sums = [torch.zeros_like(k), torch.zeros_like(v)]
                for a in range(g * c["h_q"] // c["h_kv"], (g + 1) * c["h_q"] // c["h_kv"]):
                    x = [t.detach().requires_grad_(c["grad"])
                         for t in (s["q"][b, a].reshape(c["S"], c["d"]).double(), k, v)]
                    z = torch.einsum("id,jd->ij", x[0], x[1]) * c["d"] ** -0.5
                    z = c["cap"] * torch.tanh(z / c["cap"]) if c["cap"] else z
                    z = z - s["slopes"][a].double() * (at - key).abs() if c["alibi"] else z
                    z = z.masked_fill(hidden, -math.inf)
                    o = torch.softmax(z, -1) @ x[2]
                    group["o"].append(o.detach())
                    group["lse"].append(torch.logsumexp(z, -1).detach())
                    if c["grad"]:
                        dq, dk, dv = torch.autograd.grad(o, x, s["do"][b, a].double())
                        group["dq"].append(dq)
                        sums = [sums[0] + dk, sums[1] + dv]
                if c["grad"]:
                    group["dk"].append(sums[0])
                    group["dv"].append(sums[1])
            for m in outs:
                outs[m].append(torch.stack(group[m]))
        outs = {m: torch.stack(t) for m, t in outs.items()}
        outs["o"], outs["lse"] = outs["o"].view(s["q"].shape), outs["lse"].view(s["q"].shape[:-1])
        return outs
    if c["op"] == "weights":
        w = s["w"].double() if c["accumulate"] else torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        q = s["q"].reshape(B, c["h_q"], c["S"], c["d"]).double()
        lse = s["lse"].reshape(B, c["h_q"], c["S"]).double()
        for b, n in enumerate(_lengths(c)):
            at = torch.arange(n - S, n, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")[None, :]
            hidden = key > at
            if c["window"]:
                hidden |= at - key >= c["window"]
            for a in range(c["h_q"]):
                g = a // (c["h_q"] // c["h_kv"])
                if c["page"]:
                    k = s["k"][s["table"][b].long(), g].reshape(-1, c["d"])[:n].double()
                else:
                    k = s["k"][b, g, :n].double()
                logp = torch.einsum("id,jd->ij", q[b, a], k) * c["d"] ** -0.5 - lse[b, a][:, None]
                w[b, g, :n] += logp.exp().masked_fill(hidden, 0.0).sum(0)
        return w
    kept = torch.full((B, c["h_kv"], c["budget"]), -1, dtype=torch.int32)
    w_out = torch.zeros(s["w_out"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        for g in range(c["h_kv"]):
            if n <= c["budget"]:
                keep = list(range(n))
            else:
                middle = range(c["sink"], n - c["recent"])
                w = s["w"][b, g].tolist()
                best = sorted(middle, key=lambda j: (-w[j], j))[:c["budget"] - c["sink"] - c["recent"]]
                keep = sorted([*range(c["sink"]), *best, *range(n - c["recent"], n)])
            at = torch.tensor(keep, device="cuda")
            m = len(keep)
            kept[b, g, :m] = at.to("cpu", torch.int32)
            w_out[b, g, :m] = s["w"][b, g, at].double()
            if c["page"]:
                p = c["page"]
                src, to = s["table"][b].long()[at // p], torch.arange(m, device="cuda")
                for name in ("k", "v"):
                    s[name][s["table_out"][b].long()[to // p], g, to % p] = s[name][src, g, at % p]
            else:
                s["k_out"][b, g, :m], s["v_out"][b, g, :m] = s["k"][b, g, at], s["v"][b, g, at]
    end = "" if c["page"] else "_out"
    new_len = torch.tensor([min(n, c["budget"]) for n in _lengths(c)], dtype=torch.int32)
    return {"k": s["k" + end].double(), "v": s["v" + end].double(), "w": w_out, "kept": kept, "len": new_len}
