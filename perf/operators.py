"""Cases of the serving operators around the sharded paged KV cache: attention of a chunk of new tokens over the cache,
the attention weight that each cached token has received, the eviction of the lightest tokens, and rotary positions.

``run`` makes one pass through an operator: in its plain form (elementary torch operations in 32 bits), or, where
``own`` is true, by the framework's call."""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------- cases

def _cache(Hq, Hkv, d, bs, I, pcp, dcp):
    return {"Hq": Hq, "Hkv": Hkv, "d": d, "bs": bs, "I": I, "pcp": pcp, "dcp": dcp}


def listed():
    wide = _cache(32, 8, 128, 128, 16, 2, 4)      # the decode benchmark's heads, blocks and 2 x 4 device grid
    return [
        # a handful of users, each waiting for one token: latency
        {"name": "chunk: 4 single tokens", "op": "chunk", **wide, "R": 4, "n_lo": 1, "n_hi": 1, "every": 1,
         "ctx_lo": 200, "ctx_hi": 2000, "lens": 1, "pad": 0},
        # a serving batch that verifies a few drafted tokens per request: the cache's bandwidth
        {"name": "chunk: drafts of 48 requests", "op": "chunk", **wide, "R": 48, "n_lo": 1, "n_hi": 6, "every": 1,
         "ctx_lo": 2048, "ctx_hi": 16384, "lens": 2, "pad": 0},
        # one piece of a chunked prefill: the tensor cores
        {"name": "chunk: 4096 of a prompt", "op": "chunk", **wide, "R": 1, "n_lo": 4096, "n_hi": 4096, "every": 1,
         "ctx_lo": 32768, "ctx_hi": 32768, "lens": 3, "pad": 0},
        # prefill pieces and decoding requests in one padded batch; small pages, an odd group, one device
        {"name": "chunk: mixed batch", "op": "chunk", **_cache(24, 8, 64, 16, 16, 1, 1), "R": 12, "n_lo": 300,
         "n_hi": 511, "every": 6, "ctx_lo": 600, "ctx_hi": 4099, "lens": 4, "pad": 5},
        # one user far into a long document: few rows, a long axis
        {"name": "chunk: a token at 131072", "op": "chunk", **wide, "R": 1, "n_lo": 1, "n_hi": 1, "every": 1,
         "ctx_lo": 131072, "ctx_hi": 131072, "lens": 5, "pad": 0},
        # the weights that a decode step adds
        {"name": "weights: 32 single tokens", "op": "weights", **wide, "R": 32, "n_lo": 1, "n_hi": 1, "every": 1,
         "ctx_lo": 2048, "ctx_hi": 16384, "lens": 6, "acc": True},
        # the last queries of a prompt vote on what the cache keeps of it
        {"name": "weights: last 64 of prompts", "op": "weights", **wide, "R": 4, "n_lo": 64, "n_hi": 64, "every": 1,
         "ctx_lo": 8192, "ctx_hi": 16384, "lens": 7, "acc": False},
        # two short chats over their budget, small odd caches
        {"name": "evict: 2 short requests", "op": "evict", **_cache(8, 2, 64, 32, 32, 1, 1), "R": 2, "ctx_lo": 900,
         "ctx_hi": 1301, "lens": 8, "keep": 512, "sink": 4, "recent": 129, "dt": "float32"},
        # a batch of prompts cut to a budget after their prefill
        {"name": "evict: 16 prompts to 2048", "op": "evict", **wide, "R": 16, "ctx_lo": 8192, "ctx_hi": 16384,
         "lens": 9, "keep": 2048, "sink": 4, "recent": 256, "dt": "bfloat16"},
        # q and k heads of one decode step, part of the head, pairs side by side
        {"name": "rope: decode step", "op": "rope", "rows": 64, "H": 40, "extra": 8, "d": 128, "rot": 64,
         "style": "interleaved", "scaling": "none", "factor": 1.0, "far": 131072, "backward": False,
         "dt": "bfloat16"},
        # q and k of a long prompt out of the fused projection, whole head, scaled to four times the trained length
        {"name": "rope: 32768 of a prompt", "op": "rope", "rows": 32768, "H": 40, "extra": 8, "d": 128, "rot": 128,
         "style": "half", "scaling": "yarn", "factor": 4.0, "far": 131072, "backward": False, "dt": "bfloat16"},
        # the gradient on its way back through the rotation, 32 bits, odd sizes
        {"name": "rope: gradient", "op": "rope", "rows": 8191, "H": 13, "extra": 0, "d": 80, "rot": 40,
         "style": "interleaved", "scaling": "linear", "factor": 8.0, "far": 32768, "backward": True,
         "dt": "float32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "weights", "evict", "rope"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 192, 256])
        c = {"op": op, "rows": _log(rng, 1, 32768), "H": rng.randint(1, 48), "extra": rng.choice([0, 0, 8, 3]), "d": d,
             "rot": rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]),
             "style": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
             "factor": float(rng.choice([2, 4, 8, 16])), "far": _log(rng, 1000, 1000000),
             "backward": rng.random() < 0.4, "dt": rng.choice(["bfloat16", "float32"])}
        while c["rows"] * c["H"] * d * (2 if c["dt"] == "bfloat16" else 4) > 300e6:
            c["rows"] = c["rows"] * 2 // 3
        return c
    Hkv = rng.choice([1, 2, 4, 8])
    bs = rng.choice([16, 32, 64, 128])
    I = rng.choice([i for i in (1, 4, 16, 32, 64, 128) if bs % i == 0])
    pcp, dcp = rng.choice([(1, 1), (1, 1), (2, 1), (1, 4), (2, 4)])
    c = {"op": op, **_cache(Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv, rng.choice([64, 128]), bs, I, pcp, dcp)}
    hi = _log(rng, 64, 32768)
    c.update(R=_log(rng, 1, 64), ctx_lo=max(1, int(hi * rng.uniform(0.1, 1.0))), ctx_hi=hi, lens=rng.randrange(1 << 20))
    if op == "evict":
        c["dt"] = rng.choice(["bfloat16", "bfloat16", "float32"])
        c["keep"] = max(8, int(hi * rng.uniform(0.05, 0.9)))
        c["sink"] = rng.choice([0, 1, 4])
        c["recent"] = rng.randint(0, c["keep"] - c["sink"])
    else:
        n = rng.choice([1, rng.randint(2, 8), _log(rng, 8, 4096)])
        c.update(n_lo=max(1, n // 2), n_hi=n, every=rng.choice([1, 1, 3, 6]))
        c["ctx_lo"], c["ctx_hi"] = max(c["ctx_lo"], n), max(c["ctx_hi"], n)
        c["pad" if op == "chunk" else "acc"] = rng.choice([0, 0, 7]) if op == "chunk" else rng.random() < 0.5
    while c["R"] > 1 and _cost(c) > 1.0:
        c["R"] = max(1, c["R"] * 2 // 3)
    while _cost(c) > 1.0:
        c["n_lo"], c["n_hi"] = max(1, c["n_lo"] * 2 // 3), max(1, c["n_hi"] * 2 // 3)
    return c


def _cost(c):
    """The plain form's work against what the largest listed cases take (1.0)."""
    tokens = c["R"] * c["ctx_hi"] * c["Hkv"] * c["d"] / (48 * 16384 * 8 * 128)
    pairs = c["R"] * c.get("n_hi", 0) * c["Hq"] * c["ctx_hi"] * c["d"] / (4096 * 32 * 32768 * 128)
    return max(tokens, pairs)


def _lens(c):
    """Contexts and new tokens of each request: part of the case, not of its inputs."""
    rng = random.Random(c["lens"])
    ctx = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["R"])]
    n = [rng.randint(c["n_lo"], c["n_hi"]) if r % c["every"] == 0 else 1 for r in range(c["R"])] if "n_lo" in c else []
    return ctx, [min(a, b) for a, b in zip(n, ctx)]


def work(case):
    c = case
    if c["op"] == "rope":
        size = 2 if c["dt"] == "bfloat16" else 4
        return {"bytes": 2 * c["rows"] * c["H"] * c["d"] * size + 4 * c["rows"], "flops": 3 * c["rows"] * c["H"] * c["rot"]}
    ctx, n = _lens(c)
    tokens = sum(ctx) * c["Hkv"]
    if c["op"] == "evict":
        size = 2 if c["dt"] == "bfloat16" else 4
        kept = sum(min(x, c["keep"]) for x in ctx) * c["Hkv"]
        return {"bytes": 4 * tokens + 2 * kept * (2 * c["d"] * size + 4) + 4 * c["R"] * c["Hkv"] * c["keep"], "flops": 0}
    pairs = sum(k * x - k * (k - 1) // 2 for x, k in zip(ctx, n)) * c["Hq"]
    rows = sum(n) * c["Hq"]
    if c["op"] == "chunk":
        return {"bytes": tokens * c["d"] * 4 + rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs}
    return {"bytes": tokens * (2 * c["d"] + (8 if c["acc"] else 4)) + rows * (2 * c["d"] + 4), "flops": 2 * c["d"] * pairs}


# ---------------------------------------------------------------------- inputs

def _frequencies(c):
    """inv_freq (float64, on the host) and the factor on cos and sin."""
    rot, s = c["rot"], c["factor"]
    half, base = rot // 2, 10000.0
    if c["scaling"] == "ntk" and rot > 2:
        base *= s ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(half)]
    if c["scaling"] == "linear":
        f = [x / s for x in f]
    if c["scaling"] == "yarn":
        turns = [max(0.0, min(1.0, (32768 * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
        f = [x * g + x / s * (1.0 - g) for x, g in zip(f, turns)]
        return torch.tensor(f, dtype=torch.float64), 0.1 * math.log(s) + 1.0
    return torch.tensor(f, dtype=torch.float64), 1.0


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "rope":
        dt = getattr(torch, c["dt"])
        rows = torch.randn(c["rows"], c["H"] + c["extra"], c["d"], generator=g, device=DEV, dtype=torch.float32).to(dt)
        start = torch.randint(0, max(1, c["far"] - c["rows"]), (1,), generator=g, device=DEV)
        pos = (start + torch.arange(c["rows"], device=DEV)) if c["rows"] > 64 else \
            torch.randint(0, c["far"], (c["rows"],), generator=g, device=DEV)
        f, m = _frequencies(c)
        return {"case": c, "x": rows[:, :c["H"]], "pos": pos.to(torch.int32), "f": f, "m": m, "f_dev": f.to(DEV)}

    ctx, n = _lens(c)
    R, W, V = c["R"], c["pcp"] * c["dcp"], c["bs"] * c["pcp"] * c["dcp"]
    nvb = [-(-x // V) for x in ctx]
    more = -(-min(c["keep"], max(ctx)) // V) if c["op"] == "evict" else 0   # fresh blocks that take what is kept
    num_blocks = sum(nvb) + R * more + 3
    perm = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((R, max(nvb) + 1), -1, dtype=torch.int32)
    at = 0
    for r in range(R):
        table[r, :nvb[r]] = perm[at:at + nvb[r]]
        at += nvb[r]
    dt = getattr(torch, c.get("dt", "bfloat16"))
    shape = (W, num_blocks, c["Hkv"], c["bs"], c["d"])
    s = {"case": c, "table": table.to(DEV), "ctx": torch.tensor(ctx, dtype=torch.int32, device=DEV), "N": max(ctx),
         "k": torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)}
    if c["op"] != "weights":
        s["v"] = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)
    if c["op"] == "evict":
        # attention weights are positive, a few heavy ones among many light ones, and repeat where they are tiny
        w = torch.empty(shape[:4], dtype=torch.float32, device=DEV).normal_(generator=g)
        s["w"] = (w * 2.0).exp().mul_(64).floor_().div_(64)
        s["dst"] = perm[at:at + R * more].view(R, more).to(DEV)
        return s
    qsl = [0]
    for k in n:
        qsl.append(qsl[-1] + k)
    T = qsl[-1] + c.get("pad", 0)
    s["q"] = torch.empty((T, c["Hq"], c["d"]), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    s["qsl"] = torch.tensor(qsl, dtype=torch.int32, device=DEV)
    s["n_max"] = max(n)
    if c["op"] == "chunk":
        s["o"] = torch.zeros((T, c["Hq"], c["d"]), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, c["Hq"]), dtype=torch.float32, device=DEV)
        s["ws"] = torch.empty(128 << 20, dtype=torch.uint8, device=DEV)   # scratch that a program keeps beside its cache
        return s
    sc, rows, fits = _scores(s)
    s["lse"] = torch.zeros((T, c["Hq"]), dtype=torch.float32, device=DEV)
    s["lse"][rows] = torch.logsumexp(sc, -1).view(R, c["Hq"], -1).transpose(1, 2)[fits]
    s["w_in"] = torch.rand(shape[:4], generator=g, device=DEV) * 3 if c["acc"] else None
    s["w_out"] = torch.zeros(shape[:4], device=DEV)
    return s


# ---------------------------------------------------------------------- plain forms

def _where(c, table, N):
    """Device [N], block [R, N] and slot [N] of the tokens 0..N-1 of every request."""
    W = c["pcp"] * c["dcp"]
    x = torch.arange(N, device=DEV)
    o = x % (c["bs"] * W)
    lbi = o // c["I"]
    return lbi % W, table[:, x // (c["bs"] * W)].long().clamp_(min=0), lbi // W * c["I"] + o % c["I"]


def _scores(s):
    """Scaled masked scores [R, Hkv, G * n_max, N], the batch rows of the queries that there are, and which those are."""
    c = s["case"]
    R, Hkv, G = c["R"], c["Hkv"], c["Hq"] // c["Hkv"]
    dev, blk, off = _where(c, s["table"], s["N"])
    k = s["k"][dev, blk, :, off].float()                                          # [R, N, Hkv, d]
    start, n = s["qsl"][:-1].long(), (s["qsl"][1:] - s["qsl"][:-1]).long()
    i = torch.arange(s["n_max"], device=DEV)
    fits = i < n[:, None]
    row = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(R, -1, Hkv, G, c["d"]).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, c["d"])
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(c["d"]))
    x = torch.arange(s["N"], device=DEV)
    sees = x <= (s["ctx"].long() - n)[:, None, None] + i[:, None]                 # [R, n_max, N]
    sees = (sees & (x < s["ctx"][:, None, None]))[:, None, None]
    return sc.view(R, Hkv, G, s["n_max"], -1).masked_fill_(~sees, -math.inf).view(sc.shape), row[fits], fits


def _chunk(s):
    c = s["case"]
    sc, rows, fits = _scores(s)
    dev, blk, off = _where(c, s["table"], s["N"])
    v = s["v"][dev, blk, :, off].float()
    v = v.masked_fill_((torch.arange(s["N"], device=DEV) >= s["ctx"][:, None])[:, :, None, None], 0.0)
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / l
    heads = (c["R"], c["Hq"], -1)
    s["o"][rows] = o.view(*heads, c["d"]).transpose(1, 2)[fits].to(s["o"].dtype)
    s["lse"][rows] = (m + l.log()).view(heads).transpose(1, 2)[fits]
    return s["o"], s["lse"]


def _weights(s):
    c = s["case"]
    sc, rows, fits = _scores(s)
    lse = torch.full((c["R"], s["n_max"], c["Hq"]), math.inf, device=DEV)
    lse[fits] = s["lse"][rows]
    lse = lse.transpose(1, 2).reshape(c["R"], c["Hkv"], -1, 1)
    w = (sc - lse).exp_().sum(2, dtype=torch.float64).transpose(1, 2)             # [R, N, Hkv]
    dev, blk, off = _where(c, s["table"], s["N"])
    x = torch.arange(s["N"], device=DEV)
    n = (s["qsl"][1:] - s["qsl"][:-1])[:, None]
    if s["w_in"] is not None:
        old = s["w_in"][dev, blk, :, off]
        w = w + old * (x < s["ctx"][:, None] - n)[:, :, None]
    live = x < s["ctx"][:, None]
    dev, off = dev.expand_as(blk)[live], off.expand_as(blk)[live]
    s["w_out"][dev, blk[live], :, off] = w[live].float()
    return s["w_out"]


def _evict(s):
    c = s["case"]
    R, Hkv, keep, N = c["R"], c["Hkv"], c["keep"], s["N"]
    dev, blk, off = _where(c, s["table"], N)
    x = torch.arange(N, device=DEV)
    ctx = s["ctx"].long()[:, None]
    w = s["w"][dev, blk, :, off].transpose(1, 2)                                  # [R, Hkv, N]
    stays = ((x < c["sink"]) | (x >= ctx - c["recent"]) | (ctx <= keep))[:, None] & (x < ctx)[:, None]
    rank = torch.where(stays, math.inf, w).masked_fill((x >= ctx)[:, None], -math.inf)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = torch.minimum(ctx, torch.tensor(keep, device=DEV))
    first = torch.sort(torch.where(torch.arange(first.shape[-1], device=DEV) < new[:, None], first, N), dim=-1).values
    n = first.shape[-1]
    kept = torch.full((R, Hkv, keep), -1, dtype=torch.int32, device=DEV)
    kept[..., :n] = torch.where(first < N, first, -1)
    live = first < N                                                              # [R, Hkv, n]
    r, h, j = (t.expand(R, Hkv, n)[live] for t in (torch.arange(R, device=DEV)[:, None, None],
                                                    torch.arange(Hkv, device=DEV)[:, None], torch.arange(n, device=DEV)))
    t = first[live]
    ddev, dblk, doff = _where(c, s["dst"], n)
    src, dst = (dev[t], blk[r, t], h, off[t]), (ddev[j], dblk[r, j], h, doff[j])
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    s["w"][dst] = s["w"][src]
    return kept, new[:, 0].to(torch.int32), s["k"], s["v"], s["w"]


def _rope(s):
    c = s["case"]
    a = s["pos"].double()[:, None] * s["f_dev"]
    cos, sin = ((t(a) * s["m"]).float()[:, None] for t in (torch.cos, torch.sin))
    sin = -sin if c["backward"] else sin
    x = s["x"][..., :c["rot"]].float()
    if c["style"] == "half":
        u, v = x[..., :c["rot"] // 2], x[..., c["rot"] // 2:]
        y = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    else:
        u, v = x[..., 0::2], x[..., 1::2]
        y = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    return torch.cat([y.to(s["x"].dtype), s["x"][..., c["rot"]:]], -1)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"chunk": _chunk, "weights": _weights, "evict": _evict, "rope": _rope}[c["op"]](s)
    from context_long_sequence_ring_gb300 import ringattn as ra
    if c["op"] == "rope":
        return ra.rope_apply(s["x"], s["pos"], s["f"], mscale=s["m"], style=c["style"], backward=c["backward"])
    if c["op"] == "chunk":
        return ra.cp_chunk_attn(s["q"], s["k"], s["v"], s["table"], s["qsl"], s["ctx"], c["I"], c["pcp"], c["dcp"],
                                workspace=s["ws"], o=s["o"], lse=s["lse"])
    if c["op"] == "weights":
        return ra.cp_attn_weights(s["q"], s["lse"], s["k"], s["table"], s["qsl"], s["ctx"], c["I"], c["pcp"], c["dcp"],
                                  w_in=s["w_in"], w_out=s["w_out"])
    kept, new = ra.cp_evict(s["k"], s["v"], s["w"], s["table"], s["ctx"], c["keep"], c["I"], c["pcp"], c["dcp"],
                            n_sink=c["sink"], n_recent=c["recent"], dst_block_table=s["dst"])
    return kept, new, s["k"], s["v"], s["w"]


# ---------------------------------------------------------------------- from the definitions, in 64 bits

def _slots(c, row, tokens):
    """(device, block, slot) lists of some tokens of the request whose block table row is given."""
    W = c["pcp"] * c["dcp"]
    vb, o = tokens // (c["bs"] * W), tokens % (c["bs"] * W)
    piece = o // c["I"]
    return piece % W, row[vb].long(), piece // W * c["I"] + o % c["I"]


def exact(case, seed):
    c = case
    if c["op"] in ("chunk", "weights") and work(c)["flops"] > 4e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        x, half = s["x"].double(), c["rot"] // 2
        turn = torch.polar(torch.full((), s["m"], dtype=torch.float64, device=DEV),
                           (-1.0 if c["backward"] else 1.0) * s["pos"].double()[:, None] * s["f_dev"])[:, None]
        a, b = (slice(0, half), slice(half, c["rot"])) if c["style"] == "half" else (slice(0, c["rot"], 2), slice(1, c["rot"], 2))
        z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
        y = x.clone()
        y[..., a], y[..., b] = z.real, z.imag
        return y
    ctx, n = _lens(c)
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "evict":
        k, v, w = (t.double() for t in (s["k"], s["v"], s["w"]))
        kept = torch.full((c["R"], c["Hkv"], c["keep"]), -1, dtype=torch.int32)
        for r in range(c["R"]):
            pos = torch.arange(ctx[r], device=DEV)
            dev, blk, off = _slots(c, s["table"][r], pos)
            for h in range(c["Hkv"]):
                wt = w[dev, blk, h, off]
                ids = pos
                if ctx[r] > c["keep"]:
                    mid = pos[c["sink"]:ctx[r] - c["recent"]]
                    # heavier first, and of equal ones the earlier: sort by index, then stably by weight
                    order = torch.argsort(-wt[mid], stable=True)[:c["keep"] - c["sink"] - c["recent"]]
                    ids = torch.cat([pos[:c["sink"]], mid[order].sort().values, pos[ctx[r] - c["recent"]:]])
                kept[r, h, :len(ids)] = ids.to(torch.int32).cpu()
                a = _slots(c, s["dst"][r], torch.arange(len(ids), device=DEV))
                b = (dev[ids], blk[ids], off[ids])
                for t in (k, v, w):
                    t[a[0], a[1], h, a[2]] = t[b[0], b[1], h, b[2]]
        return kept, torch.tensor([min(x, c["keep"]) for x in ctx], dtype=torch.int32), k, v, w
    out = torch.zeros((s["q"].shape[0], c["Hq"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["q"].shape[0], c["Hq"]), dtype=torch.float64, device=DEV)
    w_out = torch.zeros(s["k"].shape[:4], dtype=torch.float64, device=DEV)
    first = 0
    for r in range(c["R"]):
        pos = torch.arange(ctx[r], device=DEV)
        dev, blk, off = _slots(c, s["table"][r], pos)
        hidden = pos > torch.arange(ctx[r] - n[r], ctx[r], device=DEV)[:, None]
        for h in range(c["Hq"]):
            key = s["k"][dev, blk, h // G, off].double()
            a = s["q"][first:first + n[r], h].double() @ key.T / c["d"] ** 0.5
            a[hidden] = -math.inf
            if c["op"] == "chunk":
                lse[first:first + n[r], h] = torch.logsumexp(a, -1)
                out[first:first + n[r], h] = torch.softmax(a, -1) @ s["v"][dev, blk, h // G, off].double()
            else:
                a = torch.exp(a - s["lse"][first:first + n[r], h].double()[:, None]).sum(0)
                w_out[dev, blk, h // G, off] += a
        if c["op"] == "weights" and c["acc"]:
            old = pos[:ctx[r] - n[r]]
            dev, blk, off = _slots(c, s["table"][r], old)
            w_out[dev, blk, :, off] += s["w_in"][dev, blk, :, off].double()
        first += n[r]
    return (out, lse) if c["op"] == "chunk" else w_out
