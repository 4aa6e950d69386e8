"""Cases of attention with a sliding window and first tokens that stay visible, over the paged cache and on packed
sequences with its gradient, of the store that rotates new keys on their way into the cache, and of rotary positions
with several axes.

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
    heads = {"Hq": 32, "Hkv": 8, "d": 128}
    return [
        # one decode step of a serving batch: q, k and v of 48 new tokens; latency
        {"name": "append: 48 single tokens", "op": "append", **wide, "R": 48, "n_lo": 1, "n_hi": 1, "every": 1,
         "ctx_lo": 2048, "ctx_hi": 16384, "lens": 1, "rot": 128, "style": "half", "scaling": "yarn", "factor": 4.0,
         "sections": "", "ladder": "shared", "dt": "bfloat16"},
        # a piece of a long prompt out of the fused projection: bandwidth
        {"name": "append: 16384 of a prompt", "op": "append", **wide, "R": 1, "n_lo": 16384, "n_hi": 16384, "every": 1,
         "ctx_lo": 32768, "ctx_hi": 32768, "lens": 2, "rot": 128, "style": "half", "scaling": "none", "factor": 1.0,
         "sections": "", "ladder": "shared", "dt": "bfloat16"},
        # pieces of prompts with pictures among single tokens, 32 bits, half the head, small pages, an odd group
        {"name": "append: mixed batch", "op": "append", **_cache(6, 2, 80, 16, 4, 1, 2), "R": 13, "n_lo": 60,
         "n_hi": 333, "every": 4, "ctx_lo": 340, "ctx_hi": 2001, "lens": 3, "rot": 40, "style": "interleaved",
         "scaling": "linear", "factor": 8.0, "sections": "8,6,6", "ladder": "shared", "dt": "float32"},
        # q and k heads of the frames of a film: time, height and width take the frequencies in sections
        {"name": "axes: frames of a film", "op": "axes", "grid": "20,36,44", "H": 40, "extra": 8, "d": 128, "rot": 128,
         "style": "half", "scaling": "none", "factor": 1.0, "sections": "16,24,24", "ladder": "shared",
         "backward": False, "dt": "bfloat16"},
        # the gradient of a picture's patches, height and width with frequencies of their own, 32 bits, odd sizes
        {"name": "axes: gradient of a picture", "op": "axes", "grid": "1,37,53", "H": 13, "extra": 0, "d": 72, "rot": 64,
         "style": "interleaved", "scaling": "none", "factor": 1.0, "sections": "0,16,16", "ladder": "own",
         "backward": True, "dt": "float32"},
        # a handful of users, each waiting for one token: latency
        {"name": "window: 4 single tokens", "op": "window", **wide, "R": 4, "n_lo": 1, "n_hi": 1, "every": 1,
         "ctx_lo": 200, "ctx_hi": 6000, "lens": 6, "window": 1024, "sink": 4, "pad": 0},
        # a serving batch far into its texts, of which the window and the first tokens are kept: the cache's bandwidth
        {"name": "window: 64 single tokens", "op": "window", **wide, "R": 64, "n_lo": 1, "n_hi": 1, "every": 1,
         "ctx_lo": 16384, "ctx_hi": 131072, "lens": 7, "window": 4096, "sink": 4, "pad": 0},
        # one piece of a chunked prefill: the tensor cores
        {"name": "window: 4096 of a prompt", "op": "window", **wide, "R": 1, "n_lo": 4096, "n_hi": 4096, "every": 1,
         "ctx_lo": 32768, "ctx_hi": 32768, "lens": 8, "window": 4096, "sink": 4, "pad": 0},
        # prefill pieces and decoding requests in one padded batch; small pages, an odd group, an odd window
        {"name": "window: mixed batch", "op": "window", **_cache(24, 8, 64, 16, 16, 1, 1), "R": 12, "n_lo": 300,
         "n_hi": 511, "every": 6, "ctx_lo": 600, "ctx_hi": 4099, "lens": 9, "window": 501, "sink": 1, "pad": 5},
        # a whole prompt at once, out of the fused projection
        {"name": "packed: 32768 of a prompt", "op": "packed", **heads, "R": 1, "n_lo": 32768, "n_hi": 32768, "lens": 10,
         "window": 4096, "sink": 4, "train": False},
        # a step of long-context training: forward and backward
        {"name": "packed: training step", "op": "packed", **heads, "R": 3, "n_lo": 2000, "n_hi": 9000, "lens": 11,
         "window": 2048, "sink": 0, "train": True},
        # documents of odd lengths packed to a short step, heads of 64 in groups of three
        {"name": "packed: short documents", "op": "packed", "Hq": 6, "Hkv": 2, "d": 64, "R": 9, "n_lo": 1, "n_hi": 700,
         "lens": 12, "window": 257, "sink": 4, "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotation(rng, d):
    """Rotated part, pairing, frequencies and how 0, 2 or 3 axes share them; rot a multiple of 8 bytes' pairs."""
    rot = rng.choice([d, d, 16 * rng.randint(1, d // 16)])
    half = rot // 2
    kind = rng.choice([0, 0, 2, 3])
    if kind == 0:
        sections = ""
    else:
        a = rng.randint(1, half - 2)
        b = rng.randint(1, half - a - 1) if kind == 3 else half - a
        sections = "%d,%d,%d" % ((0, a, b) if kind == 2 else (a, b, half - a - b))
    return {"rot": rot, "style": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
            "factor": float(rng.choice([2, 4, 8])), "sections": sections, "ladder": rng.choice(["shared", "own"]),
            "dt": rng.choice(["bfloat16", "bfloat16", "float32"])}


def draw(rng):
    op = rng.choice(["append", "axes", "window", "window", "packed", "packed"])
    if op == "axes":
        d = rng.choice([32, 64, 72, 80, 96, 128, 192, 256])
        c = {"op": op, **_draw_rotation(rng, d), "H": rng.randint(1, 48), "extra": rng.choice([0, 0, 8, 3]), "d": d,
             "backward": rng.random() < 0.4}
        if not c["sections"]:
            c["sections"] = "%d,%d,%d" % (c["rot"] // 2 - 2, 1, 1)
        grid = [_log(rng, 1, 30), _log(rng, 1, 64), _log(rng, 1, 64)]
        while grid[0] * grid[1] * grid[2] * c["H"] * d * (2 if c["dt"] == "bfloat16" else 4) > 300e6:
            grid = [-(-g * 2 // 3) for g in grid]
        c["grid"] = "%d,%d,%d" % tuple(grid)
        return c
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "packed":
        n = _log(rng, 8, 16384)        # a sequence of one token has no gradient of q and k to speak of
        c = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": rng.choice([64, 128]), "R": rng.choice([1, 1, 2, 5, 24]),
             "n_lo": rng.choice([n, 5, n // 2]), "n_hi": n, "lens": rng.randrange(1 << 20),
             "window": rng.choice([_log(rng, 3, 8192), _log(rng, 100, 4096), 1 << 30]),
             "sink": rng.choice([0, 1, 4, 4, 130]), "train": rng.random() < 0.7}
        while c["R"] > 1 and _cost(c) > 1.0:
            c["R"] = max(1, c["R"] * 2 // 3)
        while _cost(c) > 1.0:
            c["n_lo"], c["n_hi"] = max(4, c["n_lo"] * 2 // 3), c["n_hi"] * 2 // 3
        return c
    bs = rng.choice([16, 32, 64, 128])
    I = rng.choice([i for i in (1, 4, 16, 32, 64, 128) if bs % i == 0])
    pcp, dcp = rng.choice([(1, 1), (1, 1), (2, 1), (1, 4), (2, 4)])
    c = {"op": op, **_cache(Hq, Hkv, rng.choice([64, 128]), bs, I, pcp, dcp)}
    hi = _log(rng, 64, 65536)
    c.update(R=_log(rng, 1, 64), ctx_lo=max(1, int(hi * rng.uniform(0.1, 1.0))), ctx_hi=hi, lens=rng.randrange(1 << 20))
    n = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 8, 4096)])
    c.update(n_lo=max(1, n // 2), n_hi=n, every=rng.choice([1, 1, 3, 6]))
    c["ctx_lo"], c["ctx_hi"] = max(c["ctx_lo"], n), max(c["ctx_hi"], n)
    if op == "append":
        c["d"] = rng.choice([64, 80, 128])
        c.update(_draw_rotation(rng, c["d"]))
    else:
        c.update(window=rng.choice([_log(rng, 1, 8192), _log(rng, 128, 4096)]), sink=rng.choice([0, 1, 4, 4, 130]),
                 pad=rng.choice([0, 0, 7]))
    while c["R"] > 1 and _cost(c) > 1.0:
        c["R"] = max(1, c["R"] * 2 // 3)
    while _cost(c) > 1.0:
        c["n_lo"], c["n_hi"] = max(1, c["n_lo"] * 2 // 3), max(1, c["n_hi"] * 2 // 3)
    return c


def _cost(c):
    """The plain form's work against what the largest listed cases take (1.0)."""
    if c["op"] == "packed":
        pairs = c["R"] * c["n_hi"] * min(c["n_hi"], c["window"] + c["sink"]) * c["Hq"] * c["d"] * (3.5 if c["train"] else 1.0)
        tokens = c["R"] * c["n_hi"] * c["Hq"] * c["d"]
        return max(pairs / (32768 * 4096 * 32 * 128), tokens / (32768 * 32 * 128))
    if c["op"] == "append":
        cached = c["R"] * c["ctx_hi"] * c["Hkv"] * c["d"] / (64 * 16384 * 8 * 128)
        return max(cached, c["R"] * c["n_hi"] * (c["Hq"] + 2 * c["Hkv"]) * c["d"] / (16384 * 48 * 128))
    span = min(c["ctx_hi"], c["sink"] + c["window"] + c["n_hi"] - 1)
    tokens = c["R"] * span * c["Hkv"] * c["d"] / (64 * 4100 * 8 * 128)
    return max(tokens, c["R"] * c["n_hi"] * span * c["Hq"] * c["d"] / (4096 * 8196 * 32 * 128))


def _lens(c):
    """Contexts and new tokens of each request: part of the case, not of its inputs."""
    rng = random.Random(c["lens"])
    if c["op"] == "packed":
        n = [rng.randint(c["n_lo"], c["n_hi"]) for _ in range(c["R"])]
        return n, n
    ctx = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["R"])]
    n = [rng.randint(c["n_lo"], c["n_hi"]) if r % c["every"] == 0 else 1 for r in range(c["R"])]
    return ctx, [min(a, b) for a, b in zip(n, ctx)]


def _below(x, cap):
    """Sum of min(i, cap) over i = 1 .. x."""
    m = min(x, cap)
    return m * (m + 1) // 2 + (x - m) * cap


def _pairs(ctx, n, window, sink):
    """Visible (query, token) pairs of a head: positions ctx - n .. ctx - 1, each with its window and the first tokens."""
    in_window = _below(ctx, window) - _below(ctx - n, window)
    before = lambda x: _below(max(x - window, 0), sink)        # first tokens that have left the window of positions < x
    return in_window + before(ctx) - before(ctx - n)


def _seen(ctx, n, window, sink):
    """Tokens of a request that some query sees."""
    first = max(0, ctx - n - window + 1)
    return ctx - first + min(first, sink)


def work(case):
    c = case
    size = 2 if c.get("dt", "bfloat16") == "bfloat16" else 4
    if c["op"] == "axes":
        rows = math.prod(_grid(c))
        return {"bytes": 2 * rows * c["H"] * c["d"] * size + 12 * rows, "flops": 3 * rows * c["H"] * c["rot"]}
    ctx, n = _lens(c)
    T = sum(n)
    if c["op"] == "append":
        axes = 3 if c["sections"] else 1
        return {"bytes": T * (2 * (c["Hq"] + 2 * c["Hkv"]) * c["d"] * size + 4 * axes),
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    pairs = sum(_pairs(x, k, c["window"], c["sink"]) for x, k in zip(ctx, n)) * c["Hq"]
    rows = T * c["Hq"]
    if c["op"] == "window":
        tokens = sum(_seen(x, k, c["window"], c["sink"]) for x, k in zip(ctx, n)) * c["Hkv"]
        return {"bytes": tokens * c["d"] * 4 + rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs}
    kv = T * c["Hkv"] * c["d"] * 4
    if not c["train"]:
        return {"bytes": kv + rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs}
    return {"bytes": 2 * kv + rows * (8 * c["d"] + 4), "flops": 14 * c["d"] * pairs}


# ---------------------------------------------------------------------- inputs

def _grid(c):
    return [int(x) for x in c["grid"].split(",")]


def _frequencies(c):
    """inv_freq (float64, on the host), the axis of each of them (None: one axis) and the factor on cos and sin."""
    rot, s, base = c["rot"], c["factor"], 10000.0

    def ladder(n):
        b = base * s ** (n / (n - 1)) if c["scaling"] == "ntk" and n > 1 else base
        f = [b ** (-i / n) for i in range(n)]
        if c["scaling"] == "linear":
            f = [x / s for x in f]
        if c["scaling"] == "yarn":
            turns = [max(0.0, min(1.0, (32768 * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
            f = [x * g + x / s * (1.0 - g) for x, g in zip(f, turns)]
        return f

    m = 0.1 * math.log(s) + 1.0 if c["scaling"] == "yarn" else 1.0
    if not c["sections"]:
        return torch.tensor(ladder(rot // 2), dtype=torch.float64), None, m
    parts = [int(x) for x in c["sections"].split(",")]
    axis = torch.tensor([a for a, k in enumerate(parts) for _ in range(k)], dtype=torch.int32)
    f = ladder(rot // 2) if c["ladder"] == "shared" else [x for k in parts if k for x in ladder(k)]
    return torch.tensor(f, dtype=torch.float64), axis, m


def _table(c, ctx, n, g):
    """Block table: blocks in random order for the tokens that some query sees (all of them in the store), -1 elsewhere."""
    V = c["bs"] * c["pcp"] * c["dcp"]
    keep = []
    for x, k in zip(ctx, n):
        vbs = range(-(-x // V))
        if c["op"] == "window":
            first = max(0, x - k - c["window"] + 1)
            vbs = [b for b in vbs if b * V < min(c["sink"], x) or (b + 1) * V > first]
        keep.append(list(vbs))
    num_blocks = sum(len(b) for b in keep) + 3
    perm = torch.randperm(num_blocks, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(-(-x // V) for x in ctx) + 1), -1, dtype=torch.int32)
    at = 0
    for r, vbs in enumerate(keep):
        table[r, torch.tensor(vbs)] = perm[at:at + len(vbs)]
        at += len(vbs)
    return table, num_blocks


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, dt=torch.bfloat16):
        return torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)

    dt = getattr(torch, c.get("dt", "bfloat16"))
    s = {"case": c}
    if c["op"] in ("axes", "append"):
        s["f"], s["axis"], s["m"] = _frequencies(c)
        s["f_dev"] = s["f"].to(DEV)
        s["axis_dev"] = None if s["axis"] is None else s["axis"].long().to(DEV)
    if c["op"] == "axes":
        frames, height, width = _grid(c)
        rows = frames * height * width
        start = int(torch.randint(0, 4096, (1,), generator=torch.Generator().manual_seed(seed)))   # text before it
        i = torch.arange(rows, device=DEV)
        s["x"] = normal((rows, c["H"] + c["extra"], c["d"]), dt)[:, :c["H"]]
        s["pos"] = (start + torch.stack([i // (height * width), i // width % height, i % width])).to(torch.int32)
        return s

    ctx, n = _lens(c)
    T, Hq, Hkv, d = sum(n), c["Hq"], c["Hkv"], c["d"]
    qsl = [0]
    for k in n:
        qsl.append(qsl[-1] + k)
    s["qsl"] = torch.tensor(qsl, dtype=torch.int32, device=DEV)
    if c["op"] == "packed":
        x = normal((T, Hq + 2 * Hkv, d))           # out of the fused projection
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["n"], s["qsl_host"] = n, qsl
        s["ws"] = torch.empty(160 << 20, dtype=torch.uint8, device=DEV)   # scratch that a program keeps
        s["o"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device=DEV)
        if c["train"]:
            s["do"] = normal((T, Hq, d))
            dx = torch.zeros_like(x)               # the fused projection's gradient
            s["dq"], s["dk"], s["dv"] = dx[:, :Hq], dx[:, Hq:Hq + Hkv], dx[:, Hq + Hkv:]
        return s

    table, num_blocks = _table(c, ctx, n, torch.Generator().manual_seed(seed))
    shape = (c["pcp"] * c["dcp"], num_blocks, Hkv, c["bs"], d)
    s.update(table=table.to(DEV), ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV), n_max=max(n))
    if c["op"] == "append":
        s["kc"], s["vc"] = torch.zeros(shape, dtype=dt, device=DEV), torch.zeros(shape, dtype=dt, device=DEV)
        x = normal((T, Hq + 2 * Hkv, d), dt)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["qo"] = torch.zeros((T, Hq, d), dtype=dt, device=DEV)
        place = torch.cat([torch.arange(x - k, x) for x, k in zip(ctx, n)])
        # positions run on where a context has been cut; pictures give three of them
        pos = place + 1000
        s["pos"] = (pos if s["axis"] is None else torch.stack([pos, pos // 40, pos % 40])).to(torch.int32).to(DEV)
        return s
    s["kc"], s["vc"] = normal(shape), normal(shape)
    s["q"] = normal((T + c["pad"], Hq, d))
    s["o"] = torch.zeros((T + c["pad"], Hq, d), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((T + c["pad"], Hq), dtype=torch.float32, device=DEV)
    s["ws"] = torch.empty(128 << 20, dtype=torch.uint8, device=DEV)   # scratch that a program keeps beside its cache
    s["width"] = max(min(x, c["sink"] + c["window"] + k - 1) for x, k in zip(ctx, n))
    return s


# ---------------------------------------------------------------------- plain forms

def _where(c, x):
    """Device, virtual block and slot of tokens."""
    W = c["pcp"] * c["dcp"]
    o = x % (c["bs"] * W)
    lbi = o // c["I"]
    return lbi % W, x // (c["bs"] * W), lbi // W * c["I"] + o % c["I"]


def _turned(x, pos, s, backward=False):
    """The rotated heads x [rows, H, d] in 32 bits, rounded once; angles in 64 bits."""
    c = s["case"]
    m = pos.double()[:, None] if s["axis"] is None else pos.double()[s["axis_dev"]].T
    a = m * s["f_dev"]
    cos, sin = ((t(a) * s["m"]).float()[:, None] for t in (torch.cos, torch.sin))
    sin = -sin if backward else sin
    y = x[..., :c["rot"]].float()
    if c["style"] == "half":
        u, v = y[..., :c["rot"] // 2], y[..., c["rot"] // 2:]
        y = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    else:
        u, v = y[..., 0::2], y[..., 1::2]
        y = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., c["rot"]:]], -1)


def _append(s):
    c = s["case"]
    T = s["k"].shape[0]
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(s["qsl"].long(), t, right=True) - 1
    place = s["ctx"].long()[r] - (s["qsl"].long()[r + 1] - t)
    dev, vb, off = _where(c, place)
    at = (dev, s["table"][r, vb].long(), slice(None), off)
    s["kc"][at] = _turned(s["k"], s["pos"], s)
    s["vc"][at] = s["v"]
    s["qo"].copy_(_turned(s["q"], s["pos"], s))
    return s["qo"], s["kc"], s["vc"]


def _window(s):
    """The tokens that a request's queries see, first ones and window, side by side; then masked attention."""
    c = s["case"]
    R, Hkv, G, d, n_max = c["R"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"], s["n_max"]
    ctx, start = s["ctx"].long()[:, None], s["qsl"][:-1].long()[:, None]
    n = s["qsl"][1:].long()[:, None] - start
    lo = (ctx - n - c["window"] + 1).clamp_(min=0)                                 # first token of the request's windows
    i = torch.arange(s["width"], device=DEV)
    sinks = lo.clamp(max=c["sink"])
    x = torch.where(i < sinks, i, lo + i - sinks)                                   # [R, width] positions
    there = x < ctx
    dev, vb, off = _where(c, torch.where(there, x, 0))
    blk = s["table"].gather(1, vb).long().clamp_(min=0)
    k = s["kc"][dev, blk, :, off].float()                                           # [R, width, Hkv, d]
    v = s["vc"][dev, blk, :, off].float().masked_fill_(~there[..., None, None], 0.0)
    j = torch.arange(n_max, device=DEV)
    fits = j < n
    row = (start + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(R, n_max, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * n_max, d)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    at = (ctx - n + j)[:, :, None]                                                  # [R, n_max, 1] positions of the queries
    x = x[:, None]
    sees = there[:, None] & (x <= at) & ((x > at - c["window"]) | (x < c["sink"]))
    sc = sc.view(R, Hkv, G, n_max, -1).masked_fill_(~sees[:, None, None], -math.inf).view(sc.shape)
    m = sc.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = (sc - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / l
    s["o"][row[fits]] = o.view(R, c["Hq"], n_max, d).transpose(1, 2)[fits].to(s["o"].dtype)
    s["lse"][row[fits]] = (m + l.log()).view(R, c["Hq"], n_max).transpose(1, 2)[fits]
    return s["o"], s["lse"]


def _packed(s):
    """Blocks of queries of each sequence against the keys that they see."""
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G, scale, block = Hq // Hkv, 1.0 / math.sqrt(d), 1024
    if c["train"]:
        dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float32, device=DEV) for _ in range(2))
    for first, n in zip(s["qsl_host"], s["n"]):
        for b0 in range(0, n, block):
            b1 = min(n, b0 + block)
            lo = max(0, b0 - c["window"] + 1)
            x = torch.cat([torch.arange(min(c["sink"], lo), device=DEV), torch.arange(lo, b1, device=DEV)])
            i = torch.arange(b0, b1, device=DEV)[:, None]
            sees = (x <= i) & ((x > i - c["window"]) | (x < c["sink"]))
            rows = slice(first + b0, first + b1)
            k, v = (s[t][first + x].float().permute(1, 0, 2) for t in "kv")                # [Hkv, keys, d]
            q = s["q"][rows].float().view(-1, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
            sc = (torch.matmul(q, k.transpose(1, 2)) * scale).view(Hkv, G, b1 - b0, -1)
            sc = sc.masked_fill_(~sees, -math.inf).view(Hkv, G * (b1 - b0), -1)
            m = sc.amax(-1, keepdim=True)
            p = sc.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            p = p.div_(l)
            o = torch.matmul(p, v)
            back = lambda t: t.view(Hkv, G, b1 - b0, -1).permute(2, 0, 1, 3).reshape(b1 - b0, Hq, -1)
            s["o"][rows] = back(o).to(s["o"].dtype)
            s["lse"][rows] = back(m + l.log())[..., 0]
            if not c["train"]:
                continue
            do = s["do"][rows].float().view(-1, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
            dv.index_add_(0, first + x, torch.matmul(p.transpose(1, 2), do).permute(1, 0, 2))
            ds = torch.matmul(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            s["dq"][rows] = back(torch.matmul(ds, k)).to(s["dq"].dtype)
            dk.index_add_(0, first + x, torch.matmul(ds.transpose(1, 2), q).permute(1, 0, 2))
    if not c["train"]:
        return s["o"], s["lse"]
    s["dk"].copy_(dk)
    s["dv"].copy_(dv)
    return s["o"], s["lse"], s["dq"], s["dk"], s["dv"]


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "axes":
            return _turned(s["x"], s["pos"], s, c["backward"])
        return {"append": _append, "window": _window, "packed": _packed}[c["op"]](s)
    from context_long_sequence_ring_gb300 import ringattn as ra
    if c["op"] == "axes":
        return ra.rope_apply_axes(s["x"], s["pos"], s["f"], s["axis"], mscale=s["m"], style=c["style"], backward=c["backward"])
    if c["op"] == "append":
        ra.cp_rope_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["qsl"], s["ctx"], c["I"], c["pcp"], c["dcp"],
                          positions=s["pos"], inv_freq=s["f"], axis=s["axis"], mscale=s["m"], style=c["style"], q=s["q"],
                          q_out=s["qo"])
        return s["qo"], s["kc"], s["vc"]
    if c["op"] == "window":
        return ra.cp_window_attn(s["q"], s["kc"], s["vc"], s["table"], s["qsl"], s["ctx"], c["window"], c["I"], c["pcp"],
                                 c["dcp"], n_sink=c["sink"], workspace=s["ws"], o=s["o"], lse=s["lse"])
    o, lse = ra.window_attn_fwd(s["q"], s["k"], s["v"], s["qsl"], c["window"], n_sink=c["sink"], workspace=s["ws"],
                                o=s["o"], lse=s["lse"])
    if not c["train"]:
        return o, lse
    dq, dk, dv = ra.window_attn_bwd(s["do"], s["q"], s["k"], s["v"], o, lse, s["qsl"], c["window"], n_sink=c["sink"],
                                    workspace=s["ws"], dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return o, lse, dq, dk, dv


# ---------------------------------------------------------------------- from the definitions, in 64 bits

def _turn64(x, pos, s, backward):
    """Pairs as complex numbers, times m e^{i angle}."""
    c = s["case"]
    half = c["rot"] // 2
    x = x.double()
    per_pair = pos.double().expand(half, -1) if s["axis"] is None else torch.stack([pos[int(a)].double() for a in s["axis"]])
    sign = -1.0 if backward else 1.0
    turn = torch.polar(torch.full((), s["m"], dtype=torch.float64, device=DEV), sign * per_pair.T * s["f_dev"])[:, None]
    a, b = (slice(0, half), slice(half, c["rot"])) if c["style"] == "half" else (slice(0, c["rot"], 2), slice(1, c["rot"], 2))
    z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _rows(c, row, tokens):
    """(device, block, slot) of some tokens of the request whose block table row is given."""
    V = c["bs"] * c["pcp"] * c["dcp"]
    piece = tokens % V // c["I"]
    W = c["pcp"] * c["dcp"]
    return piece % W, row[tokens // V].long(), piece // W * c["I"] + tokens % V % c["I"]


def exact(case, seed):
    c = case
    if c["op"] in ("window", "packed") and work(c)["flops"] > 4e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "axes":
        return _turn64(s["x"], s["pos"], s, c["backward"])
    ctx, n = _lens(c)
    if c["op"] == "append":
        kc, vc = s["kc"].double(), s["vc"].double()
        k, t = _turn64(s["k"], s["pos"], s, False), 0
        for r in range(c["R"]):
            dev, blk, off = _rows(c, s["table"][r], torch.arange(ctx[r] - n[r], ctx[r], device=DEV))
            kc[dev, blk, :, off] = k[t:t + n[r]]
            vc[dev, blk, :, off] = s["v"][t:t + n[r]].double()
            t += n[r]
        return _turn64(s["q"], s["pos"], s, False), kc, vc
    T, Hq, d = s["q"].shape
    G, train = Hq // c["Hkv"], c.get("train", False)
    o = torch.zeros((T, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=DEV)
    grads = [torch.zeros((T, h, d), dtype=torch.float64, device=DEV) for h in (Hq, c["Hkv"], c["Hkv"])] if train else []
    first = 0
    for r in range(c["R"]):
        before = ctx[r] - n[r]
        for h in range(Hq):
            for b0 in range(0, n[r], 2048):
                b1 = min(n[r], b0 + 2048)
                at = torch.arange(before + b0, before + b1, device=DEV)[:, None]
                far = max(0, before + b0 - c["window"] + 1)
                tok = torch.arange(before + b1, device=DEV)
                tok = tok[(tok < c["sink"]) | (tok >= far)]                # the others are hidden from all of these queries
                hidden = (tok > at) | ((tok <= at - c["window"]) & (tok >= c["sink"]))
                q = s["q"][first + b0:first + b1, h].double()
                if c["op"] == "window":
                    dev, blk, off = _rows(c, s["table"][r], tok)
                    k, v = (s[t][dev, blk, h // G, off].double() for t in ("kc", "vc"))
                else:
                    k, v = (s[t][first + tok, h // G].double() for t in "kv")
                leaves = [t.requires_grad_(train) for t in (q, k, v)]
                a = (q @ k.T / d ** 0.5).masked_fill(hidden, -math.inf)
                y = torch.softmax(a, -1) @ v
                if train:
                    gq, gk, gv = torch.autograd.grad(y, leaves, s["do"][first + b0:first + b1, h].double())
                    grads[0][first + b0:first + b1, h] = gq
                    grads[1][:, h // G].index_add_(0, first + tok, gk)
                    grads[2][:, h // G].index_add_(0, first + tok, gv)
                o[first + b0:first + b1, h] = y.detach()
                lse[first + b0:first + b1, h] = torch.logsumexp(a.detach(), -1)
        first += n[r]
    return (o, lse, *grads)
