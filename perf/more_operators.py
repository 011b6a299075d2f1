"""The operators of a serving step around the paged cache, as cases to measure: queries and keys normed per head and
rotated by their positions (lora_qk_rope), the same with the keys and values going into their cache slots
(lora_kv_append), one new token per sequence that sees a sliding window and some first tokens (lora_attn_decode_window),
and chunks of new tokens over the paged cache (lora_attn_chunk).

Each case is a dict of sizes; `prepare` makes its inputs on the GPU from a seed, `run` makes one pass through the
operator (`own`: through the framework's entry points; otherwise in elementary torch operations in 32 bits, angles in
64, rounded once at the end), and `exact` gives the same outputs from the definition in 64 bits.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
DECODE_WORKSPACE = 16 << 20   # scratch of the decode call, zero-filled once by the program
CHUNK_WORKSPACE = 48 << 20    # scratch of the chunk call, likewise
EVERY = 2**31 - 1             # a window that holds every token
EPS = 1e-6                    # of the norms


def listed():
    return [
        # The queries and keys of a decode step of four users: latency.
        dict(name="rope_step", op="rope", n=4, kv=8, g=4, d=128, rot=128, axes=1, inter=0, norm=1, far=131072, mix=1),
        # A prompt of text and images: three position axes, 28 query heads, no norms, odd count.
        dict(name="rope_images", op="rope", n=16411, kv=4, g=7, d=128, rot=128, axes=3, inter=0, norm=0, far=20000, mix=2),
        # The new tokens of a decode step of 32 users go into an 8-bit cache: latency.
        dict(name="append_step_e4m3", op="append", n=32, kv=4, g=8, d=128, rot=128, axes=1, inter=0, norm=1, far=131072, page=16, fmt="e4m3", mix=3),
        # A long prompt into a cache of 8-bit integers: smaller heads, half of each rotated in neighbouring pairs.
        dict(name="append_prompt_int8_d64", op="append", n=40009, kv=8, g=4, d=64, rot=32, axes=1, inter=1, norm=0, far=40009, page=64, fmt="int8", mix=4),
        # One user far into a conversation; the layer sees the last 1024 tokens and the first four.
        dict(name="window_one", op="window", batch=1, lmax=9001, window=1024, sinks=4, kv=4, g=8, d=128, page=16, fmt="bf16", mix=5),
        # An ordinary batch over an 8-bit cache.
        dict(name="window_batch_e4m3", op="window", batch=64, lmax=20011, window=4096, sinks=4, kv=4, g=8, d=128, page=64, fmt="e4m3", mix=6),
        # A large batch, BF16: as much cache as a step of such a layer reads.
        dict(name="window_large_bf16", op="window", batch=128, lmax=24576, window=8192, sinks=64, kv=4, g=4, d=128, page=32, fmt="bf16", mix=7),
        # A short question behind a cached prompt: latency.
        dict(name="chunk_one_short", op="chunk", batch=1, lmax=16, prefix=1000, window=EVERY, sinks=0, kv=4, g=8, d=128, page=16, fmt="bf16", mix=8),
        # A few drafted tokens of each of 32 users are verified over their contexts: bandwidth.
        dict(name="chunk_drafts_bf16", op="chunk", batch=32, lmax=6, prefix=8192, window=EVERY, sinks=0, kv=8, g=4, d=128, page=16, fmt="bf16", mix=9),
        # Chunks of several prompts in a layer with a sliding window: small heads, none shared, 8-bit integers.
        dict(name="chunk_window_int8_d64", op="chunk", batch=5, lmax=701, prefix=9000, window=2048, sinks=16, kv=16, g=1, d=64, page=32, fmt="int8", mix=10),
        # Packed chunks of prompts, some of them just begun: arithmetic.
        dict(name="chunk_packed_bf16", op="chunk", batch=4, lmax=1500, prefix=4000, window=EVERY, sinks=0, kv=8, g=4, d=128, page=64, fmt="bf16", mix=11),
        # One chunk of a long document over an 8-bit cache.
        dict(name="chunk_long_e4m3", op="chunk", batch=1, lmax=2048, prefix=30000, window=EVERY, sinks=0, kv=4, g=8, d=128, page=16, fmt="e4m3", mix=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(("rope", "append", "window", "chunk", "chunk"))
        c = dict(op=op, kv=rng.choice((1, 2, 4, 8)), g=rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), d=rng.choice((64, 128)), mix=rng.randrange(1 << 20))
        if op in ("rope", "append"):
            c.update(n=log_int(1, 40009), rot=rng.choice((c["d"], c["d"], c["d"] // 2, 48)), axes=rng.choice((1, 1, 2, 3)),
                     inter=rng.choice((0, 0, 1)), norm=rng.choice((0, 1)), far=log_int(1000, 1000000))
            if c["n"] * c["kv"] * c["d"] * (c["g"] + 2) > 40009 * 8 * 64 * 6:
                continue
        if op != "rope":
            c.update(page=rng.choice((1, 8, 16, 20, 32, 64, 128)), fmt=rng.choice(("bf16", "e4m3", "int8")))
        if op in ("window", "chunk"):
            c.update(window=rng.choice((log_int(1, 16384), log_int(64, 16384), EVERY)), sinks=rng.choice((0, 0, 1, 4, 16, 200)))
        if op == "window":
            c.update(batch=log_int(1, 128), lmax=log_int(1, 32768))
            if c["batch"] * c["lmax"] * c["kv"] > 128 * 24576 * 4 or c["batch"] * min(c["lmax"], c["window"]) * c["kv"] * max(4, c["g"]) > 128 * 8192 * 16:
                continue
        if op == "chunk":
            c.update(batch=log_int(1, 32), lmax=log_int(1, 2048), prefix=rng.choice((0, log_int(1, 30000), log_int(1, 30000))))
            if c["batch"] * c["lmax"] * (c["lmax"] + c["prefix"]) * c["kv"] * c["g"] * c["d"] > 2048 * 32048 * 32 * 128:
                continue
        return c


# ---- sizes ------------------------------------------------------------------

def lengths(c):
    """Cached tokens of each sequence of a decode step: from a quarter of the longest up to it (one sequence: all of
    it), and in a batch of 16 or more an idle entry without tokens."""
    r = random.Random(c["mix"])
    if c["batch"] == 1:
        return [c["lmax"]]
    ls = [max(1, int(round(c["lmax"] * r.uniform(0.25, 1.0)))) for _ in range(c["batch"])]
    ls[r.randrange(c["batch"])] = c["lmax"]
    if c["batch"] >= 16:
        ls[r.randrange(c["batch"])] = 0
    return ls


def chunks(c):
    """(new rows, cached tokens with them) of each sequence: from a quarter of the longest up to it; every fourth
    prompt has just begun."""
    r = random.Random(c["mix"] + 1)
    ns = [c["lmax"]] if c["batch"] == 1 else [max(1, int(round(c["lmax"] * r.uniform(0.25, 1.0)))) for _ in range(c["batch"])]
    ns[r.randrange(c["batch"])] = c["lmax"]
    return [(n, n + (0 if i % 4 == 3 else int(round(c["prefix"] * (1.0 if c["batch"] == 1 else r.uniform(0.25, 1.0)))))) for i, n in enumerate(ns)]


def seen(c, last):
    """Cached tokens that the rows at positions last[0] .. last[1] see between them."""
    first, end = last
    low = max(0, first - c["window"] + 1)
    return end + 1 if c["sinks"] >= low else c["sinks"] + end + 1 - low


def pairs(c, n, total):
    """(row, token) pairs of the last n of `total` tokens."""
    w, s = c["window"], c["sinks"]
    p = range(total - n, total)
    if w >= total:
        return sum(p) + n
    return sum(min(x + 1, w + min(s, max(0, x + 1 - w))) for x in p)


def work(c):
    d, kv, h = c["d"], c["kv"], c["kv"] * c["g"]
    held = 0 if c["op"] == "rope" else kv * 2 * (d * 2 if c["fmt"] == "bf16" else d + 4)      # one token of the cache
    if c["op"] in ("rope", "append"):
        n = c["n"]
        flops = n * (h + kv) * ((4 * d if c["norm"] else 0) + 3 * c["rot"])
        rows = 4 * h * d + 4 * c["axes"]                           # q read and written, the positions
        if c["op"] == "rope":
            return {"bytes": n * (rows + 4 * kv * d), "flops": flops}
        # k and v read and stored; read back into rows; the slots both times
        return {"bytes": n * (rows + 4 * kv * d + held + held + 4 * kv * d + 16), "flops": flops}
    if c["op"] == "window":
        ls = lengths(c)
        tokens = [seen(c, (n - 1, n - 1)) if n else 0 for n in ls]
        entries = sum(-(-t // c["page"]) for t in tokens)
        return {"bytes": sum(tokens) * held + 4 * c["batch"] * h * d + 4 * (entries + c["batch"]), "flops": 4 * d * h * sum(tokens)}
    nl = chunks(c)
    tokens = [seen(c, (t - n, t - 1)) for n, t in nl]
    entries = sum(-(-t // c["page"]) for t in tokens)
    return {"bytes": sum(tokens) * held + 4 * sum(n for n, _ in nl) * h * d + 4 * (entries + 2 * c["batch"] + 1),
            "flops": 4 * d * h * sum(pairs(c, n, t) for n, t in nl)}


# ---- inputs -----------------------------------------------------------------

def frequencies(c):
    """Angle per position of each pair, in 64 bits."""
    return [10000.0 ** (-2.0 * j / c["rot"]) for j in range(c["rot"] // 2)]


def sections(c):
    """Pairs of each axis, in order."""
    half = c["rot"] // 2
    first = half // (c["axes"] + 1) if c["axes"] > 1 else half
    rest = [(half - first) // (c["axes"] - 1)] * (c["axes"] - 1) if c["axes"] > 1 else []
    if rest:
        rest[-1] = half - first - sum(rest[:-1])
    return [first] + rest


def quantise(x, fmt):
    """Codes and scales of rows [..., d] held in 8 bits, as the cache stores them."""
    x = x.float()
    a = x.abs().amax(-1, keepdim=True)
    keep = a >= 2.0 ** -100
    y = x * torch.where(keep, QMAX[fmt] / a, 0.0)
    y = y.clamp(-QMAX[fmt], QMAX[fmt])
    return (y.round() if fmt == "int8" else y).to(CODE[fmt]), torch.where(keep, a / QMAX[fmt], 0.0)[..., 0]


def keys_like(shape, gen, dev):
    """Keys as projections give them: some channels of a head are several times larger than the rest."""
    x = torch.randn(shape, generator=gen, device=dev)
    return x * (1 + 3 * (torch.rand(shape[-1], generator=gen, device=dev) > 0.9))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = case
    kv, d, h = c["kv"], c["d"], c["kv"] * c["g"]
    s = {"case": c}
    if c["op"] in ("rope", "append"):
        n = c["n"]
        # [Q|K|V] rows as the projections and folds leave them
        rows = torch.randn(n, (h + 2 * kv) * d, generator=gen, device=dev)
        rows[:, h * d:(h + kv) * d] = keys_like((n, kv, d), gen, dev).view(n, kv * d)
        s["rows"] = rows.bfloat16()
        # text positions run on from where the cached part ends; the second and third axis step through rows and columns
        t = c["far"] - n + torch.arange(n, device=dev) if n < c["far"] else torch.arange(n, device=dev)
        grid = 8 + int(torch.randint(0, 24, (1,), generator=gen, device=dev))
        axes = [t, t // grid, t - t % grid // 2]
        s["positions"] = torch.stack(axes[:c["axes"]]).int()
        if c["norm"]:
            s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(d, generator=gen, device=dev)).bfloat16() for _ in range(2))
        s["q_out"] = torch.empty(n, h * d, dtype=torch.bfloat16, device=dev)
        s["k_out"], s["v_out"] = (torch.empty(n, kv * d, dtype=torch.bfloat16, device=dev) for _ in range(2))
        s["freq"] = torch.tensor(frequencies(c), dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor([a for a, m in enumerate(sections(c)) for _ in range(m)], device=dev)
        pages = -(-n // c["page"]) if c["op"] == "append" else 0
    elif c["op"] == "window":
        ls = lengths(c)
        pages = sum(-(-n // c["page"]) for n in ls)
    else:
        ls = [t for _, t in chunks(c)]
        pages = sum(-(-n // c["page"]) for n in ls)
    if c["op"] != "rope":
        # The cache: pages handed out in no order, [pages, kv heads, page, d] for keys and for values.
        pool = pages + pages // 8 + 1
        shape = (pool, kv, c["page"], d)
        order = torch.randperm(pool, generator=gen, device=dev)[:pages]
    if c["op"] == "append":
        t = torch.randperm(pages * c["page"], generator=gen, device=dev)[:n].sort().values
        s["slots"] = order[t // c["page"]] * c["page"] + t % c["page"]
        s["k_pages"], s["v_pages"] = (torch.zeros(shape, dtype=CODE[c["fmt"]], device=dev) for _ in range(2))
        if c["fmt"] != "bf16":
            s["k_scale"], s["v_scale"] = (torch.zeros(shape[:3], device=dev) for _ in range(2))
    if c["op"] in ("window", "chunk"):
        for x in ("k", "v"):
            made = [], []
            for at in range(0, pool, max(1, (1 << 27) // (kv * c["page"] * d))):   # in parts: the 32-bit values are large
                part = (min(pool - at, max(1, (1 << 27) // (kv * c["page"] * d))), *shape[1:])
                y = keys_like(part, gen, dev) if x == "k" else torch.randn(part, generator=gen, device=dev)
                for to, v in zip(made, (y.bfloat16(),) if c["fmt"] == "bf16" else quantise(y.bfloat16(), c["fmt"])):
                    to.append(v)
            s[x + "_pages"] = torch.cat([v.view(torch.int8) if v.dtype == torch.float8_e4m3fn else v for v in made[0]]).view(CODE[c["fmt"]])
            if c["fmt"] != "bf16":
                s[x + "_scale"] = torch.cat(made[1])
        width = max(1, -(-max(ls) // c["page"]))
        table = torch.full((c["batch"], width), -1, dtype=torch.int32)     # -1: no page
        at, order = 0, order.cpu()
        for b, n in enumerate(ls):
            m = -(-n // c["page"])
            table[b, :m] = order[at:at + m].int()
            at += m
        s["table"] = table.to(dev)
        s["lens"] = torch.tensor(ls, dtype=torch.int32, device=dev)
        news = [1] * c["batch"] if c["op"] == "window" else [n for n, _ in chunks(c)]
        s["cu"] = torch.tensor([sum(news[:b]) for b in range(c["batch"] + 1)], dtype=torch.int32, device=dev)
        s["q"] = torch.randn(sum(news), h * d, generator=gen, device=dev).bfloat16()
        s["out"] = torch.empty(sum(news), h * d, dtype=torch.bfloat16, device=dev)
        s["workspace"] = torch.zeros(DECODE_WORKSPACE if c["op"] == "window" else CHUNK_WORKSPACE, dtype=torch.uint8, device=dev)
    if own:
        from gather_lora_gb300 import lib
        if c["op"] in ("rope", "append"):
            s["rope"] = lib.Rope(d, rotary_dim=c["rot"], freqs=frequencies(c), sections=sections(c), interleaved=bool(c["inter"]))
        if c["op"] != "rope":
            s["cache"] = lib.KvCache(s["k_pages"], s["v_pages"], s.get("k_scale"), s.get("v_scale"))
    return s


# ---- one pass ---------------------------------------------------------------

def run(s):
    c = s["case"]
    return {"rope": run_rope, "append": run_append, "window": run_window, "chunk": run_chunk}[c["op"]](s, c)


def turned(s, c, x, norm):
    """Rows [n, heads, d] in 32 bits, normed by the weights `norm` (if any) and rotated; the angles in 64 bits."""
    x = x.float()
    if norm is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * norm.float()
    angle = s["positions"].double()[s["axis"]].T * s["freq"]                  # [n, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot, half = c["rot"], c["rot"] // 2
    x0, x1 = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :half], x[..., half:rot])
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack((y0, y1), -1).flatten(-2) if c["inter"] else torch.cat((y0, y1), -1)
    return torch.cat((y, x[..., rot:]), -1)


def run_rope(s, c):
    kv, d, n, h = c["kv"], c["d"], c["n"], c["kv"] * c["g"]
    rows = s["rows"]
    if own:
        from gather_lora_gb300 import lib
        stride = rows.stride(0)
        lib.lora_qk_rope(rows, stride, s["q_out"], h * d, rows.data_ptr() + 2 * h * d, stride, s["k_out"], kv * d, n, h, kv, s["rope"],
                         s["positions"], s["positions"].stride(0), q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS)
        return s["q_out"], s["k_out"]
    q = turned(s, c, rows[:, :h * d].reshape(n, h, d), s.get("q_norm"))
    k = turned(s, c, rows[:, h * d:(h + kv) * d].reshape(n, kv, d), s.get("k_norm"))
    return q.bfloat16().view(n, h * d), k.bfloat16().view(n, kv * d)


def run_append(s, c):
    """The rotated queries, and what the cache holds of the new keys and values, read back."""
    kv, d, n, h = c["kv"], c["d"], c["n"], c["kv"] * c["g"]
    rows, slots = s["rows"], s["slots"]
    if own:
        from gather_lora_gb300 import lib
        stride, at = rows.stride(0), rows.data_ptr()
        lib.lora_kv_append(rows, stride, s["q_out"], h * d, h, at + 2 * h * d, stride, at + 2 * (h + kv) * d, stride, slots, n, s["cache"],
                           s["rope"], s["positions"], s["positions"].stride(0), q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS)
        lib.lora_kv_read(s["k_out"], kv * d, s["v_out"], kv * d, slots, n, s["cache"])
        return s["q_out"], s["k_out"], s["v_out"]
    q = turned(s, c, rows[:, :h * d].reshape(n, h, d), s.get("q_norm"))
    k = turned(s, c, rows[:, h * d:(h + kv) * d].reshape(n, kv, d), s.get("k_norm"))
    v = rows[:, (h + kv) * d:].reshape(n, kv, d)
    page, slot = slots // c["page"], slots % c["page"]
    return (q.bfloat16().view(n, h * d), *(stored(s, c, x, y, page, slot) for x, y in (("k", k), ("v", v))))


def stored(s, c, x, y, page, slot):
    """Rows y into their slots of the pages of x, and back."""
    pages = s[x + "_pages"]
    if c["fmt"] == "bf16":
        pages[page, :, slot] = y.bfloat16()
        back = pages[page, :, slot]
    else:
        code, scale = quantise(y, c["fmt"])
        pages.view(torch.int8)[page, :, slot] = code.view(torch.int8)
        s[x + "_scale"][page, :, slot] = scale
        back = pages.view(torch.int8)[page, :, slot].view(CODE[c["fmt"]]).float() * s[x + "_scale"][page, :, slot][..., None]
    return back.bfloat16().reshape(c["n"], -1)


def values(s, c, x, t):
    """What the cache holds of tokens t [b, l] of each sequence, in 32 bits: [b, l, kv, d]."""
    page = s["table"].long().clamp(min=0).gather(1, t // c["page"])
    y, slot = s[x + "_pages"], t % c["page"]
    if c["fmt"] == "bf16":
        return y[page, :, slot].float()
    return y.view(torch.int8)[page, :, slot].view(CODE[c["fmt"]]).float() * s[x + "_scale"][page, :, slot][..., None]


def run_window(s, c):
    kv, g, d, b = c["kv"], c["g"], c["d"], c["batch"]
    h = kv * g
    if own:
        from gather_lora_gb300 import lib
        lib.lora_attn_decode_window(s["q"], h * d, s["out"], h * d, b, h, d ** -0.5, s["cache"], s["table"], s["table"].stride(0),
                                    s["table"].shape[1], s["lens"], c["window"], c["sinks"], s["workspace"], DECODE_WORKSPACE)
        return s["out"]
    # the first tokens, then the window (of each sequence its own), what is in both only once
    n = s["lens"].long()[:, None]
    first = torch.arange(min(c["sinks"], c["lmax"]), device=n.device).expand(b, -1)
    last = n - min(c["window"], c["lmax"]) + torch.arange(min(c["window"], c["lmax"]), device=n.device)
    t = torch.cat((first, last), 1)
    live = torch.cat((first < n, (last >= 0) & (last >= first.shape[1])), 1)
    t = t.clamp(min=0, max=c["lmax"] - 1)
    q = s["q"].float().view(b, kv, g, d)
    z = torch.matmul(q, values(s, c, "k", t).permute(0, 2, 3, 1)) * d ** -0.5          # [b, kv, g, l]
    z = z.masked_fill(~live[:, None, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38))
    del z
    o = torch.matmul(p, values(s, c, "v", t).permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(b, h * d).bfloat16()


def run_chunk(s, c):
    kv, g, d, b = c["kv"], c["g"], c["d"], c["batch"]
    h, tq = kv * g, s["q"].shape[0]
    if own:
        from gather_lora_gb300 import lib
        lib.lora_attn_chunk(s["q"], h * d, s["out"], h * d, s["cu"], b, tq, h, d ** -0.5, s["cache"], s["table"], s["table"].stride(0),
                            s["table"].shape[1], s["lens"], c["window"], c["sinks"], s["workspace"], CHUNK_WORKSPACE)
        return s["out"]
    # the packed rows into one padded batch, and back
    lq, lk = c["lmax"], max(t for _, t in chunks(c))
    nq, nk = s["cu"].diff().long(), s["lens"].long()
    i, j = torch.arange(lq, device=nq.device), torch.arange(lk, device=nq.device)
    q = s["q"].float()[(s["cu"][:-1, None] + i).clamp(max=tq - 1)].view(b, lq, kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, kv, g * lq, d)
    t = torch.minimum(j, (nk - 1).clamp(min=0)[:, None])
    p = (i + (nk - nq)[:, None])[..., None]                                             # [b, lq, 1]: positions
    live = (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]))                        # [b, lq, lk]
    z = torch.matmul(q * d ** -0.5, values(s, c, "k", t).permute(0, 2, 3, 1)).view(b, kv, g, lq, lk)
    z = z.masked_fill_(~live[:, None, None], -math.inf)
    z -= z.amax(-1, keepdim=True).clamp(min=-3e38)
    w = z.exp_()
    o = torch.matmul(w.view(b, kv, g * lq, lk), values(s, c, "v", t).permute(0, 2, 1, 3))
    o = o.view(b, kv, g, lq, d) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(b, lq, h * d)[i < nq[:, None]].bfloat16()


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    kv, g, d = c["kv"], c["g"], c["d"]
    h = kv * g
    if c["op"] in ("rope", "append"):
        n, rot = c["n"], c["rot"]
        out = []
        for first, heads, norm in ((0, h, "q_norm"), (h, kv, "k_norm"), (h + kv, kv, None)):
            if norm is None and c["op"] == "rope":
                continue
            x = s["rows"][:, first * d:(first + heads) * d].double().view(n, heads, d).clone()
            if norm is not None:
                if c["norm"]:
                    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * s[norm].double()
                pair = 0
                for a, m in enumerate(sections(c)):
                    for _ in range(m):
                        angle = s["positions"][a].double() * 10000.0 ** (-2.0 * pair / rot)
                        u, v = (2 * pair, 2 * pair + 1) if c["inter"] else (pair, pair + rot // 2)
                        z = torch.complex(x[..., u], x[..., v]) * torch.polar(torch.ones_like(angle), angle)[:, None]
                        x[..., u], x[..., v] = z.real, z.imag
                        pair += 1
            if first >= h and c["op"] == "append" and c["fmt"] != "bf16":
                # the code is chosen by the format's own 32-bit operations (BF16 rows often lie on ties of the exact quotient)
                a = x.abs().amax(-1, keepdim=True).float()
                y = (x.float() * (QMAX[c["fmt"]] / a)).double()
                step = torch.ones_like(y)
                if c["fmt"] == "e4m3":      # 3 bits after the leading one, down to 2^-9
                    step = torch.exp2(torch.log2(y.abs().clamp(min=2.0 ** -6)).floor() - 3)
                x = torch.round(y / step) * step * (a.double() / QMAX[c["fmt"]])
            out.append(x.reshape(n, heads * d))
        return tuple(out)
    news = [1] * c["batch"] if c["op"] == "window" else [n for n, _ in chunks(c)]
    totals = lengths(c) if c["op"] == "window" else [t for _, t in chunks(c)]
    rows, at = [], 0
    for b, (n, m) in enumerate(zip(news, totals)):
        o = torch.zeros(n, kv, g, d, dtype=torch.float64, device="cuda")
        if m:
            ids = s["table"][b, :-(-m // c["page"])].long()
            held = []
            for x in ("k", "v"):
                y = s[x + "_pages"].view(torch.int8)[ids].view(CODE[c["fmt"]]).double()       # [pages, kv, page, d]
                if c["fmt"] != "bf16":
                    y = y * s[x + "_scale"][ids].double()[..., None]
                held.append(y.transpose(0, 1).reshape(kv, -1, d)[:, :m])
            p = torch.arange(m - n, m, device="cuda")[:, None]
            t = torch.arange(m, device="cuda")
            hide = (t > p) | ((t <= p - c["window"]) & (t >= c["sinks"]))
            q = s["q"][at:at + n].double().view(n, kv, g, d)
            for a in range(kv):
                for e in range(g):
                    z = (q[:, a, e] @ held[0][a].T / math.sqrt(d)).masked_fill(hide, -math.inf)
                    o[:, a, e] = torch.softmax(z, -1) @ held[1][a]
        rows.append(o.reshape(n, -1))
        at += n
    return torch.cat(rows)
