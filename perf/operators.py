"""The attention operators around the folds, as cases to measure: a paged key-value cache written and read back
(lora_kv_write, lora_kv_read), one new token per sequence over that cache (lora_attn_decode) and whole prompts
or prompt chunks (lora_attn_prefill).

Each case is a dict of sizes; `prepare` makes its inputs on the GPU from a seed, `run` makes one pass through the
operator (`own`: through the framework's entry points; otherwise in elementary torch operations in 32 bits, rounded
once at the end), and `exact` gives the same outputs from the definition in 64 bits.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
WORKSPACE_BYTES = 16 << 20   # the decode call's scratch, zero-filled once by the program


def listed():
    return [
        # The new tokens of one decode step of a small batch go into their pages (and are read back): latency.
        dict(name="cache_step_e4m3", op="cache", n=32, kv=4, d=128, page=16, fmt="e4m3", mix=1),
        # One prompt chunk of a few thousand tokens, smaller heads, odd count.
        dict(name="cache_chunk_int8_d64", op="cache", n=4099, kv=8, d=64, page=32, fmt="int8", mix=2),
        # A long prefix stored in 8 bits and read back for a later chunk: bandwidth.
        dict(name="cache_prefix_e4m3", op="cache", n=65536, kv=8, d=128, page=64, fmt="e4m3", mix=3),
        # One user, a short conversation: latency counts, 4 KV heads only.
        dict(name="decode_one_short", op="decode", batch=1, lmax=700, kv=4, g=8, d=128, page=16, fmt="bf16", mix=4),
        # An ordinary serving batch of ragged conversations, BF16 cache.
        dict(name="decode_batch_bf16", op="decode", batch=32, lmax=4096, kv=8, g=4, d=128, page=16, fmt="bf16", mix=5),
        # The same kind of batch over an 8-bit cache, eight query heads per KV head, odd longest length.
        dict(name="decode_batch_e4m3", op="decode", batch=64, lmax=8191, kv=4, g=8, d=128, page=64, fmt="e4m3", mix=6),
        # A few very long contexts, no shared heads, small heads, 8-bit integers.
        dict(name="decode_long_int8_d64", op="decode", batch=5, lmax=100003, kv=16, g=1, d=64, page=128, fmt="int8", mix=7),
        # The largest batch: as much cache as a step reads in one layer.
        dict(name="decode_large_bf16", op="decode", batch=128, lmax=16384, kv=8, g=8, d=128, page=32, fmt="bf16", mix=8),
        # One short prompt: latency.
        dict(name="prefill_one_short", op="prefill", batch=1, lmax=37, prefix=0, kv=4, g=8, d=128, mix=9),
        # Packed prompts of different lengths.
        dict(name="prefill_packed", op="prefill", batch=12, lmax=1100, prefix=0, kv=8, g=4, d=128, mix=10),
        # Chunks of prompts whose first parts are already cached: more keys than queries; no shared heads, small heads.
        dict(name="prefill_chunk_d64", op="prefill", batch=3, lmax=513, prefix=6000, kv=16, g=1, d=64, mix=11),
        # One long prompt.
        dict(name="prefill_long", op="prefill", batch=1, lmax=8192, prefix=0, kv=4, g=8, d=128, mix=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(("cache", "decode", "decode", "prefill", "prefill"))
        c = dict(op=op, kv=rng.choice((1, 2, 4, 8)), d=rng.choice((64, 128)), mix=rng.randrange(1 << 20))
        if op == "cache":
            c.update(n=log_int(1, 65536), page=rng.choice((1, 8, 16, 20, 32, 64, 128)), fmt=rng.choice(("bf16", "e4m3", "int8")))
            sizes = (c["n"],)
        else:
            c["g"] = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
            if op == "decode":
                c.update(batch=log_int(1, 128), lmax=log_int(1, 32768), page=rng.choice((8, 16, 20, 32, 64, 128)),
                         fmt=rng.choice(("bf16", "e4m3", "int8")))
                if c["batch"] * c["lmax"] * c["kv"] * c["g"] > 128 * 16384 * 16 or c["batch"] * c["lmax"] * c["kv"] > 128 * 16384 * 8:
                    continue
            else:
                c.update(batch=log_int(1, 16), lmax=log_int(1, 8192), prefix=rng.choice((0, 0, log_int(1, 8192))))
                pairs = c["batch"] * c["lmax"] * (c["lmax"] + c["prefix"]) * c["kv"] * c["g"]
                if pairs > 32 * 8192 * 8192 // 2:
                    continue
            sizes = (c["batch"], c["lmax"], c["kv"] * c["g"], c["kv"] * c["g"] * c["d"], (2 + c["g"]) * c["kv"] * c["d"])
        if 3072 not in sizes:
            return c


def lengths(c):
    """The sequences' lengths: from a quarter of the longest up to it (one sequence: all of it), and in a batch of 16
    or more now and then an idle entry without tokens (decode)."""
    r = random.Random(c["mix"])
    if c["batch"] == 1:
        return [c["lmax"]]
    ls = [max(1, int(round(c["lmax"] * r.uniform(0.25, 1.0)))) for _ in range(c["batch"])]
    ls[r.randrange(c["batch"])] = c["lmax"]
    if c["op"] == "decode" and c["batch"] >= 16:
        ls[r.randrange(c["batch"])] = 0
    return ls


def chunks(c):
    """(new rows, keys) of each prompt: the keys are the cached prefix and the new rows."""
    r = random.Random(c["mix"] + 1)
    return [(n, n + (int(round(c["prefix"] * r.uniform(0.25, 1.0))) if c["prefix"] else 0)) for n in lengths(c)]


def work(c):
    d, kv = c["d"], c["kv"]
    if c["op"] != "prefill":
        held = kv * 2 * (d * 2 if c["fmt"] == "bf16" else d + 4)       # one token of the cache
    if c["op"] == "cache":   # written from BF16 rows, read back into BF16 rows; the slots both times
        return {"bytes": 2 * c["n"] * (kv * 2 * d * 2 + held + 8), "flops": 0}
    h = kv * c["g"]
    if c["op"] == "decode":
        ls = lengths(c)
        pages = sum(-(-n // c["page"]) for n in ls)
        return {"bytes": sum(ls) * held + 2 * c["batch"] * h * d * 2 + 4 * (pages + c["batch"]), "flops": 4 * d * h * sum(ls)}
    qk = chunks(c)
    pairs = sum(q * k - q * (q - 1) // 2 for q, k in qk)
    return {"bytes": sum(q for q, _ in qk) * h * d * 4 + sum(k for _, k in qk) * kv * d * 4, "flops": 4 * d * h * pairs}


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
    kv, d = c["kv"], c["d"]
    s = {"case": c}
    if c["op"] == "prefill":
        h = kv * c["g"]
        qk = chunks(c)
        tq, tk = sum(q for q, _ in qk), sum(k for _, k in qk)
        # The new rows lie in [Q|K|V] rows, as the projections and folds leave them; with a cached prefix the keys
        # and values of each prompt (read back from the cache, the new ones after them) have rows of their own.
        s["q_rows"] = torch.randn(tq, (h + 2 * kv) * d, generator=gen, device=dev).bfloat16()
        s["q"] = s["q_rows"]
        if c["prefix"]:
            s["k"] = keys_like((tk, kv, d), gen, dev).bfloat16().view(tk, kv * d)
            s["v"] = torch.randn(tk, kv * d, generator=gen, device=dev).bfloat16()
        else:
            s["k"], s["v"] = s["q_rows"][:, h * d:(h + kv) * d], s["q_rows"][:, (h + kv) * d:]
        starts = [[0], [0]]
        for n in qk:
            for at, v in zip(starts, n):
                at.append(at[-1] + v)
        s["cu_q"], s["cu_k"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in starts)
        s["out"] = torch.empty(tq, h * d, dtype=torch.bfloat16, device=dev)
        return s
    # The cache: pages handed out in no order, [pages, kv heads, page, d] for keys and for values.
    if c["op"] == "cache":
        tokens, pages = c["n"], -(-c["n"] // c["page"])
    else:
        ls = lengths(c)
        pages = sum(-(-n // c["page"]) for n in ls)
    pool = pages + pages // 8 + 1
    shape = (pool, kv, c["page"], d)
    order = torch.randperm(pool, generator=gen, device=dev)[:pages]
    if c["op"] == "cache":
        rows = torch.randn(c["n"], 2 * kv * d, generator=gen, device=dev)
        rows[:, :kv * d] = keys_like((c["n"], kv, d), gen, dev).view(c["n"], kv * d)
        s["rows"] = rows.bfloat16()
        t = torch.randperm(pages * c["page"], generator=gen, device=dev)[:tokens].sort().values
        s["slots"] = order[t // c["page"]] * c["page"] + t % c["page"]
        s["k_pages"], s["v_pages"] = (torch.zeros(shape, dtype=CODE[c["fmt"]], device=dev) for _ in range(2))
        if c["fmt"] != "bf16":
            s["k_scale"], s["v_scale"] = (torch.zeros(shape[:3], device=dev) for _ in range(2))
        s["k_out"], s["v_out"] = (torch.empty(c["n"], kv * d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    else:
        h = kv * c["g"]
        for x in ("k", "v"):
            made = [], []
            for at in range(0, pool, max(1, (1 << 27) // (kv * c["page"] * d))):   # in parts: the 32-bit values are large
                n = min(pool - at, max(1, (1 << 27) // (kv * c["page"] * d)))
                part = (n, *shape[1:])
                y = keys_like(part, gen, dev) if x == "k" else torch.randn(part, generator=gen, device=dev)
                for to, v in zip(made, (y.bfloat16(),) if c["fmt"] == "bf16" else quantise(y.bfloat16(), c["fmt"])):
                    to.append(v)
            s[x + "_pages"] = torch.cat([v.view(torch.int8) if v.dtype == torch.float8_e4m3fn else v for v in made[0]]).view(CODE[c["fmt"]])
            if c["fmt"] != "bf16":
                s[x + "_scale"] = torch.cat(made[1])
        width = max(1, -(-c["lmax"] // c["page"]))
        table = torch.full((c["batch"], width), -1, dtype=torch.int32)     # -1: no page
        at, order = 0, order.cpu()
        for b, n in enumerate(ls):
            m = -(-n // c["page"])
            table[b, :m] = order[at:at + m].int()
            at += m
        s["table"] = table.to(dev)
        s["lens"] = torch.tensor(ls, dtype=torch.int32, device=dev)
        s["q"] = torch.randn(c["batch"], h * d, generator=gen, device=dev).bfloat16()
        s["out"] = torch.empty(c["batch"], h * d, dtype=torch.bfloat16, device=dev)
        s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    if own:
        from gather_lora_gb300 import lib
        s["cache"] = lib.KvCache(s["k_pages"], s["v_pages"], s.get("k_scale"), s.get("v_scale"))
    return s


def run(s):
    c = s["case"]
    return {"cache": run_cache, "decode": run_decode, "prefill": run_prefill}[c["op"]](s, c)


def run_cache(s, c):
    kv, d, n = c["kv"], c["d"], c["n"]
    rows, slots = s["rows"], s["slots"]
    if own:
        from gather_lora_gb300 import lib
        stride = rows.stride(0)
        lib.lora_kv_write(rows, stride, rows.data_ptr() + kv * d * 2, stride, slots, n, s["cache"])
        lib.lora_kv_read(s["k_out"], kv * d, s["v_out"], kv * d, slots, n, s["cache"])
        return s["k_out"], s["v_out"]
    page, slot = slots // c["page"], slots % c["page"]
    out = []
    for x, cols in (("k", rows[:, :kv * d]), ("v", rows[:, kv * d:])):
        y = cols.reshape(n, kv, d)
        pages = s[x + "_pages"]
        if c["fmt"] == "bf16":
            pages[page, :, slot] = y
            back = pages[page, :, slot]
        else:
            code, scale = quantise(y, c["fmt"])
            pages.view(torch.int8)[page, :, slot] = code.view(torch.int8)
            s[x + "_scale"][page, :, slot] = scale
            back = pages.view(torch.int8)[page, :, slot].view(CODE[c["fmt"]]).float() * s[x + "_scale"][page, :, slot][..., None]
        out.append(back.bfloat16().reshape(n, kv * d))
    return tuple(out)


def run_decode(s, c):
    kv, g, d, b = c["kv"], c["g"], c["d"], c["batch"]
    h = kv * g
    if own:
        from gather_lora_gb300 import lib
        lib.lora_attn_decode(s["q"], h * d, s["out"], h * d, b, h, d ** -0.5, s["cache"], s["table"], s["table"].stride(0),
                             s["table"].shape[1], s["lens"], s["workspace"], WORKSPACE_BYTES)
        return s["out"]
    t = torch.arange(c["lmax"], device=s["lens"].device)
    seen = t < s["lens"][:, None]                                             # [b, l]
    page = s["table"].long().clamp(min=0)[:, t // c["page"]]
    slot = (t % c["page"]).expand_as(page)

    def values(x):
        y = s[x + "_pages"]
        if c["fmt"] == "bf16":
            return y[page, :, slot].float()                                   # [b, l, kv, d]
        return y.view(torch.int8)[page, :, slot].view(CODE[c["fmt"]]).float() * s[x + "_scale"][page, :, slot][..., None]

    q = s["q"].float().view(b, kv, g, d)
    z = torch.matmul(q, values("k").permute(0, 2, 3, 1)) * d ** -0.5          # [b, kv, g, l]
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    del z
    o = torch.matmul(p, values("v").permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(b, h * d).bfloat16()


def run_prefill(s, c):
    kv, g, d, b = c["kv"], c["g"], c["d"], c["batch"]
    h = kv * g
    tq, tk = s["q"].shape[0], s["k"].shape[0]
    if own:
        from gather_lora_gb300 import lib
        lib.lora_attn_prefill(s["q"], s["q"].stride(0), s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["out"], h * d,
                              s["cu_q"], s["cu_k"], b, tq, tk, h, kv, d, d ** -0.5)
        return s["out"]
    # The packed rows into one padded batch, and back.
    lq, lk = c["lmax"], max(k for _, k in chunks(c))
    nq, nk = s["cu_q"].diff(), s["cu_k"].diff()
    i, j = torch.arange(lq, device=nq.device), torch.arange(lk, device=nq.device)
    rq = (s["cu_q"][:-1, None] + i).clamp(max=tq - 1)
    rk = (s["cu_k"][:-1, None] + j).clamp(max=tk - 1)
    q = s["q"][:, :h * d].float()[rq].view(b, lq, kv, g, d).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[rk].view(b, lk, kv, 1, d).permute(0, 2, 3, 4, 1)
    v = s["v"].float()[rk].view(b, lk, kv, 1, d).permute(0, 2, 3, 1, 4)
    seen = (j <= i[:, None] + (nk - nq)[:, None, None]) & (j < nk[:, None, None])
    z = torch.matmul(q * d ** -0.5, k).masked_fill_(~seen[:, None, None], -math.inf)
    z -= z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = z.exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, lq, h * d)
    return o[i < nq[:, None]].bfloat16()


def exact(case, seed):
    """The outputs in 64 bits, one sequence at a time, from the definitions."""
    c, s = case, prepare(case, seed)
    kv, d = c["kv"], c["d"]
    if c["op"] == "cache":
        out = []
        for cols in (s["rows"][:, :kv * d], s["rows"][:, kv * d:]):
            x = cols.double().reshape(c["n"], kv, d)
            if c["fmt"] != "bf16":
                unit = x.abs().amax(-1, keepdim=True) / QMAX[c["fmt"]]
                y = x / unit
                step = torch.ones_like(y)
                if c["fmt"] == "e4m3":      # 3 bits after the leading one, down to 2^-9
                    step = torch.exp2(torch.log2(y.abs().clamp(min=2.0 ** -6)).floor() - 3)
                x = torch.round(y / step) * step * unit
            out.append(x.reshape(c["n"], kv * d))
        return tuple(out)
    g = c["g"]
    rows = []
    if c["op"] == "decode":
        for b, n in enumerate(lengths(c)):
            if n == 0:
                rows.append(torch.zeros(1, kv * g * d, dtype=torch.float64, device="cuda"))
                continue
            ids = s["table"][b, :-(-n // c["page"])].long()

            def held(x):
                y = s[x + "_pages"].view(torch.int8)[ids].view(CODE[c["fmt"]]).double()       # [pages, kv, page, d]
                if c["fmt"] != "bf16":
                    y = y * s[x + "_scale"][ids].double()[..., None]
                return y.transpose(0, 1).reshape(kv, -1, d)[:, :n]

            q = s["q"][b].double().view(kv, g, d)
            z = torch.einsum("kgd,kld->kgl", q, held("k")) / math.sqrt(d)
            rows.append(torch.einsum("kgl,kld->kgd", torch.softmax(z, -1), held("v")).reshape(1, -1))
        return torch.cat(rows)
    at_q = at_k = 0
    for n, m in chunks(c):
        q = s["q"][at_q:at_q + n, :kv * g * d].double().view(n, kv, g, d)
        k = s["k"][at_k:at_k + m].double().view(m, kv, d)
        v = s["v"][at_k:at_k + m].double().view(m, kv, d)
        o = torch.empty(n, kv, g, d, dtype=torch.float64, device="cuda")
        hide = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        for a in range(kv):
            for e in range(g):
                z = (q[:, a, e] @ k[:, a].T / math.sqrt(d)).masked_fill(hide, -math.inf)
                o[:, a, e] = torch.softmax(z, -1) @ v[:, a]
        rows.append(o.reshape(n, -1))
        at_q, at_k = at_q + n, at_k + m
    return torch.cat(rows)
