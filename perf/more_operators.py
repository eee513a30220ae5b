"""What stands around the quantized key/value cache in a serving step: measured cases and their plain forms.

* ``plan``     the page table, slot numbers, positions and row offsets of a step, on the GPU, from the sequences' lengths
               and a stack of free pages;
* ``release``  a step planned, then taken back: its pages return to the stack;
* ``write``    norms of each head of queries and keys and the rotation by their positions, the keys quantized into the cache
               with the values in the same pass;
* ``rotate``   the same norms and rotation without a cache;
* ``attend``   attention over the cache whose scores are capped by a tanh, biased by their distance, or which sees a prefix
               in both directions.

Cache layout: codes ``[pages, kv_heads, page, D]`` (INT8 int8, E4M3 bytes in uint8) or ``[..., D / 2]`` (INT4, element 2i in
the low nibble); one record per token and head: a float32 scale, or for INT4 a float16 pair of scale and zero-point.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a decode step of a small batch: latency
        dict(name="plan_step", op="plan", batch=16, q_len=1, kv_len=2000, pad=0, page=16, short=0, ragged=False),
        # chunks of prompts beside decode steps, rows padded to a captured size, the last sequences without pages
        dict(name="plan_chunks", op="plan", batch=300, q_len=701, kv_len=8192, pad=1000, page=64, short=90, ragged=True),
        # one verified draft of a small batch is taken back
        dict(name="release_step", op="release", batch=24, q_len=7, kv_len=1500, pad=0, page=16, short=0, ragged=False),
        # a large batch's drafts are taken back
        dict(name="release_batch", op="release", batch=2048, q_len=33, kv_len=4096, pad=77, page=16, short=0, ragged=True),
        # a decode step's rows: latency
        dict(name="write_step_int8", op="write", fmt="int8", dtype="bf16", tokens=16, kv_heads=8, group=4, dim=128, rot=128,
             near=False, norm=True, base=10000.0, far=32768, page=16),
        # a long prompt, with padding rows, at far positions
        dict(name="write_prompt_fp8", op="write", fmt="fp8", dtype="bf16", tokens=16383, kv_heads=8, group=4, dim=128, rot=128,
             near=False, norm=True, base=500000.0, far=1000000, page=64),
        # wide heads of which a part is rotated, neighbours paired, 4 bits
        dict(name="write_prompt_int4", op="write", fmt="int4", dtype="f16", tokens=4099, kv_heads=4, group=2, dim=256, rot=64,
             near=True, norm=True, base=10000.0, far=131072, page=32),
        # queries and keys of narrow heads that go elsewhere than the cache
        dict(name="rotate_prompt", op="rotate", dtype="bf16", tokens=8191, kv_heads=8, group=2, dim=64, rot=64,
             near=False, norm=True, base=10000.0, far=131072),
        # 32-bit rows without norms
        dict(name="rotate_step_f32", op="rotate", dtype="f32", tokens=33, kv_heads=8, group=4, dim=128, rot=32,
             near=True, norm=False, base=10000.0, far=4096),
        # a decode step of a serving batch with capped scores
        dict(name="attend_batch_fp8", op="attend", fmt="fp8", dtype="bf16", batch=32, q_len=1, kv_len=8192, ragged=True,
             kv_heads=8, group=4, dim=128, page=64, window=0, sinks=0, cap=30.0, slopes=False, prefix=0.0),
        # a chunk of a long prompt in a sliding-window layer with capped scores
        dict(name="attend_chunk_fp8", op="attend", fmt="fp8", dtype="bf16", batch=1, q_len=2048, kv_len=16384, ragged=False,
             kv_heads=8, group=4, dim=128, page=64, window=4096, sinks=0, cap=50.0, slopes=False, prefix=0.0),
        # prompts of several users, scores biased by distance, each with a prefix that is seen whole
        dict(name="attend_ragged_int8", op="attend", fmt="int8", dtype="f16", batch=6, q_len=701, kv_len=2999, ragged=True,
             kv_heads=4, group=7, dim=128, page=16, window=0, sinks=0, cap=0.0, slopes=True, prefix=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= 4.7e8 and w["flops"] <= 1.3e11:
            return c


def _draw(rng):
    while True:
        op = rng.choice(("plan", "release", "write", "write", "rotate", "attend", "attend", "attend"))
        if op in ("plan", "release"):
            c = dict(op=op, batch=_log(rng, 1, 2048), q_len=_log(rng, 1, 2048), kv_len=_log(rng, 1, 32768), pad=rng.choice((0, 0, 1, 500)),
                     page=rng.choice((16, 32, 64, 128)), short=0, ragged=rng.random() < 0.6)
            if op == "plan" and rng.random() < 0.4:
                c["short"] = rng.randrange(1, c["batch"] + 1)
            if c["batch"] * c["q_len"] <= 2 ** 17 and c["batch"] * c["kv_len"] <= c["page"] * 2 ** 20:
                return c
            continue
        shape = dict(kv_heads=rng.choice((1, 2, 4, 8)), group=rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), dim=rng.choice((64, 128, 128, 256)))
        c = dict(op=op, dtype=rng.choice(("bf16", "f16")), **shape)
        if op == "attend":
            c.update(fmt=rng.choice(("int8", "fp8", "int4")), batch=_log(rng, 1, 64), q_len=1, kv_len=_log(rng, 1, 65536),
                     ragged=rng.random() < 0.5, page=rng.choice((16, 32, 64, 128)))
            if rng.random() < 0.5:
                c["q_len"] = _log(rng, 1, 2048)
            c["window"] = rng.choice((0, 0, _log(rng, 1, 8192)))
            c["sinks"] = rng.choice((0, 1, 4, 17)) if c["window"] else 0
            c["cap"] = rng.choice((0.0, 5.0, 20.0, 30.0, 50.0, 1000.0))
            c["slopes"] = rng.random() < 0.5
            c["prefix"] = rng.choice((0.0, 0.0, 0.3, 1.0)) if c["cap"] or c["slopes"] else 0.7
            c["kv_len"] += c["q_len"]
            rows = c["batch"] * c["q_len"] * c["kv_heads"] * c["group"]
            if rows * c["kv_len"] <= 2 ** 29 and c["batch"] * c["kv_len"] * c["kv_heads"] * c["dim"] <= 2 ** 28:
                return c
            continue
        c.update(tokens=_log(rng, 1, 16383), rot=rng.choice((c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4)), near=rng.random() < 0.5,
                 norm=rng.random() < 0.7, base=rng.choice((10000.0, 500000.0)), far=_log(rng, 10, 1000000))
        if op == "write":
            c.update(fmt=rng.choice(("int8", "fp8", "int4")), page=rng.choice((16, 32, 64, 128)))
        elif rng.random() < 0.3:
            c["dtype"] = "f32"
        return c


# ----------------------------------------------------------------- inputs ----

def _spread(most, least, n, ragged):
    """n lengths up to `most`, the first of them `most`: the same for every seed."""
    if not ragged:
        return [most] * n
    return [most if i == 0 else max(least, int(most * (0.3 + 0.7 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]


def _steps(case):
    """Lengths of a planned step: (before, new) of each sequence; some have nothing new."""
    before = _spread(case["kv_len"], 0, case["batch"], case["ragged"])
    new = _spread(case["q_len"], 1, case["batch"], case["ragged"])
    if case["ragged"]:
        new = [0 if i % 11 == 5 else 1 if i % 4 == 3 else n for i, n in enumerate(new)]
        before = [0 if i % 9 == 7 else n for i, n in enumerate(before)]
    return before, new


def _lengths(case):
    q = _spread(case["q_len"], 1, case["batch"], case["ragged"] and case["q_len"] > 1)
    kv = [max(a, b) for a, b in zip(_spread(case["kv_len"], 1, case["batch"], case["ragged"]), q)]
    return q, kv


def _prefixes(case):
    """Positions that all of a sequence's queries see: other shares of their lengths."""
    return [int(n * case["prefix"] * (0.5 + 0.5 * ((i * 0.6180339887) % 1.0))) for i, n in enumerate(_lengths(case)[1])]


def _tokens(g, n, heads, dim, dev):
    """Keys: channels of different spread and mean. Values: tokens of different size."""
    spread = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device=dev))
    mean = 0.5 * torch.randn(heads, dim, generator=g, device=dev)
    k = torch.randn(n, heads, dim, generator=g, device=dev) * spread + mean
    v = torch.randn(n, heads, dim, generator=g, device=dev) * torch.exp(0.3 * torch.randn(n, heads, 1, generator=g, device=dev))
    return k, v


def _empty_cache(fmt, pages, heads, page, dim, dev):
    c = {"fmt": fmt}
    for t in ("k", "v"):
        c[t] = torch.zeros(pages, heads, page, dim // 2 if fmt == "int4" else dim, device=dev,
                           dtype=torch.int8 if fmt == "int8" else torch.uint8)
        c[t + "_scale"] = (torch.ones(pages, heads, page, 2, device=dev, dtype=torch.float16) if fmt == "int4"
                           else torch.ones(pages, heads, page, device=dev))
    return c


def _handle(c):
    from bit_gemm_w4_amd import ops
    return ops.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"], {"int8": ops.I8, "fp8": ops.FP8_E4M3, "int4": ops.U4}[c["fmt"]])


def _prepare_plan(case, g, dev):
    page, batch = case["page"], case["batch"]
    before, new = _steps(case)
    held = [-(-n // page) for n in before]
    need = [-(-(n + m) // page) - h for n, m, h in zip(before, new, held)]
    spare = sum(need) + 7
    if case["short"]:  # not enough for the last sequences
        spare = sum(need[:batch - case["short"]])
    per = max(h + n for h, n in zip(held, need)) + 1
    pages = sum(held) + spare + 1
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    h = torch.tensor(held, device=dev)
    first = torch.cumsum(h, 0) - h
    i = torch.arange(per, device=dev)
    # one entry more than the table has: where rows that write nothing write
    store = torch.full((batch * per + 1,), -1, dtype=torch.int32, device=dev)
    store[:-1].view(batch, per).copy_(torch.where(i < h[:, None], ids[(first[:, None] + i).clamp(max=pages - 1)], -1))
    free = torch.full((pages,), -1, dtype=torch.int32, device=dev)
    free[:spare] = ids[sum(held):sum(held) + spare]
    s = {"op": case["op"], "store": store, "table": store[:-1].view(batch, per), "free": free, "page": page, "count": torch.tensor([spare, 0], dtype=torch.int32, device=dev),
         "lens": torch.tensor(before, dtype=torch.int32, device=dev), "gone": torch.zeros(batch, dtype=torch.int32, device=dev),
         "q_lens": torch.tensor(new, dtype=torch.int32, device=dev), "keep": torch.tensor(before, dtype=torch.int32, device=dev),
         "tokens": sum(new) + case["pad"]}
    if own:
        from bit_gemm_w4_amd import ops
        s["pool"] = ops.KVPool(s["table"], s["lens"], s["gone"], s["free"], s["count"], page)
    return s


def _prepare_rows(case, g, dev):
    n, h, group, d, dt = case["tokens"], case["kv_heads"], case["group"], case["dim"], DTYPES[case["dtype"]]
    k, v = _tokens(g, n, h, d, dev)
    q = torch.randn(n, h * group * d, generator=g, device=dev)
    # the rows as the fused projection leaves them: queries, keys and values side by side
    row = torch.cat((q, k.view(n, h * d), v.view(n, h * d)), 1).to(dt)
    q, k, v = row.split([h * group * d, h * d, h * d], 1)
    s = {"op": case["op"], "dtype": dt, "q": q.view(n, h * group, d), "k": k.view(n, h, d), "v": v.view(n, h, d), "near": case["near"], "rot": case["rot"],
         "eps": 1e-6, "q_weight": None, "k_weight": None}
    if case["norm"]:
        for t in ("q_weight", "k_weight"):
            s[t] = (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
    # a chunk of one long sequence, and rows of others anywhere before it
    near = torch.arange(n, device=dev) + max(0, case["far"] - n)
    far = torch.randint(0, case["far"], (n,), generator=g, device=dev)
    s["positions"] = torch.where(torch.arange(n, device=dev) % 4 == 3, far, near).to(torch.int32)
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev)
    s["inv_freq"] = case["base"] ** (-2.0 * i / case["rot"])
    if case["op"] == "write":
        page = case["page"]
        pages = n // page + 2
        slots = torch.randperm(pages, generator=g, device=dev).repeat_interleave(page) * page
        slots = (slots + torch.arange(page, device=dev).repeat(pages))[:n].contiguous()
        if n > 100:  # padding
            slots[torch.rand(n, generator=g, device=dev) < 0.02] = -1
        s["slots"] = slots
        s["cache"] = _empty_cache(case["fmt"], pages, h, page, d, dev)
    if own:
        from bit_gemm_w4_amd import ops
        s["freqs"] = ops.rope_freqs(s["inv_freq"])
        if case["op"] == "write":
            s["handle"] = _handle(s["cache"])
    return s


def _prepare_attention(case, g, dev):
    dt = DTYPES[case["dtype"]]
    h, d, page, fmt, batch, group = case["kv_heads"], case["dim"], case["page"], case["fmt"], case["batch"], case["group"]
    q_len, kv_len = _lengths(case)
    total = sum(q_len)
    per = -(-max(kv_len) // page)
    pages = batch * per + 1
    c = _empty_cache(fmt, pages, h, page, d, dev)
    table = (torch.randperm(pages - 1, generator=g, device=dev) + 1).view(batch, per).to(torch.int32)
    k, v = _tokens(g, pages * page, h, d, dev)
    for t, x in (("k", k), ("v", v)):
        x = x.to(dt).view(pages, page, h, d).transpose(1, 2).contiguous()
        c[t], c[t + "_scale"] = _quantize(x, fmt)
    del k, v
    if case["window"]:
        # pages that no query of this call or a later one sees were given back
        first = torch.tensor([b - a - case["window"] + 1 for a, b in zip(q_len, kv_len)], device=dev)
        p = torch.arange(per, device=dev)[None]
        table = torch.where(((p + 1) * page <= first[:, None]) & (p * page >= case["sinks"]), -1, table)
    row = torch.randn(total, (group + 2) * h * d, generator=g, device=dev) * 4.0
    cu = [0]
    for a in q_len:
        cu.append(cu[-1] + a)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"op": "attend", "dtype": dt, "cache": c, "q": row.to(dt)[:, :group * h * d].view(total, group * h, d), "table": table.contiguous(),
         "kv_lens": ints(kv_len), "cu_q": ints(cu), "max_q": max(q_len), "max_kv": max(kv_len), "window": case["window"], "sinks": case["sinks"],
         "cap": case["cap"], "slopes": None, "prefix_lens": None}
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, group * h + 1, device=dev) / (group * h))
    if case["prefix"]:
        s["prefix_lens"] = ints(_prefixes(case))
    if own:
        s["handle"] = _handle(c)
    return s


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] in ("plan", "release"):
        return _prepare_plan(case, g, dev)
    if case["op"] == "attend":
        return _prepare_attention(case, g, dev)
    return _prepare_rows(case, g, dev)


# ------------------------------------------------------------- plain forms ----

def _over(x, by):
    """x / by as a quotient: torch divides by a plain number through its reciprocal."""
    return x / torch.full_like(x, by)


def _quantize(x, fmt):
    """Codes and records of rows x[..., D]."""
    x = x.float()
    if fmt == "int4":
        lo, hi = x.amin(-1, keepdim=True).clamp(max=0.0), x.amax(-1, keepdim=True).clamp(min=0.0)
        scale = _over(hi - lo, 15.0).clamp(2.0 ** -24, 65504.0).half().float()
        scale = torch.where(hi == lo, 1.0, scale)
        zero = torch.round(-lo / scale).clamp(0.0, 15.0)
        u = (torch.round(x / scale) + zero).clamp(0.0, 15.0).to(torch.uint8)
        return u[..., 0::2] | u[..., 1::2] << 4, torch.cat((scale, zero), -1).half()
    most = 127.0 if fmt == "int8" else 448.0
    scale = _over(x.abs().amax(-1, keepdim=True), most)
    scale = torch.where(scale == 0.0, 1.0, scale)
    if fmt == "int8":
        return torch.round(x / scale).clamp(-127.0, 127.0).to(torch.int8), scale[..., 0]
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale[..., 0]


def _values(codes, record, fmt):
    """The float32 values that codes and records stand for."""
    if fmt == "int4":
        u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
        r = record.float()
        return (u - r[..., 1:]) * r[..., :1]
    if fmt == "fp8":
        codes = codes.view(torch.float8_e4m3fn)
    return codes.float() * record[..., None]


def _plain_plan(s, advance):
    page, per, batch, rows = s["page"], s["table"].shape[1], s["table"].shape[0], s["tokens"]
    lens, new, count = s["lens"].long(), s["q_lens"].long().clamp(min=0), s["count"][0].long()
    end = torch.cumsum(new, 0)
    start, after = end - new, lens + new
    held = (lens + page - 1) // page
    fits = (end <= rows) & (after <= per * page)
    need = torch.where(fits, (after + page - 1) // page - held, 0)
    taken = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (taken <= count))
    t = torch.arange(rows, device=lens.device)
    b = torch.searchsorted(end, t, right=True).clamp(max=batch - 1)
    real = t < end[-1]
    at = torch.where(real, lens[b] + t - start[b], 0)
    ok, p = real & served[b], at // page
    fresh = (count - 1 - (taken[b] - need[b] + p - held[b])).clamp(min=0, max=s["free"].shape[0] - 1)
    entry = torch.where(ok, b * per + p, batch * per)
    page_id = torch.where(p < held[b], s["store"][entry], s["free"][fresh])
    s["store"][entry] = torch.where(ok, page_id, -1)
    slots = torch.where(ok & (page_id >= 0), page_id.long() * page + at % page, -1)
    kv = torch.where(served, after, lens).to(torch.int32)
    cu = torch.cat((torch.zeros_like(end[:1]), end.clamp(max=rows))).to(torch.int32)
    if advance:
        s["lens"].copy_(kv)
        s["count"][0] -= torch.where(served, need, 0).sum().to(torch.int32)
    return [cu, kv, at.to(torch.int32), slots, served.to(torch.int32)]


def _plain_release(s):
    page, per, batch = s["page"], s["table"].shape[1], s["table"].shape[0]
    pages, count = s["free"].shape[0], s["count"][0].long()
    lens, keep = s["lens"].long(), s["keep"].long().clamp(min=0)
    low, high = (torch.minimum(lens, keep) + page - 1) // page, (lens + page - 1) // page
    end = torch.cumsum(high - low, 0)
    j = torch.arange(pages, device=lens.device)
    b = torch.searchsorted(end, j, right=True).clamp(max=batch - 1)
    real = j < end[-1]
    entry = torch.where(real, b * per + low[b] + j - (end - high + low)[b], batch * per)
    to = torch.where(real, count + end[-1] - 1 - j, pages)
    grown = torch.cat((s["free"], s["free"][:1]))
    grown[to] = s["store"][entry]
    s["free"].copy_(grown[:pages])
    s["store"][entry] = -1
    s["lens"].copy_(torch.minimum(lens, keep).to(torch.int32))
    s["count"][0] += end[-1].to(torch.int32)


def _turned(x, s, weight, wide):
    """Heads x [T][heads][D], normed and rotated, in 64 bits (wide) or 32; angles are of far positions: in 64."""
    x = x.double() if wide else x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.to(x.dtype)
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    rot = s["rot"]
    if s["near"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rows(s):
    q = _turned(s["q"], s, s["q_weight"], False).to(s["dtype"])
    if s["op"] == "rotate":
        return [q, _turned(s["k"], s, s["k_weight"], False).to(s["dtype"])]
    c, slots = s["cache"], s["slots"]
    n, page = c["k"].shape[0], c["k"].shape[2]
    held = (slots >= 0) & (slots < n * page)
    # a skipped token writes to a spare page, which no sequence owns
    at = torch.where(held, slots, n * page)
    p, o = at // page, at % page
    out = [q]
    # keys in 64 bits: the codes stand next to the borders of their rounding
    for t, x in (("k", _turned(s["k"], s, s["k_weight"], True).float()), ("v", s["v"])):
        codes, record = _quantize(x, c["fmt"])
        for name, new in ((t, codes), (t + "_scale", record)):
            old = c[name]
            grown = torch.cat((old, old[:1]))
            grown[p, :, o] = new
            old.copy_(grown[:n])
        y = _values(c[t][p % n, :, o], c[t + "_scale"][p % n, :, o], c["fmt"])
        out.append(torch.where(held[:, None, None], y, 0.0).to(s["dtype"]))
    return out


def _plain_attention(s):
    c, q, lens, cu = s["cache"], s["q"], s["kv_lens"].long(), s["cu_q"].long()
    n, heads, page, _ = c["k"].shape
    batch, per = s["table"].shape
    total, q_heads, d = q.shape
    dev, group, m, length = q.device, q_heads // heads, s["max_q"], s["max_kv"]
    there = (s["table"] >= 0) & (s["table"] < n)
    pages = torch.where(there, s["table"], 0).long()
    k, v = (_values(c[t][pages], c[t + "_scale"][pages], c["fmt"]).transpose(1, 2).reshape(batch, heads, per * page, d)[:, :, :length]
            for t in ("k", "v"))
    i, j = torch.arange(m, device=dev), torch.arange(length, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=total - 1)
    x = q.float()[rows].view(batch, m, heads, group, d).permute(0, 2, 1, 3, 4).reshape(batch, heads, m * group, d)
    held = there.repeat_interleave(page, 1)[:, :length] & (j < lens[:, None])
    at, kv = ((lens - cu[1:] + cu[:-1])[:, None] + i)[:, :, None], j[None, None]
    seen = kv <= at
    if s["prefix_lens"] is not None:
        seen = seen | (kv < s["prefix_lens"].long()[:, None, None])
    if s["window"]:
        seen = seen & ((kv > at - s["window"]) | (kv < s["sinks"]))
    seen = (seen & held[:, None]).view(batch, 1, m, 1, length)
    score = torch.matmul(x, k.transpose(2, 3).contiguous()).view(batch, heads, m, group, length) * d ** -0.5
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    if s["slopes"] is not None:
        score = score - s["slopes"].view(1, heads, 1, group, 1) * (at - kv).abs().float().view(batch, 1, m, 1, length)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    weight = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, heads, m * group, length), v).view(batch, heads, m, group, d)
    o = torch.where(weight > 0.0, o / weight, 0.0)
    t = torch.arange(total, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    return o.permute(0, 2, 1, 3, 4)[b, t - cu[b]].reshape(total, q_heads, d).to(q.dtype)


def run(s):
    if not own:
        if s["op"] == "plan":
            return _plain_plan(s, False) + [s["table"]]
        if s["op"] == "release":
            out = _plain_plan(s, True)
            _plain_release(s)
            return out + [s["table"], s["lens"], s["free"], s["count"][:1]]
        return _plain_attention(s) if s["op"] == "attend" else _plain_rows(s)
    from bit_gemm_w4_amd import ops
    if s["op"] in ("plan", "release"):
        x = ops.kv_plan(s["pool"], s["q_lens"], s["tokens"], advance=s["op"] == "release")
        out = [x.cu_q, x.kv_lens, x.positions, x.slots, x.served, s["table"]]
        if s["op"] == "release":
            ops.kv_release(s["pool"], s["keep"])
            out += [s["lens"], s["free"], s["count"][:1]]
        return out
    if s["op"] == "attend":
        return ops.kv_attn(s["q"], s["handle"], s["table"], s["kv_lens"], s["cu_q"], s["max_q"], max_kv_len=s["max_kv"],
                           window=s["window"], sinks=s["sinks"], softcap=s["cap"], slopes=s["slopes"], prefix_lens=s["prefix_lens"])
    how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], interleaved=s["near"])
    if s["op"] == "rotate":
        return list(ops.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], **how))
    q = ops.kv_cache_write_rope(s["q"], s["k"], s["v"], s["handle"], s["slots"], s["positions"], s["freqs"], **how)
    return [q, *ops.kv_cache_read(s["handle"], s["slots"], s["dtype"])]


# ------------------------------------------------------- work and exactness ----

def work(case):
    if case["op"] in ("plan", "release"):
        before, new = _steps(case)
        page = case["page"]
        need = sum(-(-(n + m) // page) + -n // page for n, m in zip(before, new))
        rows = sum(new) + case["pad"]
        # lengths read, offsets, lengths and flags written; positions and slots of the rows; new pages read and written
        step = 4 * case["batch"] * 5 + 12 * rows + 8 * need
        return {"bytes": step if case["op"] == "plan" else step + 4 * case["batch"] * 3 + 8 * need, "flops": 0}
    h, d, group = case["kv_heads"], case["dim"], case["group"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotate":
        # read and write the rows of queries and keys
        return {"bytes": case["tokens"] * ((group + 1) * h * d * size * 2 + 4), "flops": case["tokens"] * (group + 1) * h * d * 7}
    token = h * 2 * ((d // 2 if case["fmt"] == "int4" else d) + 4)  # codes and records of a token's keys and values
    if case["op"] == "write":
        # read the rows, write the queries, write and read the codes, write their values
        rows = (group + 2) * h * d * size + group * h * d * size + 2 * h * d * size
        return {"bytes": case["tokens"] * (rows + 2 * token + 12), "flops": case["tokens"] * h * d * ((group + 1) * 7 + 8)}
    q_len, kv_len = _lengths(case)
    window, sinks = case["window"], case["sinks"]
    seen, pairs = 0, 0
    for a, b, prefix in zip(q_len, kv_len, _prefixes(case)):
        low = max(0, b - a - window + 1) if window else 0
        seen += b - low + min(low, sinks)
        for at in range(b - a, b):
            first = max(0, at - window + 1) if window else 0
            pairs += max(at + 1, prefix) - first + min(first, sinks)
    heads = h * group
    return {"bytes": seen * token + sum(q_len) * heads * d * 2 * 2, "flops": pairs * heads * d * 4}


def _exact_rows(x, fmt):
    """What a quantized row stands for: the codes are defined by quotients in 32 bits, the rest is in 64."""
    quotient = lambda a, b: (a / b).float().double()  # noqa: E731  (the nearest 32-bit quotient of 32-bit values)
    if fmt == "int4":
        lo = torch.minimum(x.min(-1, keepdim=True).values, torch.zeros((), device=x.device, dtype=x.dtype))
        hi = torch.maximum(x.max(-1, keepdim=True).values, torch.zeros((), device=x.device, dtype=x.dtype))
        s = quotient((hi - lo).float().double(), 15.0).clamp(2.0 ** -24, 65504.0).half().double()
        s[hi == lo] = 1.0
        z = quotient(-lo, s).round().clamp(0, 15)
        return ((quotient(x, s).round() + z).clamp(0, 15) - z) * s
    s = quotient(x.abs().max(-1, keepdim=True).values, 127.0 if fmt == "int8" else 448.0)
    s[s == 0.0] = 1.0
    y = quotient(x, s)
    if fmt == "int8":
        return y.round().clamp(-127, 127) * s
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(y / step) * step).clamp(-448, 448) * s


def _exact_pages(codes, record, fmt):
    if fmt == "int8":
        return codes.double() * record.double().unsqueeze(-1)
    if fmt == "fp8":
        b = torch.arange(256, dtype=torch.float64)
        e, f = (b // 8) % 16, b % 8
        size = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e - 10))
        return (torch.where(b >= 128, -size, size).to(codes.device)[codes.long()]) * record.double().unsqueeze(-1)
    pairs = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    pairs[..., ::2], pairs[..., 1::2] = codes % 16, codes // 16
    return (pairs - record[..., 1:2].double()) * record[..., 0:1].double()


def _exact_heads(x, weight, s, case):
    """Pairs as complex numbers, turned by exp(i angle)."""
    x = x.double()
    if weight is not None:
        x = x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + s["eps"]).sqrt() * weight.double()
    half, rot = case["rot"] // 2, case["rot"]
    lower = torch.arange(half, device=x.device) * (2 if case["near"] else 1)
    upper = lower + (1 if case["near"] else half)
    turns = s["positions"].double()[:, None] * case["base"] ** (-torch.arange(0, rot, 2, device=x.device, dtype=torch.float64) / rot)
    z = torch.complex(x[..., lower], x[..., upper]) * torch.polar(torch.ones_like(turns), turns)[:, None]
    y = x.clone()
    y[..., lower], y[..., upper] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] in ("plan", "release"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] in ("write", "rotate"):
        q, k = (_exact_heads(s[t], s[t + "_weight"], s, case) for t in ("q", "k"))
        if case["op"] == "rotate":
            return [q, k]
        keep = (s["slots"] != -1).double()[:, None, None]
        return [q, *(_exact_rows(x, case["fmt"]) * keep for x in (k.float().double(), s["v"].double()))]
    c, q = s["cache"], s["q"].double()
    out = torch.zeros_like(q)
    q_len, kv_len = _lengths(case)
    first, page, group, d = 0, case["page"], case["group"], case["dim"]
    for b, (a, length) in enumerate(zip(q_len, kv_len)):
        safe = torch.tensor([max(i, 0) for i in s["table"][b, :-(-length // page)].tolist()], device=q.device)
        j = torch.arange(length, device=q.device)
        at = torch.arange(length - a, length, device=q.device)[:, None]
        see = j <= at if not case["prefix"] else (j <= at) | (j < int(s["prefix_lens"][b]))
        if case["window"]:
            see = see & ((at - j < case["window"]) | (j < case["sinks"]))
        for head in range(case["kv_heads"]):
            k, v = (_exact_pages(c[t][safe, head], c[t + "_scale"][safe, head], case["fmt"]).reshape(-1, d)[:length] for t in ("k", "v"))
            for i in range(head * group, (head + 1) * group):
                x = q[first:first + a, i] @ k.T / math.sqrt(d)
                if case["cap"]:
                    e = torch.exp(-2.0 * x.abs() / case["cap"])
                    x = case["cap"] * torch.sign(x) * -torch.expm1(-2.0 * x.abs() / case["cap"]) / (1.0 + e)
                if case["slopes"]:
                    x = x - float(s["slopes"][i]) * (at - j).abs()
                x = x.masked_fill(~see, -math.inf)
                out[first:first + a, i] = torch.softmax(x, -1) @ v
        first += a
    return out
