"""The quantized key/value cache and the attention that reads it: measured cases and their plain forms.

Three operators over one paged cache, each in the cache's three formats (INT8, OCP E4M3, asymmetric INT4):

* ``cache``   the keys and values of new tokens are quantized as they are written, and slots are read back;
* ``attend``  causal attention of ragged query tokens over the cache, with a sliding window and a few first
              tokens that stay visible (no window: every earlier token is visible);
* ``tree``    attention of a tree of drafted tokens: each sees the whole prefix and its own ancestors.

Cache layout: codes ``[pages, kv_heads, page, D]`` (INT8 int8, E4M3 bytes in uint8) or ``[..., D / 2]`` (INT4,
element 2i in the low nibble); one record per token and head: a float32 scale, or for INT4 a float16 pair of
scale and zero-point.  A block table gives each sequence's pages; a page outside the cache holds nothing.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decode step of a small batch: its new tokens enter the cache
        dict(name="cache_step_int8", op="cache", fmt="int8", dtype="bf16", tokens=16, kv_heads=8, dim=128, page=16),
        # a long prompt's keys and values, with padding tokens that are skipped
        dict(name="cache_prompt_fp8", op="cache", fmt="fp8", dtype="bf16", tokens=16383, kv_heads=8, dim=128, page=64),
        # a prompt into a 4-bit cache, wide heads
        dict(name="cache_prompt_int4", op="cache", fmt="int4", dtype="f16", tokens=4099, kv_heads=4, dim=256, page=32),
        # one sequence early in its answer: latency
        dict(name="decode_one_int8", op="attend", fmt="int8", dtype="bf16", batch=1, q_len=1, kv_len=1031, ragged=False,
             kv_heads=8, group=4, dim=128, page=16, window=0, sinks=0),
        # a serving batch of different lengths
        dict(name="decode_batch_fp8", op="attend", fmt="fp8", dtype="bf16", batch=32, q_len=1, kv_len=8192, ragged=True,
             kv_heads=8, group=4, dim=128, page=64, window=0, sinks=0),
        # a few very long contexts in 4 bits
        dict(name="decode_long_int4", op="attend", fmt="int4", dtype="f16", batch=4, q_len=1, kv_len=131072, ragged=False,
             kv_heads=8, group=4, dim=128, page=128, window=0, sinks=0),
        # a large batch of a sliding-window layer whose old pages were given back
        dict(name="decode_window_int8", op="attend", fmt="int8", dtype="bf16", batch=64, q_len=1, kv_len=16384, ragged=True,
             kv_heads=8, group=8, dim=64, page=32, window=4096, sinks=4),
        # a chunk of a long prompt in a sliding-window layer
        dict(name="chunk_window_fp8", op="attend", fmt="fp8", dtype="bf16", batch=1, q_len=2048, kv_len=16384, ragged=False,
             kv_heads=8, group=4, dim=128, page=64, window=4096, sinks=4),
        # prompts of several users in one call, odd sizes
        dict(name="chunk_ragged_int8", op="attend", fmt="int8", dtype="f16", batch=6, q_len=701, kv_len=2999, ragged=True,
             kv_heads=4, group=7, dim=128, page=16, window=0, sinks=0),
        # one user's small draft tree: latency
        dict(name="tree_one_int8", op="tree", fmt="int8", dtype="bf16", batch=1, q_len=13, kv_len=913, ragged=False,
             kv_heads=8, group=4, dim=128, page=16),
        # a serving batch's draft trees
        dict(name="tree_batch_fp8", op="tree", fmt="fp8", dtype="bf16", batch=16, q_len=64, kv_len=8192, ragged=True,
             kv_heads=8, group=4, dim=128, page=64),
        # small trees over a 4-bit cache, narrow heads
        dict(name="tree_narrow_int4", op="tree", fmt="int4", dtype="f16", batch=8, q_len=24, kv_len=6000, ragged=True,
             kv_heads=8, group=2, dim=64, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(("cache", "attend", "attend", "tree")), fmt=rng.choice(("int8", "fp8", "int4")),
                 dtype=rng.choice(("bf16", "f16")))
        shape = dict(kv_heads=rng.choice((1, 2, 4, 8)), dim=rng.choice((64, 128, 128, 256)), page=rng.choice((16, 32, 64, 128)))
        if c["op"] == "cache":
            c.update(tokens=_log(rng, 1, 16383), **shape)
            return c
        c.update(batch=_log(rng, 1, 64), q_len=1, kv_len=_log(rng, 1, 65536), ragged=rng.random() < 0.5,
                 group=rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), **shape)
        if c["op"] == "attend":
            if rng.random() < 0.5:
                c["q_len"] = _log(rng, 1, 2048)
            c["window"] = rng.choice((0, 0, _log(rng, 1, 8192)))
            c["sinks"] = rng.choice((0, 1, 4, 17)) if c["window"] else 0
        else:
            c["q_len"] = _log(rng, 1, 130)
        c["kv_len"] += c["q_len"]
        rows = c["batch"] * c["q_len"] * c["kv_heads"] * c["group"]
        if rows * c["kv_len"] <= 2 ** 29 and c["batch"] * c["kv_len"] * c["kv_heads"] * c["dim"] <= 2 ** 28:
            return c


# ----------------------------------------------------------------- inputs ----

def _spread(most, least, n, ragged):
    """n lengths up to `most`, the first of them `most`: the same for every seed."""
    if not ragged:
        return [most] * n
    return [most if i == 0 else max(least, int(most * (0.3 + 0.7 * ((i * 0.6180339887) % 1.0)))) for i in range(n)]


def _lengths(case):
    q = _spread(case["q_len"], 1, case["batch"], case["ragged"] and case["q_len"] > 1)
    kv = [max(a, b) for a, b in zip(_spread(case["kv_len"], 1, case["batch"], case["ragged"]), q)]
    return q, kv


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


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    h, d, page, fmt = case["kv_heads"], case["dim"], case["page"], case["fmt"]
    s = {"op": case["op"], "dtype": dt}
    if case["op"] == "cache":
        n = case["tokens"]
        pages = n // page + 2
        k, v = _tokens(g, n, h, d, dev)
        # the tokens as the fused projection leaves them: keys and values side by side in a row
        kv = torch.cat((k.view(n, h * d), v.view(n, h * d)), 1).to(dt)
        s["k"], s["v"] = kv[:, :h * d].view(n, h, d), kv[:, h * d:].view(n, h, d)
        slots = torch.randperm(pages, generator=g, device=dev).repeat_interleave(page) * page
        slots = (slots + torch.arange(page, device=dev).repeat(pages))[:n].contiguous()
        if n > 100:  # padding
            slots[torch.rand(n, generator=g, device=dev) < 0.02] = -1
        s["slots"] = slots
        c = _empty_cache(fmt, pages, h, page, d, dev)
    else:
        q_len, kv_len = _lengths(case)
        total, batch, group = sum(q_len), case["batch"], case["group"]
        per = -(-max(kv_len) // page)
        pages = batch * per + 1
        c = _empty_cache(fmt, pages, h, page, d, dev)
        at = (torch.randperm(pages - 1, generator=g, device=dev) + 1).view(batch, per)
        k, v = _tokens(g, pages * page, h, d, dev)
        for t, x in (("k", k), ("v", v)):
            x = x.to(dt).view(pages, page, h, d).transpose(1, 2).contiguous()
            c[t], c[t + "_scale"] = _quantize(x, fmt)
        del k, v
        table = at.to(torch.int32)
        if case["op"] == "attend" and case["window"]:
            # pages that no query of this call or a later one sees were given back
            first = torch.tensor([b - a - case["window"] + 1 for a, b in zip(q_len, kv_len)], device=dev)
            p = torch.arange(per, device=dev)[None]
            gone = ((p + 1) * page <= first[:, None]) & (p * page >= case["sinks"])
            table = torch.where(gone, -1, table)
        # queries as a view of the fused projection's rows
        row = torch.randn(total, (case["group"] + 2) * h * d, generator=g, device=dev) * 1.5
        s["q"] = row.to(dt)[:, :group * h * d].view(total, group * h, d)
        s["table"] = table.contiguous()
        s["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        cu = [0]
        for a in q_len:
            cu.append(cu[-1] + a)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["max_q"], s["max_kv"] = max(q_len), max(kv_len)
        if case["op"] == "attend":
            s["window"], s["sinks"] = case["window"], case["sinks"]
        else:
            s["tree"] = _tree_masks(rng, q_len, dev)
    s["cache"] = c
    if own:
        from bit_gemm_w4_amd import ops
        s["handle"] = ops.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"],
                                  {"int8": ops.I8, "fp8": ops.FP8_E4M3, "int4": ops.U4}[fmt])
    return s


def _tree_masks(rng, q_len, dev):
    """Ancestor bits of each drafted token, itself included: int64 words, bit j of word w is token 64 w + j."""
    words = (max(q_len) + 63) // 64
    rows = []
    for n in q_len:
        bits = []
        for i in range(n):
            up = bits[rng.randrange(max(0, i - 6), i)] if i else 0
            bits.append(up | 1 << i)
        rows += bits
    signed = lambda x: x - (1 << 64) if x >> 63 else x  # noqa: E731
    return torch.tensor([[signed(b >> 64 * w & (1 << 64) - 1) for w in range(words)] for b in rows], dtype=torch.int64, device=dev)


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


def _plain_cache(s):
    c, slots = s["cache"], s["slots"]
    n, page = c["k"].shape[0], c["k"].shape[2]
    held = (slots >= 0) & (slots < n * page)
    # a skipped token writes to the spare page, which no sequence owns
    at = torch.where(held, slots, n * page)
    p, o = at // page, at % page
    out = []
    for t in ("k", "v"):
        codes, record = _quantize(s[t], c["fmt"])
        for name, new in ((t, codes), (t + "_scale", record)):
            old = c[name]
            grown = torch.cat((old, old[:1]))
            grown[p, :, o] = new
            old.copy_(grown[:n])
        x = _values(c[t][p % n, :, o], c[t + "_scale"][p % n, :, o], c["fmt"])
        out.append(torch.where(held[:, None, None], x, 0.0).to(s["dtype"]))
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
    q_len = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + i).clamp(max=total - 1)
    x = q.float()[rows].view(batch, m, heads, group, d).permute(0, 2, 1, 3, 4).reshape(batch, heads, m * group, d)
    held = there.repeat_interleave(page, 1)[:, :length] & (j < lens[:, None])
    at = (lens - q_len)[:, None] + i
    at, kv = at[:, :, None], j[None, None]
    if s["op"] == "attend":
        seen = kv <= at
        if s["window"]:
            seen = seen & ((kv > at - s["window"]) | (kv < s["sinks"]))
    else:
        first = (lens - q_len)[:, None, None]
        bit = (kv - first).clamp(min=0).expand(batch, m, length)
        words = s["tree"][rows]
        w = torch.gather(words, 2, (bit >> 6).clamp(max=words.shape[2] - 1))
        seen = (kv < first) | ((w >> (bit & 63) & 1 == 1) & (bit >> 6 < words.shape[2]))
    seen = (seen & held[:, None]).view(batch, 1, m, 1, length)
    score = torch.matmul(x, k.transpose(2, 3).contiguous()).view(batch, heads, m, group, length) * d ** -0.5
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
        return _plain_cache(s) if s["op"] == "cache" else _plain_attention(s)
    from bit_gemm_w4_amd import ops
    if s["op"] == "cache":
        ops.kv_cache_write(s["k"], s["v"], s["handle"], s["slots"])
        return list(ops.kv_cache_read(s["handle"], s["slots"], s["dtype"]))
    if s["op"] == "attend":
        return ops.kv_attn(s["q"], s["handle"], s["table"], s["kv_lens"], s["cu_q"], s["max_q"], max_kv_len=s["max_kv"],
                           window=s["window"], sinks=s["sinks"])
    return ops.kv_attn_tree(s["q"], s["handle"], s["table"], s["kv_lens"], s["cu_q"], s["tree"], s["max_q"], max_kv_len=s["max_kv"])


# ------------------------------------------------------- work and exactness ----

def work(case):
    h, d = case["kv_heads"], case["dim"]
    token = h * 2 * ((d // 2 if case["fmt"] == "int4" else d) + 4)  # codes and records of a token's keys and values
    if case["op"] == "cache":
        # read the rows, write and read the codes, write the values
        return {"bytes": case["tokens"] * (2 * h * 2 * d * 2 + 2 * token + 16), "flops": case["tokens"] * h * 2 * d * 4}
    q_len, kv_len = _lengths(case)
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    seen, pairs = 0, 0
    for a, b in zip(q_len, kv_len):
        if case["op"] == "tree":
            seen += b
            pairs += a * (b - a) + a
            continue
        low = max(0, b - a - window + 1) if window else 0
        seen += b - low + min(low, sinks)
        for at in range(b - a, b):
            first = max(0, at - window + 1) if window else 0
            pairs += at + 1 - first + min(first, sinks)
    heads = h * case["group"]
    return {"bytes": seen * token + sum(q_len) * heads * d * 2 * 2, "flops": pairs * heads * d * 4}


def _exact_rows(x, fmt):
    """What a quantized row stands for: the codes are defined by quotients in 32 bits, the rest is in 64."""
    x = x.double()
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cache":
        keep = (s["slots"] != -1).double()[:, None, None]
        return [_exact_rows(s[t], case["fmt"]) * keep for t in ("k", "v")]
    c, q = s["cache"], s["q"].double()
    out = torch.zeros_like(q)
    q_len, kv_len = _lengths(case)
    first, page, group, d = 0, case["page"], case["group"], case["dim"]
    for b, (a, length) in enumerate(zip(q_len, kv_len)):
        used = -(-length // page)
        ids = s["table"][b, :used].tolist()
        safe = torch.tensor([max(i, 0) for i in ids], device=q.device)
        j = torch.arange(length, device=q.device)
        at = torch.arange(length - a, length, device=q.device)[:, None]
        if case["op"] == "attend":
            see = (j <= at) & ((at - j < case["window"]) | (j < case["sinks"])) if case["window"] else j <= at
        else:
            see = torch.ones(a, length, dtype=torch.bool, device=q.device)
            words = s["tree"][first:first + a].tolist()
            for i in range(a):
                row = sum((x % (1 << 64)) << 64 * n for n, x in enumerate(words[i]))
                see[i, length - a:] = torch.tensor([bool(row >> e & 1) for e in range(a)], device=q.device)
        for head in range(case["kv_heads"]):
            k, v = (_exact_pages(c[t][safe, head], c[t + "_scale"][safe, head], case["fmt"]).reshape(-1, d)[:length] for t in ("k", "v"))
            for i in range(group):
                x = q[first:first + a, head * group + i] @ k.T / math.sqrt(d)
                x = x.masked_fill(~see, -math.inf)
                out[first:first + a, head * group + i] = torch.softmax(x, -1) @ v
        first += a
    return out
