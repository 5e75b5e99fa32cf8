"""Cases over the paged 4-bit key/value cache: planning a step's pages and slots,
appending to the cache, reading rows back, and attention over the cache.

The plain forms here restate each operator with elementary torch operations;
with ``own`` true the same passes go through the library (`fa.kv4_*`).

Format of the cache, uint8 [num_pages, kv heads, record]: one record holds a
page of one head as K codes [page][d/2], K parameters [page][d/group] pairs of
bf16 (scale, minimum), V codes, V parameters.  Eight channels share a
little-endian 32-bit word: even channels in the four nibbles of its low half,
odd channels in those of its high half.  A value is minimum + scale * code.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_NIB = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble that holds channel c of its word


# ------------------------------------------------------------------ cases

def _plan(name, **k):
    return dict(name=name, op="plan", **k)


def _append(name, **k):
    return dict(name=name, op="append", **k)


def _gather(name, **k):
    return dict(name=name, op="gather", **k)


def _attn(name, **k):
    return dict(name=name, op="attention", **k)


def listed():
    return [
        # one decode step of a small batch: a page is needed now and then
        _plan("plan_decode", batch=16, page=64, max_len=4096, prompt=0, mix=1),
        # a busy server's step: prompts beside decodes, finished requests
        _plan("plan_prompts", batch=1024, page=16, max_len=8192, prompt=2048, mix=2),
        # one new token of each of 32 requests
        _append("append_decode", tokens=32, q_heads=32, kv_heads=8, d=128, group=32, page=64, mix=3),
        # prompts of a long step, ragged end
        _append("append_prompt", tokens=16381, q_heads=16, kv_heads=16, d=128, group=64, page=16, mix=4),
        # a short cached prefix read back
        _gather("gather_short", tokens=515, kv_heads=12, d=64, group=32, page=32, mix=5),
        # a long cached prefix read back for a prompt's attention
        _gather("gather_long", tokens=16384, kv_heads=16, d=128, group=32, page=128, mix=6),
        # one request, short context, as many K/V heads as query heads: latency
        _attn("attn_one_short", batch=1, queries=1, kv_heads=12, per_kv=1, d=64, group=32, page=16,
              min_len=129, max_len=129, window=-1, mix=7),
        # the ordinary decode step: ragged contexts, four query heads a K/V head
        _attn("attn_decode", batch=32, queries=1, kv_heads=8, per_kv=4, d=128, group=32, page=64,
              min_len=512, max_len=8192, window=-1, mix=8),
        # few requests, very long contexts: the longest read of the cache
        _attn("attn_decode_long", batch=3, queries=1, kv_heads=8, per_kv=8, d=128, group=64, page=128,
              min_len=65536, max_len=131072, window=-1, mix=9),
        # drafted tokens checked in one pass, wide heads, sliding window
        _attn("attn_drafts_window", batch=16, queries=5, kv_heads=4, per_kv=2, d=256, group=32, page=32,
              min_len=1024, max_len=16384, window=4096, mix=10),
        # a chunk of a prompt over its cached past
        _attn("attn_chunk", batch=2, queries=1024, kv_heads=8, per_kv=4, d=128, group=32, page=64,
              min_len=8192, max_len=16384, window=-1, mix=11),
        # a short chunk of many requests with narrow heads
        _attn("attn_chunk_short", batch=24, queries=48, kv_heads=4, per_kv=3, d=64, group=64, page=16,
              min_len=48, max_len=1024, window=-1, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "attention", "attention", "attention"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 1024), page=page, max_len=_log(rng, 64, 8192),
                    prompt=rng.choice([0, _log(rng, 8, 2048)]), mix=mix)
    d = rng.choice([64, 128, 256])
    group = rng.choice([32, 64])
    if op != "attention":
        c = dict(op=op, tokens=_log(rng, 1, 16384), kv_heads=rng.choice([1, 2, 4, 8, 12, 16]), d=d, group=group,
                 page=page, mix=mix)
        if op == "append":
            c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4])
        c["tokens"] = max(1, min(c["tokens"], 16381 * 16 * 128 // (c["kv_heads"] * d)))
        return c
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    per_kv = rng.choice([1, 2, 3, 4, 8])
    batch = _log(rng, 1, 32)
    queries = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 512)])
    max_len = max(queries, min(_log(rng, 1, 65536), (1 << 28) // (batch * kv_heads * d)))
    while batch * queries * max_len * kv_heads * per_kv * d > (1 << 35):
        batch, queries = (batch + 1) // 2, (queries + 1) // 2
    min_len = rng.randint(max(1, max_len // 8), max_len)
    window = rng.choice([-1, -1, -1, _log(rng, 1, 4096)])
    return dict(op="attention", batch=batch, queries=queries, kv_heads=kv_heads, per_kv=per_kv, d=d, group=group,
                page=page, min_len=min(min_len, max_len), max_len=max_len, window=window, mix=mix)


# ------------------------------------------------------------------ sizes that follow from a case

def _record(page, d, group):
    return 2 * page * (d // 2 + 4 * (d // group))


def _plan_lengths(c):
    r = random.Random(c["mix"])
    past, new = [], []
    for _ in range(c["batch"]):
        p = r.randint(0, c["max_len"] - 1)
        n = 1
        u = r.random()
        if c["prompt"] and u < 0.05:
            p, n = 0, min(c["max_len"], r.randint(max(1, c["prompt"] // 4), c["prompt"]))
        elif u > 0.97:
            n = -1
        past.append(p)
        new.append(n)
    return past, new


def _attn_lengths(c):
    r = random.Random(c["mix"])
    lens = [r.randint(c["min_len"], c["max_len"]) for _ in range(c["batch"])]
    lens[0] = c["max_len"]
    lo = max(1, (3 * c["queries"]) // 4)
    nq = [min(l, r.randint(lo, c["queries"])) for l in lens]
    nq[0] = min(lens[0], c["queries"])
    return lens, nq


def _visible(length, nq, window):
    """Sum over the queries of the keys each sees, and how many keys any sees."""
    first = length - nq
    if window < 0:
        return nq * first + nq * (nq + 1) // 2, length
    return sum(min(first + t, window) + 1 for t in range(nq)), min(length, nq + window)


def work(case):
    c = case
    if c["op"] == "plan":
        past, new = _plan_lengths(c)
        pg = c["page"]
        pages = sum((p + pg - 1) // pg if n < 0 else (p + n + pg - 1) // pg - (p + pg - 1) // pg
                    for p, n in zip(past, new))
        tokens = sum(max(n, 0) for n in new)
        b = 4 * (2 * c["batch"] + 2 * pages + c["batch"] + c["batch"] + 1 + tokens + 8)
        return {"bytes": b, "flops": 0}
    if c["op"] in ("append", "gather"):
        rows = c["tokens"] * c["kv_heads"]
        wide, narrow = 2 * rows * c["d"] * 2, 2 * rows * (c["d"] // 2 + 4 * (c["d"] // c["group"]))
        slots = 4 * c["tokens"]
        if c["op"] == "append":  # written, then read back
            return {"bytes": 2 * wide + 2 * narrow + slots, "flops": 0}
        return {"bytes": wide + narrow + slots, "flops": 0}
    lens, nq = _attn_lengths(c)
    heads = c["kv_heads"] * c["per_kv"]
    row = 2 * (c["d"] // 2 + 4 * (c["d"] // c["group"])) * c["kv_heads"]
    pairs = keys = 0
    for l, n in zip(lens, nq):
        p, k = _visible(l, n, c["window"])
        pairs, keys = pairs + p, keys + k
    q = sum(nq) * heads
    table = sum((l + c["page"] - 1) // c["page"] for l in lens) * 4
    return {"bytes": keys * row + q * (4 * c["d"] + 4) + table, "flops": 4.0 * c["d"] * heads * pairs}


# ------------------------------------------------------------------ plain arithmetic of the format

def _quantise(x, group):
    """bf16 [..., d] -> codes int32 [..., d], scale and minimum fp32 [..., d/group]."""
    shape = x.shape
    v = x.float().reshape(*shape[:-1], shape[-1] // group, group)
    lo, hi = v.amin(-1), v.amax(-1)
    # next to a border between two scales or two codes 32 bits are not enough
    steps = torch.full((), 15.0, dtype=torch.float64, device=x.device)
    s = ((hi.double() - lo.double()) / steps).float().bfloat16().float()
    q = ((v.double() - lo.double()[..., None]) / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None]).round()
    q = torch.where(s[..., None] > 0, q, torch.zeros_like(q)).clamp(0, 15)
    return q.to(torch.int32).reshape(shape), s, lo


def _pack(codes):
    w = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 8, 8)
    nib = torch.empty_like(w)
    nib[..., _NIB] = w
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8).flatten(-2)


def _params(s, lo):
    p = torch.stack([s.bfloat16(), lo.bfloat16()], -1).flatten(-2)
    return p.contiguous().view(torch.uint8)


def _decode(codes, params, group):
    """uint8 [..., d/2] and [..., 4 d/group] -> fp32 [..., d]."""
    w = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 4, 4)
    nib = torch.stack([w & 15, w >> 4], -1).flatten(-2)
    c = nib[..., _NIB].flatten(-2).float()
    p = params.contiguous().view(torch.bfloat16).float()
    s, lo = p[..., 0::2], p[..., 1::2]
    c = c.reshape(*s.shape, group)
    return (lo[..., None] + s[..., None] * c).flatten(-2)


def _parts(record, page, d, group):
    """Records [..., record] -> K codes, K parameters, V codes, V parameters, each [..., page, bytes]."""
    nc, np_ = page * (d // 2), page * 4 * (d // group)
    cut = torch.split(record, [nc, np_, nc, np_], -1)
    lead = record.shape[:-1]
    return [x.reshape(*lead, page, -1) for x in cut]


def _write(state, k, v):
    page, d, g, cache = state["page"], state["d"], state["group"], state["cache"]
    pg, off = state["slots"].long() // page, state["slots"].long() % page
    parts = _parts(cache, page, d, g)  # views: [pages, heads, page, bytes]
    for x, (pc, pp) in ((k, parts[:2]), (v, parts[2:])):
        codes, s, lo = _quantise(x, g)
        pc[pg, :, off] = _pack(codes)
        pp[pg, :, off] = _params(s, lo)


def _read(state):
    page, d, g, cache = state["page"], state["d"], state["group"], state["cache"]
    pg, off = state["slots"].long() // page, state["slots"].long() % page
    kc, kp, vc, vp = (x[pg, :, off] for x in _parts(cache, page, d, g))
    return _decode(kc, kp, g).bfloat16(), _decode(vc, vp, g).bfloat16()


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _keys_values(gen, n, heads, d):
    """Keys with a channel bias (as rotary-free channels have) and values, bf16 [n, heads, d]."""
    bias = torch.randn(1, heads, d, device=DEV, generator=gen)
    k = (torch.randn(n, heads, d, device=DEV, generator=gen) + bias).bfloat16()
    v = torch.randn(n, heads, d, device=DEV, generator=gen).bfloat16()
    return k, v


def _fill(gen, cache, heads, page, d, group):
    """Every row of the cache quantised from drawn keys and values, some pages at a time."""
    step = max(1, (1 << 26) // (heads * page * d))
    for i in range(0, cache.shape[0], step):
        n = min(step, cache.shape[0] - i)
        k, v = _keys_values(gen, n * page, heads, d)
        parts = _parts(cache[i:i + n], page, d, group)
        for x, pc, pp in ((k, parts[0], parts[1]), (v, parts[2], parts[3])):
            codes, s, lo = _quantise(x, group)
            pc.copy_(_pack(codes).reshape(n, page, heads, -1).transpose(1, 2))
            pp.copy_(_params(s, lo).reshape(n, page, heads, -1).transpose(1, 2))


def prepare(case, seed):
    c, gen = case, _gen(seed)
    if c["op"] == "plan":
        past, new = _plan_lengths(c)
        page, B = c["page"], c["batch"]
        width = (c["max_len"] + page - 1) // page
        held = [(p + page - 1) // page for p in past]
        taken = sum((p + max(n, 0) + page - 1) // page - h for p, n, h in zip(past, new, held))
        num_pages = sum(held) + taken + 64
        ids = torch.randperm(num_pages, device=DEV, generator=gen).to(torch.int32)
        table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
        h = torch.tensor(held, device=DEV)
        own_page = torch.arange(width, device=DEV)[None] < h[:, None]
        table[own_page] = ids[:sum(held)]
        free = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
        head = int(torch.randint(0, num_pages, (1,), device=DEV, generator=gen))
        count = num_pages - sum(held)
        free[(head + torch.arange(count, device=DEV)) % num_pages] = ids[sum(held):]
        total = sum(max(n, 0) for n in new)
        return {"op": "plan", "past": torch.tensor(past, dtype=torch.int32, device=DEV),
                "new": torch.tensor(new, dtype=torch.int32, device=DEV), "table": table, "free": free,
                "free_state": torch.tensor([head, count], dtype=torch.int32, device=DEV), "page": page,
                "max_tokens": max(8, (total + 7) // 8 * 8), "num_pages": num_pages}
    d, group, page, heads = c["d"], c["group"], c["page"], c["kv_heads"]
    if c["op"] in ("append", "gather"):
        T = c["tokens"]
        num_pages = (T + page - 1) // page + 3
        slots = torch.randperm(num_pages, device=DEV, generator=gen)[:, None] * page + \
            torch.arange(page, device=DEV)[None]
        slots = slots.flatten()[page // 3:page // 3 + T].to(torch.int32)
        cache = torch.zeros(num_pages, heads, _record(page, d, group), dtype=torch.uint8, device=DEV)
        state = {"op": c["op"], "page": page, "d": d, "group": group, "cache": cache, "slots": slots}
        if c["op"] == "gather":
            _fill(gen, cache, heads, page, d, group)
            return state
        qkv = torch.empty(T, c["q_heads"] + 2 * heads, d, dtype=torch.bfloat16, device=DEV)
        k, v = _keys_values(gen, T, heads, d)
        qkv[:, :c["q_heads"]] = torch.randn(T, c["q_heads"], d, device=DEV, generator=gen)
        qkv[:, c["q_heads"]:c["q_heads"] + heads] = k
        qkv[:, c["q_heads"] + heads:] = v
        state["k"] = qkv[:, c["q_heads"]:c["q_heads"] + heads]
        state["v"] = qkv[:, c["q_heads"] + heads:]
        return state
    lens, nq = _attn_lengths(c)
    need = [(l + page - 1) // page for l in lens]
    width, num_pages = max(need), sum(need) + 3
    cache = torch.zeros(num_pages, heads, _record(page, d, group), dtype=torch.uint8, device=DEV)
    _fill(gen, cache, heads, page, d, group)
    ids = torch.randperm(num_pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]] = ids[:sum(need)]
    q = torch.randn(sum(nq), heads * c["per_kv"], d, device=DEV, generator=gen).bfloat16()
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    return {"op": "attention", "page": page, "d": d, "group": group, "cache": cache, "table": table, "q": q,
            "cu_q": torch.tensor(cu, dtype=torch.int32, device=DEV),
            "kv_len": torch.tensor(lens, dtype=torch.int32, device=DEV), "max_q": max(nq), "window": c["window"],
            "scale": 1.0 / math.sqrt(d)}


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    s = state
    if s["op"] == "plan":
        return _plan_plain(s)
    if s["op"] == "append":
        _write(s, s["k"], s["v"])
        return dict(zip("kv", _read(s)))
    if s["op"] == "gather":
        return dict(zip("kv", _read(s)))
    return _attention_plain(s)


def _run_own(s):
    from exact_io_aware_40_gb300 import fa
    if s["op"] == "plan":
        kv_len, cu_q, slots, state = fa.kv4_plan(s["past"], s["new"], s["table"], s["free"], s["free_state"],
                                                 s["page"], s["max_tokens"], s["num_pages"])
        return {"kv_len": kv_len, "cu_q": cu_q, "slots": slots, "state": state, "table": s["table"],
                "free": s["free"]}
    if s["op"] == "append":
        fa.kv4_append(s["k"], s["v"], s["slots"], s["cache"], s["page"], s["group"])
        return dict(zip("kv", fa.kv4_gather(s["slots"], s["cache"], s["page"], s["d"], s["group"])))
    if s["op"] == "gather":
        return dict(zip("kv", fa.kv4_gather(s["slots"], s["cache"], s["page"], s["d"], s["group"])))
    o, lse = fa.kv4_attention(s["q"], s["cache"], s["table"], s["cu_q"], s["kv_len"], s["max_q"], s["page"],
                              s["group"], causal=True, scale=s["scale"], window=s["window"])
    return {"o": o, "lse": lse}


def _plan_plain(s):
    page, F, cap = s["page"], s["free"].numel(), s["max_tokens"]
    past, new, table, free = s["past"].long(), s["new"].long(), s["table"], s["free"]
    head, count = s["free_state"].long().unbind()
    width = table.shape[1]
    done = new == -1
    n = new.clamp(min=0)
    old = (past + page - 1) // page
    after = (past + n + page - 1) // page
    bad = (past < 0) | (new < -1) | (past + n > width * page)
    need = torch.where(bad, torch.full_like(n, 1 << 40), after - old)
    pages, tokens = need.cumsum(0), n.cumsum(0)
    ok = (pages <= count) & (tokens <= cap)
    n = torch.where(ok, n, torch.zeros_like(n))
    cu = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
    first = pages - need
    col = torch.arange(width, device=table.device)[None]
    taken = torch.where(ok, need, torch.zeros_like(need))
    fresh = (col >= old[:, None]) & (col < (old + taken)[:, None])
    source = free[(head + torch.where(ok, first, torch.zeros_like(first))[:, None] + col - old[:, None]) % F]
    t = torch.arange(cap, device=table.device)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n.numel() - 1)
    pos = past[b] + t - cu[b]
    idx = (pos // page).clamp(0, width - 1)
    newest = torch.where(fresh, source, table)
    slot = newest[b, idx].long() * page + pos % page
    slots = torch.where(t < cu[-1], slot, torch.full_like(slot, -1)).int()
    gone = torch.where(done, old, torch.zeros_like(old))
    at = (head + count + (gone.cumsum(0) - gone)[:, None] + col) % F
    at = torch.where(col < gone[:, None], at, torch.full_like(at, F))
    ring = torch.cat([free, free[:1]]).scatter(0, at.flatten(), newest.flatten())[:F]
    table.copy_(newest)
    free.copy_(ring)
    used = taken.sum()
    state = torch.stack([(head + used) % F, count - used + gone.sum(), cu[-1], ok.sum()]).int()
    kv_len = torch.where(done, torch.zeros_like(past), past + n).int()
    return {"kv_len": kv_len, "cu_q": cu.int(), "slots": slots, "state": state, "table": table, "free": free}


def _attention_plain(s):
    page, d, g, q = s["page"], s["d"], s["group"], s["q"]
    table, T, window = s["table"], s["max_q"], s["window"]
    B, width = table.shape
    heads = s["cache"].shape[1]
    per = q.shape[1] // heads
    kc, kp, vc, vp = _parts(s["cache"][table.long()], page, d, g)  # [B, width, heads, page, bytes]
    keys = _decode(kc, kp, g).transpose(1, 2).reshape(B, heads, width * page, d)
    values = _decode(vc, vp, g).transpose(1, 2).reshape(B, heads, width * page, d)
    kv_len, cu = s["kv_len"].long(), s["cu_q"].long()
    nq = cu[1:] - cu[:-1]
    t = torch.arange(T, device=q.device)
    padded = q.float()[(cu[:-1, None] + t).clamp(max=q.shape[0] - 1)]           # [B, T, Hq, d]
    padded = padded.reshape(B, T, heads, per, d).transpose(1, 2).reshape(B, heads, T * per, d)
    score = (padded @ keys.transpose(-1, -2)) * s["scale"]
    score = score.reshape(B, heads, T, per, width * page)
    j = torch.arange(width * page, device=q.device)
    pos = (kv_len - nq)[:, None] + t                                            # [B, T]
    see = (j < kv_len[:, None, None]) & (j <= pos[..., None])
    if window >= 0:
        see = see & (j >= pos[..., None] - window)
    score = score.masked_fill(~see[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1)
    values = values.masked_fill(~(j < kv_len[:, None])[:, None, :, None], 0.0)
    o = p.reshape(B, heads, T * per, -1) @ values
    o = o.reshape(B, heads, T, per, d) / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    lse = torch.log(total) + top[..., 0]
    row = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    at = row - cu[b]
    o = o.permute(0, 2, 1, 3, 4)[b, at].reshape(q.shape[0], heads * per, d)
    lse = lse.permute(0, 2, 1, 3)[b, at].reshape(q.shape[0], heads * per)
    return {"o": o.bfloat16(), "lse": lse}


# ------------------------------------------------------------------ 64 bits

def _to_bf16(x):
    """fp64 values rounded to eight significant bits, ties to even."""
    bits = x.contiguous().view(torch.int64)
    bits = bits + (1 << 44) - 1 + ((bits >> 45) & 1)  # 7 of 52 fraction bits stay
    return (bits >> 45 << 45).view(torch.float64)


def _values64(row_codes, row_params, d, group):
    """The fp64 values of rows of bytes, channel by channel."""
    out = torch.empty(*row_codes.shape[:-1], d, dtype=torch.float64, device=row_codes.device)
    p = row_params.contiguous().view(torch.int16).to(torch.int32) << 16
    p = p.view(torch.float32).double()
    for ch in range(d):
        nib = (ch % 2) * 4 + (ch % 8) // 2
        byte = row_codes[..., ch // 8 * 4 + nib // 2].to(torch.int32)
        code = ((byte >> (4 * (nib % 2))) & 15).double()
        gr = ch // group
        out[..., ch] = p[..., 2 * gr] * code + p[..., 2 * gr + 1]
    return out


def _request64(s, page_ids, head):
    """K and V of one head over a list of pages, fp64 [tokens, d]."""
    page, d, g = s["page"], s["d"], s["group"]
    nc, np_ = page * d // 2, page * 4 * (d // g)
    rec = s["cache"][page_ids, head]
    n = rec.shape[0] * page
    got, at = [], 0
    for _ in range(2):
        codes = rec[:, at:at + nc].reshape(n, d // 2)
        par = rec[:, at + nc:at + nc + np_].reshape(n, -1)
        got.append(_values64(codes, par, d, g))
        at += nc + np_
    return got


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            x = s[name].double()
            g = s["group"]
            v = x.unflatten(-1, (-1, g))
            lo = v.min(-1, keepdim=True).values
            span = v.max(-1, keepdim=True).values - lo
            step = _to_bf16(span / torch.full_like(span, 15.0))
            code = torch.floor((v - lo) / step.clamp(min=1e-300) + 0.5)
            tie = (v - lo) == (code - 0.5) * step
            code = torch.where(tie & (code % 2 == 1), code - 1, code).clamp(0, 15)
            out[name] = (lo + step * torch.where(step > 0, code, torch.zeros_like(code))).flatten(-2)
        return out
    if case["op"] == "gather":
        slots = s["slots"].long()
        pg, off = slots // s["page"], slots % s["page"]
        ks, vs = [], []
        for h in range(case["kv_heads"]):
            k, v = _request64(s, torch.arange(s["cache"].shape[0], device=DEV), h)
            ks.append(k[pg * s["page"] + off])
            vs.append(v[pg * s["page"] + off])
        return {"k": torch.stack(ks, 1), "v": torch.stack(vs, 1)}
    lens, nq = _attn_lengths(case)
    per, page = case["per_kv"], s["page"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    row = 0
    for b, (length, n) in enumerate(zip(lens, nq)):
        ids = s["table"][b, :(length + page - 1) // page].long()
        pos = torch.arange(length - n, length, device=DEV)
        j = torch.arange(length, device=DEV)
        hide = j[None] > pos[:, None]
        if case["window"] >= 0:
            hide = hide | (j[None] < pos[:, None] - case["window"])
        for h in range(case["kv_heads"]):
            k, v = (x[:length] for x in _request64(s, ids, h))
            for i in range(h * per, (h + 1) * per):
                z = (s["q"][row:row + n, i].double() @ k.T) / math.sqrt(case["d"])
                z = z.masked_fill(hide, -math.inf)
                l = torch.logsumexp(z, -1)
                o[row:row + n, i] = torch.exp(z - l[:, None]) @ v
                lse[row:row + n, i] = l
        row += n
    return {"o": o, "lse": lse}
