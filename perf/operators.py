"""Cases of the operators that bring prompts and new tokens into a KV cache and attend over the whole of it.

  pages   ts_extend_pages  block table, slot map and offsets of a paged cache from the requests' lengths
  write   ts_write_kv      the new tokens' K and V rows to their slots of the cache
  attn    ts_dense_attn    causal attention of each sequence's newest tokens over all of its cached tokens: whole
                           prompts, chunks of prompts, single tokens; packed or paged caches, grouped heads

`run` with `own` false computes them with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

# (h_q, h_kv, head_dim): the shapes of this repository's workloads and tests
HEADS = [(4, 2, 64), (28, 4, 128), (32, 8, 128), (8, 1, 128), (32, 2, 128), (32, 8, 64)]


def listed():
    def attn(name, heads, page, batch, cached, fresh, lens, fused=False):
        return {"name": name, "op": "attn", "h_q": heads[0], "h_kv": heads[1], "d": heads[2], "page": page, "batch": batch,
                "cached_lo": cached[0], "cached_hi": cached[1], "fresh_lo": fresh[0], "fresh_hi": fresh[1], "lens": lens,
                "fused": fused}

    return [
        # one short prompt of the tiny shape, q, k and v views of one projection's output: latency
        attn("prompt_tiny", (4, 2, 64), 0, 1, (0, 0), (257, 257), 1, True),
        # one whole prompt, before any token is generated
        attn("prompt_8k", (28, 4, 128), 0, 1, (0, 0), (8192, 8192), 2, True),
        # prompts of different lengths packed behind one another, some a few tokens long
        attn("prompts_ragged", (32, 8, 128), 0, 11, (0, 0), (1, 6000), 3, True),
        # the last chunk of a long prompt over a cache of 16-token pages
        attn("chunk_long_paged", (28, 4, 128), 16, 1, (126977, 126977), (2048, 2048), 4),
        # one step of a server: requests that decode beside chunks of prompts
        attn("step_mixed_paged", (32, 8, 128), 16, 24, (100, 30000), (1, 700), 5),
        # a small decode batch on short caches: latency
        attn("decode_small_paged", (28, 4, 128), 16, 4, (300, 2000), (1, 1), 6),
        # a decode batch of ragged long requests, 16-token pages
        attn("decode_ragged_paged", (32, 8, 128), 16, 32, (8192, 65536), (1, 1), 7),
        # one token over a million cached ones: the attention that a selection of tokens replaces
        attn("decode_1m", (28, 4, 128), 0, 1, (1048575, 1048575), (1, 1), 8),
        # a decode step of many requests: few new pages
        {"name": "pages_decode", "op": "pages", "page": 16, "batch": 256, "cached_lo": 50, "cached_hi": 32768, "fresh_lo": 1,
         "fresh_hi": 1, "lens": 9, "pad": 0},
        # prompts admitted and continued: many new pages, a padded slot map
        {"name": "pages_prompts", "op": "pages", "page": 16, "batch": 48, "cached_lo": 1, "cached_hi": 60000, "fresh_lo": 100,
         "fresh_hi": 30000, "lens": 10, "pad": 777},
        # one new token of each request of a decode batch
        {"name": "write_decode", "op": "write", "h_kv": 8, "d": 128, "page": 16, "rows": 64, "pool_rows": 8192, "pad": 3},
        # the K and V rows of a chunk, views of the fused projection's output
        {"name": "write_chunk", "op": "write", "h_kv": 4, "d": 128, "page": 16, "rows": 16384, "pool_rows": 65536, "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prompt", "chunk", "mixed", "decode", "pages", "write"])
    if kind == "pages":
        batch = _log(rng, 1, 512)
        hi = max(1, min(60000, 1500000 // batch))
        fresh = _log(rng, 1, max(1, min(30000, 300000 // batch)))
        return {"op": "pages", "page": rng.choice([8, 16, 32, 64, 128]), "batch": batch, "cached_lo": 0, "cached_hi": _log(rng, 1, hi),
                "fresh_lo": 0 if rng.random() < 0.3 else 1, "fresh_hi": fresh, "lens": rng.randrange(1 << 30), "pad": rng.choice([0, 5])}
    if kind == "write":
        rows = _log(rng, 1, 16384)
        page = rng.choice([8, 16, 64])
        return {"op": "write", "h_kv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]), "page": page, "rows": rows,
                "pool_rows": -(-(rows + rng.randrange(1, 20000)) // page) * page, "pad": rng.choice([0, 1, 9])}
    h_q, h_kv, d = rng.choice(HEADS)
    page = rng.choice([0, 8, 16, 32, 64, 256])
    c = {"op": "attn", "h_q": h_q, "h_kv": h_kv, "d": d, "page": page, "lens": rng.randrange(1 << 30), "fused": False}
    if kind == "prompt":
        batch = rng.choice([1, 1, 2, 5, 9])
        n = _log(rng, 16, 8000 // batch)
        c.update(batch=batch, cached_lo=0, cached_hi=0, fresh_lo=1 if batch > 1 else n, fresh_hi=n, page=0, fused=True)
    elif kind == "chunk":
        batch = rng.choice([1, 1, 2, 4])
        n = _log(rng, 100, 60000 // batch)
        t = _log(rng, 2, 1500)
        c.update(batch=batch, cached_lo=n, cached_hi=n + rng.randrange(1, 500), fresh_lo=t, fresh_hi=t + rng.choice([0, 13]))
    elif kind == "mixed":
        c.update(batch=rng.randrange(2, 40), cached_lo=1, cached_hi=_log(rng, 50, 12000), fresh_lo=1, fresh_hi=_log(rng, 2, 300))
    else:
        batch = _log(rng, 1, 48)
        c.update(batch=batch, cached_lo=0, cached_hi=_log(rng, 64, 800000 // batch), fresh_lo=1, fresh_hi=1)
    return c


def _lengths(case):
    """(cached, fresh) tokens of each request, spread over the logarithm of their ranges."""
    rng = random.Random(case["lens"])

    def one(lo, hi):
        return lo if hi <= lo else _log(rng, max(lo, 1), hi) if lo or rng.random() < 0.9 else 0

    cached, fresh = [], []
    for _ in range(case["batch"]):
        cached.append(one(case["cached_lo"], case["cached_hi"]))
        fresh.append(one(case["fresh_lo"], case["fresh_hi"]))
    return cached, fresh


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _stride(case):
    cached, fresh = _lengths(case)
    return max(1, max(-(-(c + f) // case["page"]) for c, f in zip(cached, fresh)))


def _keys(shape, gen):
    """Keys with the spread of channel sizes that the workloads draw; values are plain normal."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    scale = torch.exp(0.5 * torch.randn(shape[-2:], device="cuda", generator=gen)).to(torch.bfloat16)
    return x.mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"attn": _prepare_attn, "pages": _prepare_pages, "write": _prepare_write}[case["op"]](case, seed, gen)


def _pool(case, counts, gen):
    """A block table [batch, stride] (-1 where unused) over a pool half as large again, pages in random order."""
    used, stride = sum(counts), max(1, max(counts))
    pages = used + used // 2 + 1
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    have = torch.tensor(counts, device="cuda").unsqueeze(1) > torch.arange(stride, device="cuda").unsqueeze(0)
    table = torch.full((len(counts), stride), -1, dtype=torch.int32, device="cuda")
    table[have] = order[:used]
    return table, pages, order[used:].contiguous()


def _prepare_attn(case, seed, gen):
    cached, fresh = _lengths(case)
    h_q, h_kv, d, page = case["h_q"], case["h_kv"], case["d"], case["page"]
    lengths = [c + f for c, f in zip(cached, fresh)]
    off, q_off = _offsets(lengths), _offsets(fresh)
    s = {"op": "attn", "off": off, "q_off": q_off, "page": page, "table": None}
    if case["fused"]:  # the projection's output, [tokens, (h_q + 2 h_kv) d]: nothing cached before
        x = torch.empty((off[-1], h_q + 2 * h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        x[:, h_q:h_q + h_kv] = _keys((off[-1], h_kv, d), gen)
        s["q"], s["k"], s["v"] = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    else:
        rows = off[-1]
        if page:
            s["table"], pages, _ = _pool(case, [-(-n // page) for n in lengths], gen)
            rows = pages * page
        s["q"] = torch.randn((q_off[-1], h_q, d), device="cuda", generator=gen).to(torch.bfloat16)
        s["k"] = _keys((rows, h_kv, d), gen)
        s["v"] = torch.empty((rows, h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    if own:
        import query_aware_kv_ts_b200 as ts
        s["kv"] = ts.KVCache(s["k"], s["v"], off, h_q, page_table=s["table"], page_size=page)
        s["buf"] = ts.DenseBuffers(s["kv"], q_off)
    return s


def _prepare_pages(case, seed, gen):
    cached, fresh = _lengths(case)
    page = case["page"]
    used = [-(-c // page) for c in cached]
    need = sum(-(-(c + f) // page) for c, f in zip(cached, fresh)) - sum(used)
    wide, pages, free = _pool(case, used, gen)
    more = torch.arange(pages, pages + need + 3, dtype=torch.int32, device="cuda")
    free = torch.cat([free, more])
    free = free[torch.randperm(free.numel(), device="cuda", generator=gen)].contiguous()
    table = torch.full((case["batch"], _stride(case)), -1, dtype=torch.int32, device="cuda")
    table[:, :wide.shape[1]] = wide
    total = sum(fresh)

    def empty(n):
        return torch.zeros(n, dtype=torch.int64, device="cuda")

    return {"op": "pages", "page": page, "cached": torch.tensor(cached, device="cuda"), "fresh": torch.tensor(fresh, device="cuda"),
            "free": free, "pool_pages": pages + need + 3, "table": table, "seq_offsets": empty(case["batch"] + 1),
            "q_offsets": empty(case["batch"] + 1), "slots": empty(total + case["pad"]), "pages_used": empty(1)}


def _prepare_write(case, seed, gen):
    h_kv, d, rows, pool = case["h_kv"], case["d"], case["rows"], case["pool_rows"]
    x = torch.empty((rows + case["pad"], 3 * h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    slots = torch.randperm(pool, device="cuda", generator=gen)[:rows + case["pad"]].contiguous()
    slots[rows:] = -1  # rows of the padding go nowhere
    s = {"op": "write", "k_new": x[:, h_kv:2 * h_kv], "v_new": x[:, 2 * h_kv:], "slots": slots,
         "k": torch.empty((pool, h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen),
         "v": torch.empty((pool, h_kv, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)}
    if own:
        import query_aware_kv_ts_b200 as ts
        page = case["page"]
        table = torch.arange(pool // page, dtype=torch.int32, device="cuda").unsqueeze(0)
        s["kv"] = ts.KVCache(s["k"], s["v"], [0, pool // page * page], h_kv, page_table=table, page_size=page)
    return s


def run(state):
    s = state
    if own:
        import query_aware_kv_ts_b200 as ts
        if s["op"] == "attn":
            b = s["buf"]
            ts.ts_dense_attn(s["kv"], s["q"], b.q_offsets_dev, b.q_offsets_host, b.out, b.lse, b.ws)
            return {"out": b.out, "lse": b.lse}
        if s["op"] == "pages":
            ts.ts_extend_pages(s["cached"], s["fresh"], s["page"], s["free"], s["pool_pages"], s["table"], s["seq_offsets"],
                               s["q_offsets"], s["slots"], s["pages_used"])
        else:
            ts.ts_write_kv(s["kv"], s["k_new"], s["v_new"], s["slots"])
    elif s["op"] == "attn":
        return _plain_attn(s)
    elif s["op"] == "pages":
        _plain_pages(s)
    else:
        _plain_write(s)
    if s["op"] == "pages":
        return {n: s[n] for n in ("table", "seq_offsets", "q_offsets", "slots", "pages_used")}
    return {"k": s["k"], "v": s["v"]}


def _rows(s, b):
    """Where the tokens of sequence b are in k and v."""
    lo, hi = s["off"][b], s["off"][b + 1]
    if s["table"] is None:
        return slice(lo, hi)
    i = torch.arange(hi - lo, device="cuda")
    return s["table"][b, i // s["page"]].long() * s["page"] + i % s["page"]


def _plain_attn(s):
    q = s["q"]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    h_q, d, h_kv = q.shape[1], q.shape[2], s["k"].shape[1]
    for b in range(len(s["off"]) - 1):
        lo, hi = s["q_off"][b], s["q_off"][b + 1]
        n, t = s["off"][b + 1] - s["off"][b], hi - lo
        rows = _rows(s, b)
        k, v = s["k"][rows].float().transpose(0, 1), s["v"][rows].float().transpose(0, 1)  # [h_kv, n, d]
        x = q[lo:hi].float().view(t, h_kv, h_q // h_kv, d).permute(1, 2, 0, 3).reshape(h_kv, -1, d)
        x = torch.matmul(x, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(h_q, t, n)
        if t > 1:
            late = torch.arange(n, device="cuda") > torch.arange(n - t, n, device="cuda").unsqueeze(1)
            x.masked_fill_(late, -math.inf)
        top = x.amax(2, keepdim=True)
        x.sub_(top).exp_()
        z = x.sum(2, keepdim=True)
        o = torch.matmul(x.view(h_kv, -1, n), v).view(h_q, t, d) / z
        out[lo:hi] = o.transpose(0, 1)
        lse[lo:hi] = (top + z.log()).squeeze(2).t()
    return {"out": out, "lse": lse}


def _plain_pages(s):
    page, cached, fresh, free, table = s["page"], s["cached"], s["fresh"], s["free"], s["table"]
    have = (cached + page - 1) // page
    new = (cached + fresh + page - 1) // page - have
    first = new.cumsum(0) - new
    col = torch.arange(table.shape[1], device="cuda").unsqueeze(0) - have.unsqueeze(1)
    taken = free[(first.unsqueeze(1) + col).clamp(0, free.numel() - 1)]
    table.copy_(torch.where((col >= 0) & (col < new.unsqueeze(1)), taken, table))
    s["seq_offsets"][1:] = (cached + fresh).cumsum(0)
    s["q_offsets"][1:] = fresh.cumsum(0)
    s["pages_used"].copy_(new.sum().unsqueeze(0))
    i = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(s["q_offsets"][1:], i, right=True).clamp(max=cached.numel() - 1)
    at = cached[b] + i - s["q_offsets"][b]
    slot = table[b, (at // page).clamp(max=table.shape[1] - 1)].long() * page + at % page
    s["slots"].copy_(torch.where(i < s["q_offsets"][-1], slot, -1))


def _plain_write(s):
    keep = s["slots"] >= 0
    s["k"][s["slots"][keep]] = s["k_new"][keep]
    s["v"][s["slots"][keep]] = s["v_new"][keep]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "attn":
        return _exact_attn(case, s)
    if s["op"] == "pages":
        return _exact_pages(case, s)
    k, v = s["k"].double(), s["v"].double()
    at = s["slots"][:case["rows"]]
    k[at], v[at] = s["k_new"][:case["rows"]].double(), s["v_new"][:case["rows"]].double()
    return {"k": k, "v": v}


def _exact_attn(case, s):
    """One query head at a time: the weights of the tokens that it sees, and their mean of V, in 64 bits."""
    cached, fresh = _lengths(case)
    q, group = s["q"], case["h_q"] // case["h_kv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    row = 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        at = _rows(s, b)
        for h in range(case["h_q"]):
            k, v = s["k"][at, h // group].double(), s["v"][at, h // group].double()
            x = q[row:row + f, h].double() @ k.t() / case["d"] ** 0.5
            seen = torch.ones_like(x, dtype=torch.bool).tril(c)
            m = torch.logsumexp(torch.where(seen, x, -math.inf), 1)
            out[row:row + f, h] = (torch.exp(x - m.unsqueeze(1)) * seen) @ v
            lse[row:row + f, h] = m
        row += f
    return {"out": out, "lse": lse}


def _exact_pages(case, s):
    """Request by request, token by token."""
    cached, fresh = _lengths(case)
    page, free, table, slots, used = case["page"], s["free"].tolist(), s["table"].tolist(), [], 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        for p in range(-(-c // page), -(-(c + f) // page)):
            table[b][p] = free[used]
            used += 1
        slots += [table[b][i // page] * page + i % page for i in range(c, c + f)]
    slots += [-1] * case["pad"]

    def whole(v):
        return torch.tensor(v, dtype=torch.int64)

    return {"table": torch.tensor(table, dtype=torch.int32), "seq_offsets": whole(_offsets([c + f for c, f in zip(cached, fresh)])),
            "q_offsets": whole(_offsets(fresh)), "slots": whole(slots), "pages_used": whole([used])}


def work(case):
    if case["op"] == "write":
        row = case["h_kv"] * case["d"] * 2
        return {"bytes": case["rows"] * (4 * row + 8), "flops": 0}
    cached, fresh = _lengths(case)
    if case["op"] == "pages":
        page = case["page"]
        new = sum(-(-(c + f) // page) + (-c // page) for c, f in zip(cached, fresh))
        # lengths in, offsets out; each new page read and entered; a slot for each new token; the last page of a request
        return {"bytes": 16 * len(cached) + 16 * (len(cached) + 1) + 8 * new + 8 * (sum(fresh) + case["pad"]) + 4 * len(cached) + 8,
                "flops": 0}
    seen = sum(f * c + f * (f + 1) // 2 for c, f in zip(cached, fresh))
    q = sum(fresh) * case["h_q"] * case["d"]
    kv = sum(c + f for c, f in zip(cached, fresh)) * case["h_kv"] * case["d"]
    table = sum(-(-(c + f) // case["page"]) for c, f in zip(cached, fresh)) if case["page"] else 0
    return {"bytes": 2 * q + 2 * q + 4 * sum(fresh) * case["h_q"] + 2 * 2 * kv + 4 * table + 16 * (len(cached) + 1),
            "flops": 4.0 * case["h_q"] * case["d"] * seen}
