"""Cases of the paged-cache operators: what is timed and compared.

The set serves a model from a paged key/value cache: ``paged_tables`` gives
requests their pages and new tokens their slots, ``paged_append`` writes the
new keys and values there, ``attention_fwd_paged`` attends to the cache, and
``attention_fwd_paged_prefix`` does so for a batch whose requests share a long
prefix that is stored once.

A cache is [num_pages][Hkv][page_size][d].  Lengths follow from the case
alone (spread evenly between two bounds); the seed decides which request has
which length, the pages' order and all values.
"""
import math

import torch

own = False

NAMES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decoding step of a small batch: a token each
        tables_case("tables_b8_one_token", 8, 64, 100, 2000, 1, 1),
        # a full scheduler step: prompts being read in, half a million tokens
        tables_case("tables_b1024_prompts", 1024, 16, 0, 4096, 1, 1024),
        # one token of each of 16 requests
        append_case("append_16_tokens", 16, 8, 128, 64, "bf16"),
        # the prompts of one step
        append_case("append_32768_tokens", 32768, 8, 128, 16, "bf16"),
        # a lone user's short chat, one token; heads as in the benchmark's headline model
        paged_case("decode_b1_short", 1, 333, 333, 1, 1, 16, 16, 128, 64, 0, "bf16"),
        # ordinary decoding, grouped heads, lengths as in the benchmark's packed batch
        paged_case("decode_b32_ragged", 32, 333, 7506, 1, 1, 32, 8, 128, 64, 0, "bf16"),
        # a full batch of long contexts
        paged_case("decode_b64_16k", 64, 8192, 16384, 1, 1, 32, 8, 128, 128, 0, "bf16"),
        # a few drafted tokens a request under a sliding window, small heads, small pages
        paged_case("draft_b24_window", 24, 1000, 8000, 2, 4, 16, 8, 64, 16, 1024, "fp16"),
        # prompts read in by chunks behind a long context
        paged_case("chunk_b4_512_tokens", 4, 2048, 8192, 500, 512, 32, 8, 128, 64, 0, "bf16"),
        # few requests with a common instruction
        prefix_case("prefix_b4_1000", 4, 1000, 17, 101, 1, 1, 16, 2, 128, 16, 0, "fp16"),
        # a served assistant: long system prompt, short turns
        prefix_case("prefix_b64_8k", 64, 8192, 333, 1024, 1, 1, 32, 8, 128, 64, 0, "bf16"),
        # many questions about one document
        prefix_case("prefix_b256_16k", 256, 16384, 64, 2048, 1, 1, 32, 8, 128, 64, 0, "bf16"),
    ]


def tables_case(name, batch, page, len_lo, len_hi, new_lo, new_hi, short=False):
    return {"name": name, "op": "tables", "batch": batch, "page": page, "len_lo": len_lo, "len_hi": len_hi,
            "new_lo": new_lo, "new_hi": new_hi, "short": short}


def append_case(name, rows, hkv, d, page, dtype):
    return {"name": name, "op": "append", "rows": rows, "hkv": hkv, "d": d, "page": page, "dtype": dtype}


def paged_case(name, batch, len_lo, len_hi, new_lo, new_hi, hq, hkv, d, page, window, dtype):
    return {"name": name, "op": "paged", "batch": batch, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
            "new_hi": new_hi, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window, "dtype": dtype}


def prefix_case(name, batch, prefix, len_lo, len_hi, new_lo, new_hi, hq, hkv, d, page, window, dtype):
    return dict(paged_case(name, batch, len_lo, len_hi, new_lo, new_hi, hq, hkv, d, page, window, dtype),
                op="prefix", prefix=prefix)


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "append", "paged", "paged", "prefix", "prefix"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "tables":
        hi = _log(rng, 1, 1024)
        c = tables_case("", _log(rng, 1, 1024), page, 0, _log(rng, 16, 4096), rng.randint(0, hi), hi,
                        short=rng.random() < 0.3)
    elif op == "append":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        c = append_case("", _log(rng, 1, 32768), hkv, d, page, dtype)
    else:
        d, hkv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
        most = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 9, 512)])
        batch, top = _log(rng, 1, 128), _log(rng, most, 16384)
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        prefix = _log(rng, 100, 16384) if op == "prefix" else 0
        # within the largest listed cases: bytes of the cache, pairs of queries and keys
        while batch > 1 and (batch * top * hkv * d > 5e8 or batch * most * (top + prefix) * hkv * group * d > 1e10):
            batch = (batch + 1) // 2
        while top > most and most * (top + prefix) * hkv * group * d > 1e10:
            top = max(most, top // 2)
        least = rng.randint(most, top)
        args = (least, top, rng.randint(1, most), most, hkv * group, hkv, d, page, window, dtype)
        c = prefix_case("", batch, prefix, *args) if op == "prefix" else paged_case("", batch, *args)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _spread(lo, hi, n):
    """n whole numbers from hi down to lo, evenly spaced."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """(keys, new tokens) of each request; the longest has the most new ones."""
    keys = _spread(case["len_lo"], case["len_hi"], case["batch"])
    new = _spread(case["new_lo"], case["new_hi"], case["batch"])
    return keys, new


def _pages(n, page):
    return -(-n // page)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    i32 = {"dtype": torch.int32, "device": dev}

    def order(n):
        return torch.randperm(n, generator=gen, device=dev)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=NAMES[case["dtype"]])

    page = case["page"]
    s = {"case": case}
    if case["op"] == "append":
        rows, hkv, d = case["rows"], case["hkv"], case["d"]
        pages = _pages(2 * rows, page) + 1
        s["k"], s["v"] = normal(rows, hkv, d), normal(rows, hkv, d)
        s["k_cache"], s["v_cache"] = normal(pages, hkv, page, d), normal(pages, hkv, page, d)
        # whole pages in any order, a prompt's rows one behind the other inside
        slots = order(pages)[:, None] * page + torch.arange(page, device=dev)
        s["slots"] = slots.reshape(-1)[:rows].to(torch.int32).contiguous()
        return s

    batch = case["batch"]
    keys, new = _lengths(case)
    perm = order(batch)
    keys, new = (torch.tensor(x, **i32)[perm] for x in (keys, new))
    cu = torch.zeros(batch + 1, **i32)
    cu[1:] = new.cumsum(0)
    total = sum(_lengths(case)[1])
    if case["op"] == "tables":
        width = _pages(case["len_hi"] + case["new_hi"], page)
        held = _pages(case["len_hi"], page)
        need = sum(_pages(k + n, page) - _pages(k, page) for k, n in zip(*_lengths(case)))
        pages = batch * held + need + 16
        ids = order(pages).to(torch.int32)
        s["table"] = torch.full((batch, width), -1, **i32)
        have = torch.arange(held, device=dev) < ((keys + page - 1) // page)[:, None]
        s["table"][:, :held] = torch.where(have, ids[: batch * held].reshape(batch, held), -1)
        s["free"] = ids[batch * held:].contiguous()
        if case["short"]:  # a pool that runs out on the way
            s["free"] = s["free"][: 1 + need // 2].contiguous()
        s["cached"], s["new"], s["total"], s["pages"] = keys, new, total, pages
        return s

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    width = _pages(case["len_hi"], page)
    prefix = case.get("prefix", 0)
    front = _pages(prefix, page)
    pages = batch * width + front + 1
    s["q"] = normal(total, hq, d)
    s["k_cache"], s["v_cache"] = normal(pages, hkv, page, d), normal(pages, hkv, page, d)
    ids = order(pages).to(torch.int32)
    s["table"] = ids[: batch * width].reshape(batch, width).contiguous()
    s["lens"], s["cu"], s["most"] = keys.contiguous(), cu, case["new_hi"]
    s["front"], s["prefix"] = ids[batch * width:batch * width + front].contiguous(), prefix
    s["window"] = case["window"] or None
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_tables(s):
    import exact_attention_85_gb300 as fa
    out = fa.paged_tables(s["cached"], s["new"], s["table"], s["free"], page_size=s["case"]["page"],
                          num_pages=s["pages"], total=s["total"])
    return (s["table"],) + tuple(out)


def _own_append(s):
    import exact_attention_85_gb300 as fa
    fa.paged_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    return s["k_cache"], s["v_cache"]


def _own_paged(s):
    import exact_attention_85_gb300 as fa
    if s["case"]["new_hi"] == 1:  # one row a request
        return fa.attention_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], window=s["window"])
    return fa.attention_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["most"],
                                  window=s["window"])


def _own_prefix(s):
    import exact_attention_85_gb300 as fa
    args = (s["q"], s["k_cache"], s["v_cache"], s["front"], s["prefix"], s["table"], s["lens"])
    if s["case"]["new_hi"] == 1:
        return fa.attention_fwd_paged_prefix(*args, window=s["window"])
    return fa.attention_fwd_paged_prefix(*args, s["cu"], s["most"], window=s["window"])


_own = {"tables": _own_tables, "append": _own_append, "paged": _own_paged, "prefix": _own_prefix}


def _plain_tables(s):
    page, cached, new, table, free = s["case"]["page"], s["cached"], s["new"], s["table"], s["free"]
    old = (cached + page - 1) // page
    need = (cached + new + page - 1) // page - old
    last = need.cumsum(0)
    first = last - need
    room = free.numel()
    served = (need == 0) | (last <= room)
    col = torch.arange(table.shape[1], device=table.device) - old[:, None]
    take = (col >= 0) & (col < need[:, None]) & served[:, None]
    table.copy_(torch.where(take, free[(first[:, None] + col).clamp(0, room - 1)], table))
    cu = torch.zeros(new.numel() + 1, dtype=torch.int32, device=new.device)
    cu[1:] = new.cumsum(0)
    row = torch.arange(s["total"], dtype=torch.int32, device=new.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    at = cached[b] + row - cu[b]
    slots = torch.where(served[b], table[b, at // page] * page + at % page, -1).to(torch.int32)
    lens = torch.where(served, cached + new, cached)
    counts = torch.stack([torch.where(served, last, 0).max(), (last[-1] - room).clamp(min=0)]).to(torch.int32)
    return table, lens, cu, slots, counts


def _plain_append(s):
    page = s["case"]["page"]
    at, inside = s["slots"] // page, s["slots"] % page
    s["k_cache"][at, :, inside] = s["k"]
    s["v_cache"][at, :, inside] = s["v"]
    return s["k_cache"], s["v_cache"]


def _keys_of(cache, table):
    """[requests, heads, keys, d] in 32 bits from a cache and its block table."""
    pages = cache[table.long()]  # [B, width, Hkv, page, d]
    return pages.transpose(1, 2).flatten(2, 3).float()


def _plain_attention(s):
    q, table, cu, most, window = s["q"], s["table"], s["cu"], s["most"], s["window"]
    total, hq, d = q.shape
    batch, hkv = table.shape[0], s["k_cache"].shape[1]
    dev = q.device
    k, v = _keys_of(s["k_cache"], table), _keys_of(s["v_cache"], table)
    step = torch.arange(most, device=dev)
    rows = (cu[:-1, None] + step).clamp(max=total - 1).long()
    # [B, Hkv, group * most, d]
    qq = q[rows].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    place = (s["lens"] - (cu[1:] - cu[:-1]))[:, None] + step  # [B, most], within the request's own keys
    key = torch.arange(k.shape[2], device=dev)
    see = key <= place[..., None]
    if window is not None:
        see &= key > place[..., None] - window
    see = see[:, None, None].expand(batch, 1, hq // hkv, -1, -1).flatten(2, 3)
    scale = 1.0 / math.sqrt(d)
    score = (qq @ k.transpose(2, 3) * scale).masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["prefix"]:
        front_k = _keys_of(s["k_cache"], s["front"][None])[:, :, : s["prefix"]]
        front_v = _keys_of(s["v_cache"], s["front"][None])[:, :, : s["prefix"]]
        front = qq @ front_k.transpose(2, 3) * scale
        if window is not None:
            far = torch.arange(s["prefix"], device=dev) <= place[..., None] + s["prefix"] - window
            far = far[:, None, None].expand(batch, 1, hq // hkv, -1, -1).flatten(2, 3)
            front.masked_fill_(far, -math.inf)
        top = torch.maximum(top, front.amax(-1, keepdim=True))
        p, r = torch.exp(score - top), torch.exp(front - top)
        sums = p.sum(-1, keepdim=True) + r.sum(-1, keepdim=True)
        o = (p @ v + r @ front_v) / sums
    else:
        p = torch.exp(score - top)
        sums = p.sum(-1, keepdim=True)
        o = p @ v / sums
    lse = (top + torch.log(sums)).squeeze(-1)
    # back to one row a token
    row = torch.arange(total, device=dev)
    b = torch.searchsorted(cu, row.to(torch.int32), right=True) - 1
    i = row - cu[b]
    o = o.unflatten(2, (hq // hkv, most))[b, :, :, i].flatten(1, 2).to(q.dtype)
    lse = lse.unflatten(2, (hq // hkv, most))[b, :, :, i].flatten(1, 2).t().contiguous()
    return o, lse


_plain = {"tables": _plain_tables, "append": _plain_append, "paged": _plain_attention, "prefix": _plain_attention}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        out = [s["k_cache"].double(), s["v_cache"].double()]
        for cache, x in zip(out, (s["k"], s["v"])):
            flat = cache.transpose(1, 2).reshape(-1, case["hkv"], case["d"]).clone()
            flat[s["slots"].long()] = x.double()
            cache.copy_(flat.reshape(cache.shape[0], case["page"], case["hkv"], case["d"]).transpose(1, 2))
        return tuple(out)
    q = s["q"].double()
    total, hq, d = q.shape
    group = hq // case["hkv"]
    o = torch.empty(total, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(hq, total, dtype=torch.float64, device=q.device)
    prefix, page = s["prefix"], case["page"]
    lens, cu = s["lens"].tolist(), s["cu"].tolist()

    def stored(cache, ids, n):  # the first n tokens of a list of pages: [Hkv, n, d]
        return torch.cat([x for x in cache[ids.long()]], 1)[:, :n].double() if n else cache[0, :, :0].double()

    front = [stored(c, s["front"], prefix) for c in (s["k_cache"], s["v_cache"])]
    for b, n in enumerate(lens):
        used = s["table"][b, : _pages(n, page)]
        k, v = (torch.cat([f, stored(c, used, n)], 1) for f, c in zip(front, (s["k_cache"], s["v_cache"])))
        new = cu[b + 1] - cu[b]
        place = prefix + n - new + torch.arange(new, device=q.device)[:, None]
        key = torch.arange(prefix + n, device=q.device)[None]
        hidden = key > place
        if s["window"] is not None:
            hidden |= key <= place - s["window"]
        for h in range(hq):
            x = q[cu[b]:cu[b + 1], h]
            a = (x @ k[h // group].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[h, cu[b]:cu[b + 1]] = torch.logsumexp(a, 1)
            o[cu[b]:cu[b + 1], h] = torch.softmax(a, 1) @ v[h // group]
    return o, lse


# ------------------------------------------------------------------ work


def work(case):
    if case["op"] == "append":
        elements = case["rows"] * case["hkv"] * case["d"]
        return {"bytes": 2 * 2 * 2 * elements + 4 * case["rows"], "flops": 0}
    keys, new = _lengths(case)
    if case["op"] == "tables":
        page = case["page"]
        need = sum(_pages(k + n, page) - _pages(k, page) for k, n in zip(keys, new))
        # lengths and one held page a request in; pages in, cells and slots out; lengths, offsets, counts out
        return {"bytes": 4 * (3 * len(keys) + 2 * need + sum(new) + 2 * len(keys) + 3), "flops": 0}
    hq, hkv, d, window = case["hq"], case["hkv"], case["d"], case["window"]
    prefix = case.get("prefix", 0)
    read, pairs, front = 0, 0, 0
    for n, m in zip(keys, new):
        p0, p1 = prefix + n - m, prefix + n - 1  # places of the first and the last new token
        low = max(0, p0 - window + 1) if window else 0
        read += prefix + n - max(low, prefix)
        front = max(front, prefix - low)
        if window:
            pairs += sum(min(p + 1, window) for p in range(p0, p1 + 1))
        else:
            pairs += m * (p0 + p1 + 2) // 2
    read += max(0, front)
    rows = sum(new)
    return {"bytes": read * hkv * d * 2 * 2 + rows * hq * (d * 2 * 2 + 4) + 4 * (3 * len(keys)),
            "flops": 4 * d * hq * pairs}
