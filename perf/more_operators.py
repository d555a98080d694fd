"""Cases of speculative and parallel decoding on a paged cache.

The set serves requests that branch.  ``attention_fwd_paged_tree`` verifies a
tree of drafted tokens, ``paged_compact`` moves the accepted path behind the
context (or the kept tokens of a long one together), ``paged_free`` gives the
pages behind the new ends back, ``paged_fork`` lets further requests continue
from where one stands, on shared pages, and ``paged_copy`` copies the pages
that cannot be shared.

A cache is [num_pages][Hkv][page_size][d].  Lengths follow from the case
alone (spread evenly between two bounds); the seed decides which request has
which, the trees, the pages' order and all values.  Every pass leaves its
state so that the next one does the same.
"""
import math

import torch

own = False

NAMES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a lone user's chat, eight drafted tokens; heads as in the benchmark's headline model
        tree_case("tree_b1_short", 1, 333, 333, 8, 8, 16, 16, 128, 64, 0, "bf16"),
        # small trees under a sliding window, small heads, small pages
        tree_case("tree_b24_window", 24, 1000, 8000, 3, 8, 16, 8, 64, 16, 1024, "fp16"),
        # a serving batch with grouped heads and wide trees, lengths as in the benchmark's packed batch
        tree_case("tree_b32_ragged", 32, 333, 7506, 17, 63, 32, 8, 128, 64, 0, "bf16"),
        # a full batch of long contexts
        tree_case("tree_b64_16k", 64, 8192, 16384, 32, 32, 32, 8, 128, 128, 0, "bf16"),
        # eight samples of one prompt
        fork_case("fork_8_samples", 1, 8, 2000, 2000, 64),
        # 15 beams each of 64 requests with long contexts on small pages
        fork_case("fork_960_beams", 64, 960, 333, 16384, 16),
        # the half-full last pages of those eight samples, and of those beams on large pages
        copy_case("copy_8_pages", 8, 8, 128, 64, "bf16"),
        copy_case("copy_960_pages", 960, 8, 128, 256, "fp16"),
        # accepted paths of a batch of trees
        compact_case("compact_b16_paths", 16, 333, 7506, 64, 64, 1, 8, 8, 128, 64, "bf16"),
        # long contexts from which up to half of the tokens are kept
        compact_case("compact_b8_evict", 8, 4, 4, 16384, 16384, 4096, 8191, 8, 128, 128, "fp16"),
        # rejected drafts
        free_case("free_b16_drafts", 16, 400, 7570, 1, 63, 16, False),
        # a thousand requests end, half of what they hold shared between two
        free_case("free_b1024_ended", 1024, 1, 4096, 0, 0, 16, True),
    ]


def tree_case(name, batch, len_lo, len_hi, new_lo, new_hi, hq, hkv, d, page, window, dtype):
    """len: tokens of context; new: drafted tokens."""
    return {"name": name, "op": "tree", "batch": batch, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
            "new_hi": new_hi, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window, "dtype": dtype}


def fork_case(name, parents, forks, len_lo, len_hi, page, short=False):
    return {"name": name, "op": "fork", "parents": parents, "forks": forks, "len_lo": len_lo, "len_hi": len_hi,
            "page": page, "short": short}


def copy_case(name, pages, hkv, d, page, dtype):
    return {"name": name, "op": "copy", "pages": pages, "hkv": hkv, "d": d, "page": page, "dtype": dtype}


def compact_case(name, batch, len_lo, len_hi, new_lo, new_hi, keep_lo, keep_hi, hkv, d, page, dtype):
    """len: tokens that stay in any case; new: those behind them; keep: how many of these are kept."""
    return {"name": name, "op": "compact", "batch": batch, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
            "new_hi": new_hi, "keep_lo": keep_lo, "keep_hi": keep_hi, "hkv": hkv, "d": d, "page": page, "dtype": dtype}


def free_case(name, batch, len_lo, len_hi, drop_lo, drop_hi, page, shared):
    """drop: tokens that a request gives up; 0: all."""
    return {"name": name, "op": "free", "batch": batch, "len_lo": len_lo, "len_hi": len_hi, "drop_lo": drop_lo,
            "drop_hi": drop_hi, "page": page, "shared": shared}


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "fork", "copy", "compact", "free"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype, d, hkv = rng.choice(["bf16", "fp16"]), rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    if op == "tree":
        group = rng.choice([1, 2, 3, 4, 5, 8])
        most = rng.choice([_log(rng, 1, 8), _log(rng, 9, 64), _log(rng, 65, 256)])
        batch, top = _log(rng, 1, 128), _log(rng, 1, 16384)
        # within the largest listed case: bytes of the cache, pairs of queries and keys
        while batch > 1 and (batch * top * hkv * d > 5e8 or batch * most * (top + most) * hkv * group * d > 1e10):
            batch = (batch + 1) // 2
        c = tree_case("", batch, rng.randint(1, top), top, rng.randint(1, most), most, hkv * group, hkv, d, page,
                      rng.choice([0, 0, _log(rng, 16, 4096)]), dtype)
    elif op == "fork":
        parents, top = _log(rng, 1, 64), _log(rng, 1, 16384)
        c = fork_case("", parents, _log(rng, 1, 960), rng.randint(1, top), top, page, short=rng.random() < 0.3)
    elif op == "copy":
        c = copy_case("", _log(rng, 1, 960), hkv, d, page, dtype)
    elif op == "compact":
        new = _log(rng, 2, 16384)
        most = rng.randint(1, new // 2)
        batch = _log(rng, 1, 64)
        while batch > 1 and batch * new > 131072:
            batch = (batch + 1) // 2
        top = _log(rng, 1, 8192)
        c = compact_case("", batch, rng.randint(1, top), top, new, new, rng.randint(0, most), most, hkv, d, page, dtype)
    else:
        top = _log(rng, 1, 4096)
        drop = rng.choice([0, rng.randint(1, top)])
        c = free_case("", _log(rng, 1, 1024), rng.randint(max(1, drop), top), top, rng.randint(min(1, drop), drop), drop,
                      page, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _spread(lo, hi, n):
    """n whole numbers from hi down to lo, evenly spaced."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _spreads(case, *names):
    return [_spread(case[x + "_lo"], case[x + "_hi"], case["batch"]) for x in names]


def _pages(n, page):
    return -(-n // page)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    i32 = {"dtype": torch.int32, "device": dev}
    page = case["page"]
    s = {"case": case}

    def order(n):
        return torch.randperm(n, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float64)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=NAMES[case["dtype"]])

    def caches(pages):
        s["k_cache"], s["v_cache"] = (normal(pages, case["hkv"], page, case["d"]) for _ in range(2))

    def table(rows, width, more=1):
        """Pages of their own for every cell, and those left over."""
        ids = order(rows * width + more).to(torch.int32)
        s["table"] = ids[: rows * width].reshape(rows, width).contiguous()
        s["pages"] = ids.numel()
        return ids[rows * width:].contiguous()

    if case["op"] == "copy":
        n = case["pages"]
        caches(2 * n + 1)
        ids = order(2 * n + 1).to(torch.int32)
        s["src"], s["dst"] = ids[:n].contiguous(), ids[n:2 * n].contiguous()
        s["rows"] = torch.tensor(_spread(1, page - 1, n), **i32)[order(n)]
        return s

    if case["op"] == "fork":
        parents, forks = case["parents"], case["forks"]
        lens = _spread(case["len_lo"], case["len_hi"], parents)
        need = sum(1 for f in range(forks) if lens[f % parents] % page)
        spare = table(parents + forks, _pages(case["len_hi"], page), need + 5)
        s["free"] = spare[: 3 + need // 2].contiguous() if case["short"] else spare  # a pool that runs out on the way
        s["start"] = torch.tensor([2], **i32)
        rows = order(parents + forks).to(torch.int32)
        s["lens"] = torch.zeros(parents + forks, **i32)
        s["lens"][rows[:parents].long()] = torch.tensor(lens, **i32)
        s["src"] = rows[torch.arange(forks, device=dev) % parents].contiguous()
        s["dst"] = rows[parents:].contiguous()
        s["shares"] = torch.zeros(s["pages"], **i32)
        return s

    batch = case["batch"]
    perm = order(batch)
    if case["op"] == "free":
        old, drop = _spreads(case, "len", "drop")
        if case["drop_hi"] == 0:
            drop = old
        old, drop = (torch.tensor(x, **i32) for x in (old, drop))
        s["old"], s["new"] = old[perm].contiguous(), (old - drop)[perm].contiguous()
        width = _pages(case["len_hi"], page)
        spare = table(batch, width)
        s["shares"] = None
        if case["shared"]:
            # every second request branched off the one before it, halfway through its pages
            s["shares"] = torch.zeros(s["pages"], **i32)
            n = batch // 2
            half = torch.arange(width, device=dev) < ((torch.minimum(s["old"][: 2 * n: 2], s["old"][1: 2 * n: 2]) //
                                                       page + 1) // 2)[:, None]
            s["table"][1: 2 * n: 2] = torch.where(half, s["table"][: 2 * n: 2], s["table"][1: 2 * n: 2])
            s["shares"][s["table"][: 2 * n: 2].flatten().long()] = half.flatten().to(torch.int32)
        # the list once held all pages; what the requests hold has been taken from its front
        s["free"] = torch.cat([torch.full((batch * width,), -1, **i32), spare])
        s["start"] = torch.tensor([batch * width], **i32)
        return s

    keys, new = (torch.tensor(x, **i32)[perm] for x in _spreads(case, "len", "new"))
    width = _pages(case["len_hi"] + case["new_hi"], page)
    table(batch, width)
    caches(s["pages"])
    if case["op"] == "compact":
        keep = torch.tensor(_spreads(case, "keep")[0], **i32)[order(batch)]
        most = case["keep_hi"]
        # some stay where they are, the others come from behind the last one's new place
        stay = (uniform(batch) * (keep + 1)).to(torch.int32) // 2
        at = torch.arange(most, device=dev)
        place = uniform(batch, case["new_hi"])
        cols = torch.arange(case["new_hi"], device=dev)
        place = torch.where((cols >= keep[:, None]) & (cols < new[:, None]), place, 2.0)
        pick = place.argsort(1)[:, :most]  # distinct, in random order
        pick = torch.where(at < (keep - stay)[:, None], pick, 1 << 30).sort(1).values
        from_there = pick.gather(1, (at - stay[:, None]).clamp(0, max(0, most - 1)))
        s["keep"] = torch.where(at < stay[:, None], at, from_there).to(torch.int32)
        s["keep"] = torch.where(at < keep[:, None], s["keep"], -1).contiguous()
        s["base"], s["keep_lens"] = keys.contiguous(), keep.contiguous()
        return s

    cu = torch.zeros(batch + 1, **i32)
    cu[1:] = new.cumsum(0)
    total = sum(_spreads(case, "new")[0])
    s["q"] = normal(total, case["hq"], case["d"])
    # each token hangs on any earlier one, or on the context
    row = torch.arange(total, device=dev)
    i = row - cu[torch.searchsorted(cu, row.to(torch.int32), right=True) - 1]
    s["parents"] = ((uniform(total) * (i + 1)).floor().to(torch.int32) - 1).contiguous()
    s["lens"], s["cu"], s["most"] = (keys + new).contiguous(), cu, case["new_hi"]
    s["window"] = case["window"] or None
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_tree(s):
    import exact_attention_85_gb300 as fa
    return fa.attention_fwd_paged_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                                       s["parents"], s["most"], window=s["window"])


def _own_fork(s):
    import exact_attention_85_gb300 as fa
    shares = s["shares"].clone()  # the counts before the branch are kept
    copies, counts = fa.paged_fork(s["src"], s["dst"], s["lens"], s["table"], s["free"], shares,
                                   page_size=s["case"]["page"], free_start=s["start"])
    return s["table"], s["lens"], shares, copies, counts


def _own_copy(s):
    import exact_attention_85_gb300 as fa
    fa.paged_copy(s["src"], s["dst"], s["k_cache"], s["v_cache"], rows=s["rows"])
    return s["k_cache"], s["v_cache"]


def _own_compact(s):
    import exact_attention_85_gb300 as fa
    fa.paged_compact(s["keep"], s["keep_lens"], s["base"], s["table"], s["k_cache"], s["v_cache"])
    return s["k_cache"], s["v_cache"]


def _own_free(s):
    import exact_attention_85_gb300 as fa
    shares = None if s["shares"] is None else s["shares"].clone()  # the counts before are kept
    counts = fa.paged_free(s["old"], s["new"], s["table"], s["free"], s["start"], page_size=s["case"]["page"],
                           num_pages=s["pages"], shares=shares)
    return (s["free"], counts) if shares is None else (s["free"], counts, shares)


_own = {"tree": _own_tree, "fork": _own_fork, "copy": _own_copy, "compact": _own_compact, "free": _own_free}


def _plain_tree(s):
    q, table, cu, most, window = s["q"], s["table"], s["cu"], s["most"], s["window"]
    total, hq, d = q.shape
    batch, hkv = table.shape[0], s["k_cache"].shape[1]
    dev = q.device

    def keys_of(cache):  # [requests, heads, keys, d] in 32 bits
        return cache[table.long()].transpose(1, 2).flatten(2, 3).float()

    k, v = keys_of(s["k_cache"]), keys_of(s["v_cache"])
    step = torch.arange(most, device=dev)
    rows = (cu[:-1, None] + step).clamp(max=total - 1).long()
    # on[b][i][j]: j is on the path that ends in i
    on = torch.eye(most, device=dev) + (s["parents"][rows][..., None] == step).float()
    for _ in range(max(1, (most - 1).bit_length())):
        on = (on @ on).clamp(max=1.0)
    depth = on.sum(-1).to(torch.int32) - 1
    base = s["lens"] - (cu[1:] - cu[:-1])
    key = torch.arange(k.shape[2], device=dev)
    drafted = key - base[:, None]  # [B, keys]
    at = drafted.clamp(0, most - 1).long()
    see = on.bool().gather(2, at[:, None].expand(-1, most, -1)) & (drafted < (cu[1:] - cu[:-1])[:, None])[:, None]
    see |= (drafted < 0)[:, None]
    if window is not None:
        place = torch.where(drafted < 0, key, base[:, None] + depth.gather(1, at))  # [B, keys]
        see &= place[:, None] > (base[:, None] + depth)[..., None] - window
    see = see[:, None, None].expand(batch, 1, hq // hkv, -1, -1).flatten(2, 3)
    qq = q[rows].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (qq @ k.transpose(2, 3) * (1.0 / math.sqrt(d))).masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
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


def _plain_fork(s):
    page, table, free, start, lens = s["case"]["page"], s["table"], s["free"], s["start"], s["lens"]
    src, dst, shares = s["src"].long(), s["dst"].long(), s["shares"].clone()
    n = lens[src]
    full, part = n // page, n % page
    need = (part > 0).to(torch.int32)
    last = start + need.cumsum(0, dtype=torch.int32)
    served = (need == 0) | (last <= free.numel())
    fresh = torch.where(served & (need > 0), free[(last - 1).clamp(0, free.numel() - 1).long()], -1)
    col = torch.arange(table.shape[1], device=table.device)
    held = (col < full[:, None]) & served[:, None]
    mine = torch.where(held, table[src], table[dst])
    mine = torch.where((col == full[:, None]) & (fresh >= 0)[:, None], fresh[:, None], mine)
    shares.index_add_(0, table[src].flatten().long(), held.flatten().to(torch.int32))
    old = table[src].gather(1, full.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0]
    copies = torch.stack([torch.where(fresh >= 0, old, -1), fresh, torch.where(fresh >= 0, part, 0)])
    table[dst] = mine
    lens[dst] = torch.where(served, n, 0)
    counts = torch.stack([torch.where(served & (need > 0), last, start).max(), (last[-1] - free.numel()).clamp(min=0)])
    return table, lens, shares, copies.to(torch.int32), counts.to(torch.int32)


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    live = (torch.arange(s["case"]["page"], device=src.device) < s["rows"][:, None])[:, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[dst] = torch.where(live, cache[src], cache[dst])
    return s["k_cache"], s["v_cache"]


def _plain_compact(s):
    page, keep, base, table = s["case"]["page"], s["keep"], s["base"][:, None], s["table"]
    at = torch.arange(keep.shape[1], device=keep.device)
    live = at < s["keep_lens"][:, None]
    # what is not kept stands for the token before the first one, which stays where it is
    old, new = torch.where(live, base + keep, base - 1).long(), torch.where(live, base + at, base - 1).long()
    old_page, new_page = table.gather(1, old // page).long(), table.gather(1, new // page).long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[new_page, :, new % page] = cache[old_page, :, old % page]
    return s["k_cache"], s["v_cache"]


def _plain_free(s):
    page, table, free, start = s["case"]["page"], s["table"], s["free"], s["start"]
    first, last = ((s[x] + page - 1) // page for x in ("new", "old"))
    col = torch.arange(table.shape[1], device=table.device)
    gone = ((col >= first[:, None]) & (col < last[:, None])).flatten()
    pages = table.flatten().long()
    shares = None
    if s["shares"] is not None:
        drops = torch.zeros_like(s["shares"]).index_add_(0, pages, gone.to(torch.int32))
        cell = torch.arange(gone.numel(), device=table.device)
        ahead = torch.full((s["pages"],), gone.numel(), device=table.device)
        ahead.scatter_reduce_(0, pages, torch.where(gone, cell, gone.numel()), "amin")
        gone = gone & (drops > s["shares"])[pages] & (ahead[pages] == cell)
        shares = (s["shares"] - drops).clamp(min=0)
    rank = gone.cumsum(0)
    to = torch.where(gone, start + rank - 1 - rank[-1], free.numel())
    longer = torch.cat([free, free.new_zeros(1)])
    longer[to] = torch.where(gone, pages, 0).to(torch.int32)
    free.copy_(longer[:-1])
    counts = torch.cat([start - rank[-1], (rank[-1] - start).clamp(min=0)]).to(torch.int32)
    return (free, counts) if shares is None else (free, counts, shares)


_plain = {"tree": _plain_tree, "fork": _plain_fork, "copy": _plain_copy, "compact": _plain_compact, "free": _plain_free}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    if case["op"] in ("fork", "free"):
        return None  # whole numbers
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] in ("copy", "compact"):
        out = []
        for cache in (s["k_cache"], s["v_cache"]):
            flat = cache.transpose(1, 2).reshape(-1, case["hkv"], case["d"])  # a row a slot
            new = flat.clone()
            if case["op"] == "copy":
                for a, b, n in zip(s["src"].tolist(), s["dst"].tolist(), s["rows"].tolist()):
                    new[b * page:b * page + n] = flat[a * page:a * page + n]
            else:
                for b, n in enumerate(s["keep_lens"].tolist()):
                    t0 = s["base"][b].long()
                    a, z = t0 + s["keep"][b, :n].long(), t0 + torch.arange(n, device=flat.device)
                    cells = s["table"][b].long()
                    new[cells[z // page] * page + z % page] = flat[cells[a // page] * page + a % page]
            out.append(new.reshape(-1, page, case["hkv"], case["d"]).transpose(1, 2).contiguous())
        return tuple(out)
    q = s["q"].double()
    total, hq, d = q.shape
    group = hq // case["hkv"]
    o = torch.empty(total, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(hq, total, dtype=torch.float64, device=q.device)
    lens, cu, parents = s["lens"].tolist(), s["cu"].tolist(), s["parents"].tolist()
    for b, n in enumerate(lens):
        used = s["table"][b, : _pages(n, page)].long()
        k, v = (torch.cat(list(c[used]), 1)[:, :n].double() for c in (s["k_cache"], s["v_cache"]))
        r0, new = cu[b], cu[b + 1] - cu[b]
        base = n - new
        hidden = torch.ones(new, n, dtype=torch.bool)
        for i in range(new):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = parents[r0 + j]
            place = base + len(path) - 1
            low = 0 if s["window"] is None else max(0, place - s["window"] + 1)
            hidden[i, low:base] = False
            for j in path[: s["window"]]:
                hidden[i, base + j] = False
        hidden = hidden.to(q.device)
        for h in range(hq):
            a = (q[r0:r0 + new, h] @ k[h // group].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[h, r0:r0 + new] = torch.logsumexp(a, 1)
            o[r0:r0 + new, h] = torch.softmax(a, 1) @ v[h // group]
    return o, lse


# ------------------------------------------------------------------ work


def work(case):
    page = case["page"]
    if case["op"] == "copy":
        rows = sum(_spread(1, page - 1, case["pages"]))
        return {"bytes": 8 * rows * case["hkv"] * case["d"] + 12 * case["pages"], "flops": 0}
    if case["op"] == "fork":
        lens = _spread(case["len_lo"], case["len_hi"], case["parents"])
        cells = sum(lens[f % case["parents"]] // page for f in range(case["forks"]))
        # a cell read, a cell written, a count read and written; a fork's rows, lengths, new cell and copy
        return {"bytes": 16 * cells + 36 * case["forks"], "flops": 0}
    if case["op"] == "free":
        old, drop = _spreads(case, "len", "drop")
        drop = drop if case["drop_hi"] else old
        cells = sum(_pages(n, page) - _pages(n - m, page) for n, m in zip(old, drop))
        return {"bytes": (16 if case["shared"] else 8) * cells + 8 * len(old) + 12, "flops": 0}
    hkv, d, batch = case["hkv"], case["d"], case["batch"]
    if case["op"] == "compact":
        kept = sum(_spreads(case, "keep")[0])
        # about three quarters of the kept move
        return {"bytes": kept * 3 // 4 * 8 * hkv * d + 4 * kept + 8 * batch, "flops": 0}
    keys, new = _spreads(case, "len", "new")
    hq, window = case["hq"], case["window"]
    read, pairs, rows = 0, 0, sum(new)
    for n, m in zip(keys, new):
        seen = min(n, window - 1) if window else n  # of the context, by a token that hangs on it
        read += seen + m
        pairs += m * (seen + 1)
    return {"bytes": read * hkv * d * 2 * 2 + rows * (hq * (d * 2 * 2 + 4) + 4) + 12 * batch,
            "flops": 4 * d * hq * pairs}
