"""What the operators of branching requests write, request by request, with
whole numbers and lists of rows only."""
import torch

from _paged import pages_of


def fork_reference(src, dst, lens, table, free, start, shares, ps):
    """(lens, table, shares, copies, counts, unsound) of fa_paged_fork."""
    B, width = len(lens), len(table[0])
    num_pages = len(shares)
    lens, table, shares = list(lens), [list(r) for r in table], list(shares)
    copies, at, lacking, unsound = [], start, 0, False
    for s, t in zip(src, dst):
        copies.append((-1, -1, 0))
        if not (0 <= s < B and 0 <= t < B and s != t and 0 <= lens[s] <= width * ps):
            unsound = True
            continue
        n = lens[s]
        full, part = divmod(n, ps)
        if part and at + 1 > len(free):
            lacking += 1
            lens[t] = 0
            continue
        for i in range(full):
            table[t][i] = page = table[s][i]
            if 0 <= page < num_pages:
                shares[page] += 1
            else:
                unsound = True
        if part:
            table[t][full] = new = free[at]
            at += 1
            if 0 <= table[s][full] < num_pages and 0 <= new < num_pages:
                copies[-1] = (table[s][full], new, part)
            else:
                unsound = True
        lens[t] = n
    return lens, table, shares, [list(c) for c in zip(*copies)], [at, lacking], unsound


def free_reference(old, new, table, free, start, shares, ps, num_pages):
    """(free, shares, counts, unsound) of fa_paged_free."""
    free, width = list(free), len(table[0])
    drops, order, unsound = {}, [], False
    for b, (o, n) in enumerate(zip(old, new)):
        if not 0 <= n <= o <= width * ps:
            unsound = True
            continue
        for c in range(pages_of(n, ps), pages_of(o, ps)):
            page = table[b][c]
            if not 0 <= page < num_pages:
                unsound = True
                continue
            if shares is None or page not in drops:
                order.append(page)
            drops[page] = drops.get(page, 0) + 1
    if shares is not None:
        shares = list(shares)
        order = [p for p in order if drops[p] > shares[p]]
        for p, m in drops.items():
            shares[p] = max(0, shares[p] - m)
    lost = max(0, len(order) - start)
    for i, p in enumerate(order[lost:]):
        free[start - len(order) + lost + i] = p
    return free, shares, [max(0, start - len(order)), lost], unsound or lost > 0


def copy_reference(cache, src, dst, rows):
    out = cache.clone()
    for s, t, n in zip(src, dst, rows):
        if s >= 0 and t >= 0:
            out[t, :, :n] = cache[s, :, :n]
    return out


def compact_reference(cache, keep, keep_lens, base, table):
    """The tokens of `cache` [pages, Hkv, ps, d] moved together, from a copy."""
    out, ps = cache.clone(), cache.shape[2]
    for b, n in enumerate(keep_lens):
        for i in range(n):
            a, z = base[b] + keep[b][i], base[b] + i
            out[table[b][z // ps], :, z % ps] = cache[table[b][a // ps], :, a % ps]
    return out


def bits(x):
    """16-bit values as whole numbers, so that NaN equal themselves."""
    return x.view(torch.int16)
