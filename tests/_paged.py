"""Problems on a paged cache, their attention in 64 bits, and the bounds of a
kernel's error derived from its arithmetic.

Bounds.  With x = scale q.k, P = exp(x - max), O = sum P V / sum P:
  scores   a dot product of d terms in fp32 is off by at most
           d 2^-23 sum |q_i k_i| scale (accumulations that truncate counted
           as a whole step); call the largest of a row e_s
  exp      2^-22 relative for the instruction, and the argument
           x log2(e) - m with two roundings of values up to 2 max|x| log2(e):
           e_x = 2^-22 + 2^-22 max|x| log2(e)
  P V      P is rounded to the 16-bit type for the tensor cores: u relative;
           n terms summed in fp32: n 2^-23
Every weight is then off by at most e = e_s + e_x + u relatively, the sum of
the weights by as much, so O by at most (2 e + 2 n 2^-23) sum Pbar |V|, Pbar
= P / sum P; storing O adds half a step of its type (2^-25 below fp16's
normal range).  LSE = max + log(sum): e_s + e_x + n 2^-23 + 2^-22 (1 + |LSE|).
"""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def pages_of(n, ps):
    return -(-n // ps)


class Problem:
    """lens[b] keys and new[b] rows of each request; the cache holds NaN
    wherever no request's key lies, and the table names a page outside the
    pool wherever no row of the request sees a key of it."""

    def __init__(self, lens, new, Hq, Hkv, d, page_size, dtype, window=0, prefix=0, seed=0, pad_rows=0, scale=None,
                 extra_cols=1, sharp=1.0):
        g = torch.Generator().manual_seed(1000 * seed + sum(lens) + sum(new))
        self.lens, self.new, self.Hq, self.Hkv, self.d, self.ps = list(lens), list(new), Hq, Hkv, d, page_size
        self.dtype, self.window, self.prefix = dtype, window, prefix
        self.scale = d ** -0.5 if scale is None else scale
        B = len(lens)
        cols = max(pages_of(n, page_size) for n in lens) + extra_cols
        front = pages_of(prefix, page_size)
        used = sum(pages_of(n, page_size) for n in lens) + front
        self.num_pages = used + 3
        ids = torch.randperm(self.num_pages, generator=g)[:used].tolist()
        cache = [torch.full((self.num_pages, Hkv, page_size, d), float("nan"), dtype=dtype) for _ in range(2)]
        self.table = torch.full((max(B, 1), cols), self.num_pages + 7, dtype=torch.int32)

        def fill(n, pages):
            rows = [torch.randn(Hkv, n, d, generator=g).mul_(s).to(dtype) for s in (sharp, 1.0)]
            for i, page in enumerate(pages):
                part = slice(i * page_size, min(n, (i + 1) * page_size))
                for c, r in zip(cache, rows):
                    c[page, :, : part.stop - part.start] = r[:, part]
            return [r.double() for r in rows]

        self.front = [ids.pop() for _ in range(front)]
        pk, pv = fill(prefix, self.front)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            mine = [ids.pop() for _ in range(pages_of(n, page_size))]
            kb, vb = fill(n, mine)
            self.k.append(torch.cat([pk, kb], 1))
            self.v.append(torch.cat([pv, vb], 1))
            first = max(0, n - new[b] + 1 - window) if window else 0  # first key a row sees
            for i, page in enumerate(mine):
                if new[b] and (i + 1) * page_size > first:
                    self.table[b, i] = page
        self.k_cache, self.v_cache = cache
        self.rows = sum(new)
        self.total = max(1, self.rows + pad_rows)
        self.q = torch.randn(self.total, Hq, d, generator=g).to(dtype)
        self.cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.max_new = max(1, max(new))

    def reference(self):
        """O, LSE of the requests' rows and the bounds of their errors."""
        o = np.zeros((self.rows, self.Hq, self.d))
        lse = np.full((self.Hq, self.rows), -np.inf)
        o_tol, lse_tol = np.zeros_like(o), np.zeros_like(lse)
        group = self.Hq // self.Hkv
        q = self.q.double()
        r0 = 0
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            for i in range(m):
                place = self.prefix + n - m + i
                lo = max(0, place - self.window + 1) if self.window else 0
                hi = max(0, min(place + 1, self.prefix + n))
                if hi <= lo:
                    continue
                qr = q[r0 + i].view(self.Hkv, group, self.d)
                k, v = self.k[b][:, lo:hi], self.v[b][:, lo:hi]
                x = qr @ k.transpose(1, 2) * self.scale
                top = x.amax(-1, keepdim=True)
                p = torch.exp(x - top)
                s = p.sum(-1, keepdim=True)
                row_o = (p @ v / s).reshape(self.Hq, self.d).numpy()
                row_l = (top + torch.log(s)).reshape(self.Hq).numpy()
                e_s = (self.d * 2.0 ** -23 * self.scale * (qr.abs() @ k.abs().transpose(1, 2)).amax(-1)).reshape(-1)
                e_x = 2.0 ** -22 * (1 + x.abs().amax(-1).reshape(-1) * math.log2(math.e))
                e_n = (hi - lo) * 2.0 ** -23
                weight = (p @ v.abs() / s).reshape(self.Hq, self.d).numpy()
                e = (e_s + e_x).numpy()
                u = U[self.dtype]
                o[r0 + i], lse[:, r0 + i] = row_o, row_l
                o_tol[r0 + i] = (2 * (e + u) + 2 * e_n)[:, None] * weight + u * np.abs(row_o) + 2.0 ** -25
                lse_tol[:, r0 + i] = e + e_n + 2.0 ** -22 * (1 + np.abs(row_l))
            r0 += m
        return o, lse, o_tol, lse_tol


def check(got_o, got_lse, want, rows):
    """Rows 0 .. rows - 1 of a call's outputs against Problem.reference()."""
    o, lse, o_tol, lse_tol = want
    g = got_o[:rows].double().cpu().numpy()
    assert np.isfinite(g).all(), "O is not finite"
    over = np.abs(g - o) - o_tol
    assert (over <= 0).all(), f"O: {int((over > 0).sum())} elements over their bound, worst by {over.max():.3e}"
    gl = got_lse[:, :rows].double().cpu().numpy()
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty), "LSE: the rows that see nothing differ"
    if (~empty).any():
        over = np.abs(gl[~empty] - lse[~empty]) - lse_tol[~empty]
        assert (over <= 0).all(), f"LSE: over its bound by {over.max():.3e}"
    assert (g.transpose(1, 0, 2)[empty] == 0).all(), "O of a row that sees nothing must be 0"


def tables_reference(cached, new, table, free, start, page_size, total):
    """What fa_paged_tables writes, request by request."""
    table, slots, lens, cu = table.clone(), [], [], [0]
    at, ended, lacking = start, False, 0
    for b, (c, n) in enumerate(zip(cached, new)):
        old, need = pages_of(c, page_size), pages_of(c + n, page_size) - pages_of(c, page_size)
        served = need == 0 or (not ended and at + need <= len(free))
        if served:
            for i in range(need):
                table[b, old + i] = free[at + i]
            at += need
        else:
            ended = True
        lens.append(c + n if served else c)
        cu.append(cu[-1] + n)
        for t in range(c, c + n):
            slots.append(int(table[b, t // page_size]) * page_size + t % page_size if served else -1)
    wanted = sum(pages_of(c + n, page_size) - pages_of(c, page_size) for c, n in zip(cached, new))
    lacking = max(0, wanted - (len(free) - start))
    slots += [-1] * (total - len(slots))
    return table, lens, cu, slots, [at, lacking]
