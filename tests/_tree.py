"""Problems with trees of drafted tokens on a paged cache, and their attention
in 64 bits; the bounds are those of _paged, over the keys that a row sees."""
import math

import numpy as np
import torch

from _paged import U, Problem


def random_tree(r, n, kind):
    """Parents of n tokens: a chain, a star (all follow the context), the last
    few tokens only, or any earlier one."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    if kind == "comb":  # a chain with leaves
        return [max(-1, i - 1 - i % 2) for i in range(n)]
    if kind == "near":
        return [r.randint(max(-1, i - 4), i - 1) for i in range(n)]
    return [r.randint(-1, i - 1) for i in range(n)]


def path_of(parents, i):
    """The tokens from i up to the context."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path


class TreeProblem(Problem):
    def __init__(self, trees, lens, *args, **kw):
        super().__init__(lens, [len(t) for t in trees], *args, **kw)
        self.trees = trees
        flat = [p for t in trees for p in t]
        # rows of no request have any parent
        self.parents = torch.tensor(flat + [77] * (self.total - len(flat)), dtype=torch.int32)

    def visible(self, b, i):
        """Keys that row i of request b sees."""
        n, m = self.lens[b], self.new[b]
        base, path = n - m, path_of(self.trees[b], i)
        low = max(0, base + len(path) - self.window) if self.window else 0
        near = path[:self.window] if self.window else path
        return list(range(low, max(0, base))) + sorted(base + j for j in near if base + j >= 0)

    def reference(self):
        o = np.zeros((self.rows, self.Hq, self.d))
        lse = np.full((self.Hq, self.rows), -np.inf)
        o_tol, lse_tol = np.zeros_like(o), np.zeros_like(lse)
        group, u = self.Hq // self.Hkv, U[self.dtype]
        q, row = self.q.double(), 0
        for b, m in enumerate(self.new):
            for i in range(m):
                keys = self.visible(b, i)
                if keys:
                    qr = q[row].view(self.Hkv, group, self.d)
                    k, v = self.k[b][:, keys], self.v[b][:, keys]
                    x = qr @ k.transpose(1, 2) * self.scale
                    top = x.amax(-1, keepdim=True)
                    p = torch.exp(x - top)
                    s = p.sum(-1, keepdim=True)
                    row_o = (p @ v / s).reshape(self.Hq, self.d).numpy()
                    row_l = (top + torch.log(s)).reshape(self.Hq).numpy()
                    e_s = (self.d * 2.0 ** -23 * self.scale * (qr.abs() @ k.abs().transpose(1, 2)).amax(-1)).reshape(-1)
                    e_x = 2.0 ** -22 * (1 + x.abs().amax(-1).reshape(-1) * math.log2(math.e))
                    e, e_n = (e_s + e_x).numpy(), len(keys) * 2.0 ** -23
                    weight = (p @ v.abs() / s).reshape(self.Hq, self.d).numpy()
                    o[row], lse[:, row] = row_o, row_l
                    o_tol[row] = (2 * (e + u) + 2 * e_n)[:, None] * weight + u * np.abs(row_o) + 2.0 ** -25
                    lse_tol[:, row] = e + e_n + 2.0 ** -22 * (1 + np.abs(row_l))
                row += 1
        return o, lse, o_tol, lse_tol
