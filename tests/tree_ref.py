"""64-bit definitions of the drafted-tree step and plain models of the page bookkeeping, for the
tests. Written from the definitions in include/gemma_attn.h; nothing here calls the package."""
import math

import torch

SLIDING, GLOBAL, RING = 0, 1, 2


def lines(parents, n):
    """Per node of a tree: its ancestors from the root, and itself."""
    out = []
    for i in range(n):
        p = int(parents[i])
        out.append((out[p] if p >= 0 else []) + [i])
    return out


def keys_of(parents, n, base, kind, window):
    """Truth values [n][base + n]: what each node attends, by cache position."""
    see = torch.zeros(n, base + n, dtype=torch.bool)
    for i, line in enumerate(lines(parents, n)):
        depth = len(line) - 1
        if kind == GLOBAL:
            see[i, :base] = True
        else:
            see[i, :base] = base + depth - torch.arange(base) < window
        for d, m in enumerate(line):
            see[i, base + m] = kind == GLOBAL or depth - d < window
    return see


def attention(q, k, v, see, scale, softcap=0.0):
    """q [n][n_q][d], k, v [len][n_kv][d] (rows that nobody attends may hold anything), see [n][len].
    Returns out [n][n_q][d], sum_j w_j |v_j|, and the largest scale * sum_i |q_i k_i| of a row, in
    fp64."""
    q = q.double()
    see = see.to(q.device)
    any_ = see.any(0)
    k = torch.where(any_[:, None, None], k.double(), torch.zeros((), dtype=torch.float64,
                                                                 device=q.device))
    v = torch.where(any_[:, None, None], v.double(), torch.zeros((), dtype=torch.float64,
                                                                 device=q.device))
    G = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("nhd,jhd->nhj", q, k) * scale
    size = torch.einsum("nhd,jhd->nhj", q.abs(), k.abs()).amax(-1) * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    s = s.masked_fill(~see[:, None, :], -math.inf)
    w = torch.softmax(s, -1)
    return (torch.einsum("nhj,jhd->nhd", w, v), torch.einsum("nhj,jhd->nhd", w, v.abs()),
            size[..., None])


def accept(tokens, parents, nxt, n):
    """(path, token) of one sequence's tree of n >= 1 nodes (lists)."""
    path = [0]
    while True:
        want = nxt[path[-1]]
        child = [c for c in range(n) if parents[c] == path[-1] and tokens[c] == want and want >= 0]
        if not child:
            return path, want
        path.append(child[0])


class Pages:
    """The page bookkeeping one sequence and one position at a time. rows[j][page][h][slot]: the
    pools as lists of host tensors [n_pages][n_kv][page_size][...]."""

    def __init__(self, table, refs, lens, pools, page_size):
        self.table = [list(map(int, r)) for r in table]
        self.refs = list(map(int, refs))
        self.lens = list(map(int, lens))
        self.pools = [p.clone() for p in pools]
        self.ps = page_size

    def free(self, keep_from, keep_to):
        for b, row in enumerate(self.table):
            for k, page in enumerate(row):
                if page >= 0 and not ((k + 1) * self.ps > keep_from[b] and k * self.ps < keep_to[b]):
                    self.refs[page] -= 1
                    row[k] = -1

    def fork(self, src, dst):
        """Returns the forks that were refused."""
        before, refused = [list(r) for r in self.table], []
        lens = list(self.lens)
        for i, (s, d) in enumerate(zip(src, dst)):
            n = len(before)
            if not (0 <= s < n and 0 <= d < n) or d in src or d in dst[:i] or \
                    any(p >= 0 for p in before[d]) or \
                    not 0 <= lens[s] <= len(before[s]) * self.ps:
                refused.append(i)
                continue
            blocks = -(-lens[s] // self.ps)
            self.table[d] = [p if k < blocks else -1 for k, p in enumerate(before[s])]
            for p in self.table[d]:
                if p >= 0:
                    self.refs[p] += 1
            self.lens[d] = lens[s]
        return refused

    def reserve(self, add):
        """Returns True where the free pages ran out."""
        items = []
        for b, row in enumerate(self.table):
            n = self.lens[b]
            if n < 0 or add[b] < 0 or n + add[b] > len(row) * self.ps or add[b] == 0:
                continue
            for k in range(n // self.ps, (n + add[b] - 1) // self.ps + 1):
                items.append((b, k))
        writers = {}
        for b, k in items:
            writers.setdefault(self.table[b][k], []).append((b, k))
        free = [p for p, r in enumerate(self.refs) if r == 0]
        refs0, full = list(self.refs), False
        data = [p.clone() for p in self.pools]
        for b, k in items:
            page = self.table[b][k]
            if page >= 0:
                if refs0[page] == 1:
                    continue
                if refs0[page] == len(writers[page]) and writers[page][0] == (b, k):
                    continue
            if not free:
                full = True
                continue
            new = free.pop(0)
            self.table[b][k] = new
            self.refs[new] = 1
            if page >= 0:
                self.refs[page] -= 1
                rows = max(0, min(self.ps, self.lens[b] - k * self.ps))
                for x, old in zip(self.pools, data):
                    x[new][:, :rows] = old[page][:, :rows]
        return full

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        high = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(high, holes))
        for old, new in to.items():
            self.refs[new], self.refs[old] = self.refs[old], 0
            for x in self.pools:
                x[new] = x[old]
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return n
