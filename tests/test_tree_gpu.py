"""Attention of a drafted tree, acceptance and the move of the accepted rows on the GPU, against
their definitions in 64 bits (tests/tree_ref.py)."""
import math

import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref
from tree_ref import GLOBAL, RING, SLIDING

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def random_tree(gen, n, spread=1.0):
    p = [-1]
    for i in range(1, n):
        u = torch.rand(1, generator=gen).item()
        p.append(-1 if spread > 1 and u > 0.95 else min(i - 1, int(u ** (1 / spread) * i)))
    return p


class Problem:
    """Sequences with their trees in a plain, ring or paged cache; every cache row that no node
    attends is NaN."""

    def __init__(self, lens, reals, nodes, kind=GLOBAL, window=0, n_q=4, n_kv=2, d=64, k_eq_v=False,
                 softcap=0.0, page=0, dtype=torch.bfloat16, seed=0, parents=None, cap=None,
                 q_gain=1.0):
        gen = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.kind, self.window, self.n_kv, self.k_eq_v, self.softcap = kind, window, n_kv, k_eq_v, softcap
        self.lens, self.reals, self.nodes, self.dtype = lens, reals, nodes, dtype
        self.msl = max(max(lens), 1)
        self.scale = 1 / math.sqrt(d)
        self.parents = parents or [random_tree(gen, nodes, [0.5, 1.0, 2.0][b % 3]) for b in range(B)]
        self.q = (q_gain * torch.randn(B, nodes, n_q, d, generator=gen)).to(dtype).cuda()
        self.table = None
        if page:
            per = -(-self.msl // page) + 1
            order = torch.randperm(B * per, generator=gen)[:B * per].reshape(B, per)
            self.table = order.int().cuda()
            shape = (B * per + 1, n_kv, page, d)
        elif kind == RING:
            shape = (B, n_kv, cap or -(-(window + nodes - 1) // 128) * 128, d)
        else:
            shape = (B, n_kv, cap or self.msl, d)
        self.k = torch.full(shape, NAN, dtype=dtype, device="cuda")
        self.v = None if k_eq_v else torch.full(shape, NAN, dtype=dtype, device="cuda")
        self.ref, self.bound = [], []
        for b, (n_all, n) in enumerate(zip(lens, reals)):
            base = n_all - n
            see = tree_ref.keys_of(self.parents[b], n, base, kind, window)
            rows = torch.nonzero(see.any(0))[:, 0] if n else torch.zeros(0, dtype=torch.long)
            kk = torch.full((n_all, n_kv, d), NAN, dtype=dtype)
            kk[rows] = torch.randn(len(rows), n_kv, d, generator=gen).to(dtype)
            vv = kk if k_eq_v else torch.full((n_all, n_kv, d), NAN, dtype=dtype)
            if not k_eq_v:
                vv[rows] = torch.randn(len(rows), n_kv, d, generator=gen).to(dtype)
            for cache, x in ((self.k, kk), (self.v, vv)):
                if cache is not None:
                    xr = x[rows].cuda()
                    r = rows.cuda()
                    if page:
                        cache[self.table[b].long()[r // page], :, r % page] = xr
                    else:
                        cache[b][:, r % shape[2] if kind == RING else r] = xr.transpose(0, 1)
            if n:
                out, mass, size = tree_ref.attention(self.q[b, :n].cuda(), kk.cuda(), vv.cuda(), see,
                                                     self.scale, softcap)
                self.ref.append(out)
                self.bound.append(self.tolerance(out, mass, size, d, int(see.sum(1).max())))
            else:
                self.ref.append(None)
                self.bound.append(None)

    def tolerance(self, ref, mass, size, d, n_keys):
        """Half a step of each rounding. bf16: the output's rounding, and P's, which moves a weight
        by at most 2^-8 of itself in the sum and in its normaliser (errors weigh |v - out|). fp32
        sums of the d products of a score, `size` the largest sum of their absolute values, in
        matrix instructions of 16 (or lanes of 32): one rounding per addition, twice since they also
        enter the normaliser; exponentials 2^-21; a soft-cap's tanh 2^-21 of the cap; sums of the
        weighted values one rounding per 16 keys."""
        if self.dtype == torch.float32:
            rel = 2 * (d / 32 + 8) * 2.0 ** -24 * size + 2.0 ** -20 + n_keys * 2.0 ** -23
            rel = rel + 2 * self.softcap * 2.0 ** -22
            return rel * (mass + ref.abs()) + 1e-12
        rel = 2 * (d / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -20 + (n_keys / 16 + 64) * 2.0 ** -23
        rel = rel + 2 * self.softcap * 2.0 ** -21
        return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel) * (mass + ref.abs()) + 1e-12

    def run(self, stream=None, out=None, ws=None, real=True):
        B = len(self.lens)
        out = torch.full_like(self.q, NAN) if out is None else out
        n = g.gemma_attn_workspace_size_tree(B, self.kind, self.window, self.q.shape[2], self.n_kv,
                                             self.q.shape[3], self.msl, self.nodes)
        ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        err = i32([0])
        g.gemma_attn_tree(out, self.q, [self.k], [self.v], [0], 0, i32(self.lens), i32(self.parents),
                          self.msl, kind=self.kind, window=self.window, n_kv=self.n_kv,
                          k_eq_v=self.k_eq_v, scale=self.scale, softcap=self.softcap,
                          n_real=i32(self.reals) if real else None, block_table=self.table,
                          workspace=ws, device_error=err, stream=stream)
        torch.cuda.synchronize()
        self.err = err.item()
        return out

    def check(self, out, skipped=()):
        for b, n in enumerate(self.reals):
            if b in skipped:
                assert (out[b] == 0).all()
                continue
            assert (out[b, n:] == 0).all()
            if n:
                e = (out[b, :n].double() - self.ref[b]).abs()
                assert (e <= self.bound[b]).all(), (b, e.max().item(), (e / self.bound[b]).max().item())


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("group,nodes", [(1, 1), (1, 16), (2, 9), (4, 8), (8, 5), (16, 4), (16, 13),
                                         (4, 128), (1, 128), (2, 33)])
def test_every_head_dim_and_row_count(d, group, nodes):
    """1 to 512 rows per KV head, whole row tiles and odd ones, over a few hundred keys."""
    p = Problem([nodes + 301, nodes, nodes + 64], [nodes, nodes, max(1, nodes - 1)], nodes,
                n_q=2 * group, n_kv=2, d=d, seed=d + group + nodes)
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("kind,window", [(SLIDING, 1), (SLIDING, 3), (SLIDING, 64), (SLIDING, 100),
                                         (RING, 100), (RING, 1), (GLOBAL, 0)])
@pytest.mark.parametrize("d,k_eq_v", [(64, False), (256, True), (512, True), (512, False)])
def test_windows(kind, window, d, k_eq_v):
    """Windows shorter than the tree is deep, of a key tile and between; a ring that has wrapped."""
    nodes = 24
    chain = [i - 1 for i in range(nodes)]
    gen = torch.Generator().manual_seed(1)
    p = Problem([700, 24, 25, 130], [24, 24, 20, 1], nodes, kind, window, 4, 2, d, k_eq_v, seed=3,
                parents=[chain, random_tree(gen, nodes), random_tree(gen, nodes, 2.0), chain])
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("kind,window", [(GLOBAL, 0), (SLIDING, 200)])
@pytest.mark.parametrize("d", [64, 256, 512])
def test_pages_and_softcap(page, kind, window, d):
    p = Problem([1100, 129, 128, 500], [17, 2, 30, 0], 30, kind, window, 8, 2, d, False, 20.0, page,
                seed=page + d, q_gain=4.0)
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("kind,window,page", [(GLOBAL, 0, 0), (SLIDING, 40, 128), (RING, 90, 0)])
def test_fp32(d, kind, window, page):
    p = Problem([333, 5, 90], [17, 5, 9], 17, kind, window, 4, 2, d, d == 128, 30.0 if page else 0.0,
                page, torch.float32, seed=d)
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("n_q,n_kv,d,k_eq_v,lens,nodes", [
    (8, 2, 256, False, [4100], 16),                     # split over keys, one row tile per head
    (16, 1, 512, True, [5000], 32),                     # several row tiles, split
    (16, 1, 512, True, [3000, 100, 2111, 64], 64),      # ragged
    (4, 4, 128, False, [6000, 10], 128),
    (16, 8, 256, False, [1500] * 20, 32),               # many units, no split
])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
def test_long_contexts(n_q, n_kv, d, k_eq_v, lens, nodes, softcap):
    p = Problem(lens, [min(nodes, n) for n in lens], nodes, GLOBAL, 0, n_q, n_kv, d, k_eq_v, softcap,
                seed=len(lens))
    p.check(p.run())
    assert p.err == 0


def test_chain_is_the_prefill_step():
    """parents[i] = i - 1 attends as gemma_attn_prefill: both within the bound of the same values."""
    nodes = 12
    p = Problem([200, 77], [nodes, nodes], nodes, SLIDING, 50, 4, 2, 128, seed=8,
                parents=[[i - 1 for i in range(nodes)]] * 2)
    out = p.run(real=False)
    p.check(out)
    pre = torch.empty_like(out)
    g.gemma_attn_prefill(pre, p.q, [p.k], [p.v], [0], 0, i32(p.lens), p.msl, kind=SLIDING, window=50,
                         n_kv=2, k_eq_v=False, scale=p.scale)
    torch.cuda.synchronize()
    p.check(pre)


def test_shared_layers_read_their_owners_cache():
    p = Problem([100], [6], 6, n_q=4, n_kv=2, d=64)
    out = torch.empty_like(p.q)
    ws = torch.empty(max(16, g.gemma_attn_workspace_size_tree(1, GLOBAL, 0, 4, 2, 64, 100, 6)),
                     dtype=torch.uint8, device="cuda")
    g.gemma_attn_tree(out, p.q, [p.k, None, None], [p.v, None, None], [0, 0, 0], 2, i32([100]),
                      i32(p.parents), 100, kind=GLOBAL, window=0, n_kv=2, k_eq_v=False,
                      scale=p.scale, workspace=ws)
    torch.cuda.synchronize()
    p.check(out)


@pytest.mark.parametrize("d,nodes", [(64, 6), (256, 40), (512, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_sequences_are_skipped(d, nodes, dtype):
    """A bad length, n_real or tree zeros its sequence, sets its bit, and leaves the others alone."""
    def problem():
        return Problem([600, 500, 400, 300], [nodes] * 4, nodes, n_q=16, n_kv=1, d=d, k_eq_v=True,
                       dtype=dtype, seed=4)
    p = problem()
    p.lens = [600, 5, 601, 300]                          # fewer than the nodes; beyond max_seq_len
    p.check(p.run(), skipped=(1, 2))
    assert p.err == g.GEMMA_DEVERR_SEQ_LEN
    for bad in (-1, nodes + 1):
        p = problem()
        p.reals = [nodes, bad, nodes, nodes]
        p.check(p.run(), skipped=(1,))
        assert p.err == g.GEMMA_DEVERR_N_REAL
    for at, parent in ((0, 0), (nodes - 1, nodes - 1), (3, 4), (2, -2), (5, 1 << 30)):
        p = problem()
        p.parents = [list(x) for x in p.parents]
        p.parents[2][at] = parent
        p.check(p.run(), skipped=(2,))
        assert p.err == g.GEMMA_DEVERR_TREE


def test_a_bad_page_reads_as_zeros():
    """Two pages of the prefix out of range: the rest of the keys, and zeros in their place."""
    p = Problem([900], [7], 7, n_q=4, n_kv=2, d=64, page=128, seed=2)
    table = p.table.clone()
    p.table[0, 1], p.table[0, 3] = -1, p.k.shape[0]
    out = p.run()
    assert p.err == g.GEMMA_DEVERR_PAGE
    k, v = (x[table[0].long()].transpose(0, 1).reshape(2, -1, 64)[:, :900].transpose(0, 1).clone()
            for x in (p.k, p.v))
    for x in (k, v):
        x[128:256] = 0
        x[384:512] = 0
    see = tree_ref.keys_of(p.parents[0], 7, 893, GLOBAL, 0)
    ref, mass, size = tree_ref.attention(p.q[0], k, v, see, p.scale)
    assert ((out[0].double() - ref).abs() <= p.tolerance(ref, mass, size, 64, 900)).all()


def test_rows_behind_the_tree_and_unread_parents():
    """Entries of parents behind a sequence's own nodes are not read as nodes."""
    p = Problem([300, 40], [5, 1], 20, n_q=8, n_kv=1, d=128, seed=6)
    p.parents = [x[:n] + [99] * (20 - n) for x, n in zip(p.parents, p.reals)]
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens", [(8, 2, 256, 8, [2048]),
                                                   (16, 1, 512, 32, [2000, 900])])
def test_other_streams_graphs_and_workspaces(n_q, n_kv, d, nodes, lens):
    """On a side stream, captured and replayed with new contents, two graphs on one workspace."""
    p = Problem(lens, [nodes] * len(lens), nodes, n_q=n_q, n_kv=n_kv, d=d, seed=5)
    r = Problem(lens, [nodes] * len(lens), nodes, n_q=n_q, n_kv=n_kv, d=d, seed=6)
    first = p.run()
    side = torch.cuda.Stream()
    assert torch.equal(first, p.run(stream=side))
    args = dict(kind=GLOBAL, window=0, n_kv=n_kv, k_eq_v=False, scale=p.scale)
    ws = torch.empty(max(16, g.gemma_attn_workspace_size_tree(len(lens), GLOBAL, 0, n_q, n_kv, d, p.msl,
                                                     nodes)), dtype=torch.uint8, device="cuda")
    outs, graphs, keep = [], [], []
    for x in (p, r):
        out, ln, pa = torch.empty_like(x.q), i32(x.lens), i32(x.parents)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gemma_attn_tree(out, x.q, [x.k], [x.v], [0], 0, ln, pa, x.msl, workspace=ws, **args)
        outs.append(out)
        graphs.append(graph)
        keep.append((ln, pa))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first)
    r.check(outs[1])
    p.q.copy_(r.q)                                      # new contents behind the same addresses
    p.k.copy_(r.k)
    p.v.copy_(r.v)
    keep[0][1].copy_(keep[1][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_same_call_same_bits():
    p = Problem([5000, 3333], [64, 60], 64, n_q=16, n_kv=1, d=512, k_eq_v=True, seed=9)
    a = p.run()
    for _ in range(4):
        assert torch.equal(a, p.run())


# ---- acceptance ----------------------------------------------------------------------------------
@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 33, 64, 100, 128])
def test_accept(nodes):
    gen = torch.Generator().manual_seed(nodes)
    B = 70
    parents = [random_tree(gen, nodes, [0.5, 1.0, 3.0][b % 3]) for b in range(B)]
    parents[1] = [i - 1 for i in range(nodes)]           # a chain that holds to its end
    tokens = torch.randint(0, 3, (B, nodes), generator=gen)
    nxt = torch.randint(-1, 3, (B, nodes), generator=gen)
    nxt[1, :-1] = tokens[1, 1:]
    real = torch.randint(0, nodes + 1, (B,), generator=gen)
    real[1], real[2] = nodes, 0
    lens = 1000 + torch.arange(B)
    path, keep, token = (torch.full(s, -7, dtype=torch.int32, device="cuda")
                         for s in ((B, nodes), (B,), (B,)))
    ln, err = i32(lens.tolist()), i32([0])
    g.gemma_tree_accept(i32(tokens.tolist()), i32(parents), i32(nxt.tolist()), path, keep, token,
                        n_real=i32(real.tolist()), seq_lens=ln, lens_out=ln, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for b in range(B):
        n = int(real[b])
        want, tok = tree_ref.accept(tokens[b].tolist(), parents[b], nxt[b].tolist(), n) if n else ([], -1)
        assert path[b].tolist() == want + [-1] * (nodes - len(want))
        assert keep[b].item() == len(want) and token[b].item() == (tok if n else -1)
        assert ln[b].item() == int(lens[b]) - n + len(want)


def test_accept_bad_sequences():
    B, n = 6, 5
    tokens, nxt = i32([[1] * n] * B), i32([[1] * n] * B)
    parents = [[-1, 0, 1, 2, 3] for _ in range(B)]
    parents[1][3] = 3
    parents[2][0] = 0
    real = [5, 5, 5, -1, 6, 5]
    lens = [9, 9, 9, 9, 9, 4]
    path, keep, token, out = (torch.zeros(s, dtype=torch.int32, device="cuda")
                              for s in ((B, n), (B,), (B,), (B,)))
    err = i32([0])
    g.gemma_tree_accept(tokens, i32(parents), nxt, path, keep, token, n_real=i32(real),
                        seq_lens=i32(lens), lens_out=out, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == g.GEMMA_DEVERR_TREE | g.GEMMA_DEVERR_N_REAL | g.GEMMA_DEVERR_SEQ_LEN
    assert keep.tolist() == [5, 0, 0, 0, 0, 0] and token.tolist() == [1] + [-1] * 5
    assert out.tolist() == [9, 4, 4, 9, 9, 4]
    assert path[0].tolist() == [0, 1, 2, 3, 4] and (path[1:] == -1).all()


# ---- keep ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,page", [(GLOBAL, 0), (RING, 0), (GLOBAL, 128), (SLIDING, 256)])
@pytest.mark.parametrize("tail,dtype", [((256,), torch.bfloat16), ((64,), torch.float32),
                                        ((128,), torch.uint8), ((4,), torch.bfloat16),
                                        ((2,), torch.bfloat16), ((1,), torch.bfloat16)])
@pytest.mark.parametrize("nodes", [1, 7, 128])
def test_keep(kind, page, tail, dtype, nodes):
    """Rows of every width, paths from none of the nodes to all of them, rings that wrap, pages whose
    edge lies inside the tree; every other row stays."""
    gen = torch.Generator().manual_seed(nodes + len(tail))
    B, n_kv, cap = 5, 3, 512
    paths, keeps = [], [0, 1, nodes, min(nodes, 9), max(1, nodes // 2)]
    for k in keeps:
        pick = sorted(torch.randperm(nodes, generator=gen)[:k].tolist())
        paths.append(pick + [-1] * (nodes - k))
    pos = [100, 120, 250, 384, 0] if kind != RING else [500, 5000, 2 ** 31 - 200, 511, 0]
    table = None
    shape = (B, n_kv, cap)
    if page:
        per = cap // page
        table = torch.randperm(B * per, generator=gen).reshape(B, per).int().cuda()
        shape = (B * per, n_kv, page)
    caches = [torch.randint(0, 100, shape + tail, generator=gen).to(dtype).cuda() for _ in range(3)]
    want = [c.clone() for c in caches]
    for c, w in zip(caches, want):
        for b in range(B):
            for i in range(keeps[b]):
                a, z = pos[b] + paths[b][i], pos[b] + i
                if page:
                    w[int(table[b, z // page]), :, z % page] = c[int(table[b, a // page]), :, a % page]
                else:
                    w[b, :, z % cap] = c[b, :, a % cap]
    err = i32([0])
    g.gemma_kv_keep(caches, i32(pos), i32(paths), i32(keeps), kind=kind, block_table=table,
                    device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for c, w in zip(caches, want):
        assert torch.equal(c, w)


def test_keep_more_caches_than_one_launch_takes():
    caches = [torch.randn(1, 1, 16, 8, device="cuda").bfloat16() for _ in range(300)]
    want = [torch.cat([c[:, :, :5], c[:, :, 6:7], c[:, :, 6:]], 2) for c in caches]
    g.gemma_kv_keep(caches, i32([4]), i32([[0, 2, 3]]), i32([2]))
    torch.cuda.synchronize()
    assert all(torch.equal(c, w) for c, w in zip(caches, want))


def test_keep_bad_sequences():
    B = 8
    cache = torch.randn(B, 2, 32, 8, device="cuda").bfloat16()
    want = cache.clone()
    want[0, :, 4:6] = cache[0, :, 5:7]
    path = [[1, 2, 0, 0], [2, 2, 3, 0], [1, 4, 0, 0], [1, 0, 0, 0], [0, 2, 0, 0], [0, 2, 0, 0],
            [0, 2, 0, 0], [-1, 2, 0, 0]]
    keep = [2, 2, 2, 2, 5, -1, 2, 2]
    err = i32([0])
    g.gemma_kv_keep([cache], i32([4, 4, 4, 4, 4, 4, 30, 4]), i32(path), i32(keep), device_error=err)
    torch.cuda.synchronize()
    assert err.item() == g.GEMMA_DEVERR_TREE | g.GEMMA_DEVERR_WRITE_POS
    assert torch.equal(cache, want)
    # a page that is none: its rows stay, the others move
    pool = torch.randn(3, 2, 128, 8, device="cuda").bfloat16()
    want = pool.clone()
    want[1, :, 127] = pool[0, :, 1]
    err.zero_()
    g.gemma_kv_keep([pool], i32([127]), i32([[2, 0, 0, 0]]), i32([1]), block_table=i32([[1, 0]]),
                    device_error=err)
    g.gemma_kv_keep([pool], i32([126]), i32([[0, 2, 3, 0]]), i32([3]), block_table=i32([[1, 7]]),
                    device_error=err)
    torch.cuda.synchronize()
    assert err.item() == g.GEMMA_DEVERR_PAGE
    assert torch.equal(pool, want)
