"""Cases of the speculative step over a cache (attention of a tree of drafted tokens, acceptance and
the move of the accepted rows) and of the pages of a pool (fork, reserve, free, compact).

Each case is a dict of plain values. ``run`` computes the operator from elementary torch
operations while ``own`` is false, and through the package's entry points while it is true.

Tree: node i of a sequence lies in the cache at position base + i and stands at position
base + depth(i) of the text; it attends the positions before base (those inside its window on a
sliding layer), its ancestors and itself. Pages: a page is free while its reference count is 0, new
pages are the lowest free ones in the order of sequences and positions. Before holders of a shared
page write to it, each gets a copy of its own; if all its holders are about to, the first of them (in
the order of sequences) keeps the page.
"""
import math

import torch

own = False

SLIDING, GLOBAL, RING = 0, 1, 2
DEV = "cuda"


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _attn(name, kind, window, n_q, n_kv, d, k_eq_v, batch, lo, hi, nodes, ragged=False, softcap=0.0,
          page=0, dtype="bf16"):
    """lo..hi: range of the sequences' lengths (with the tree's rows); ragged: sequences bring
    between half of the bucket's nodes and all of them."""
    c = dict(op="attn", kind=kind, window=window, n_q=n_q, n_kv=n_kv, head_dim=d, k_eq_v=k_eq_v,
             batch=batch, lo=lo, hi=hi, nodes=nodes, ragged=ragged, softcap=softcap, page=page,
             dtype=dtype)
    if name:
        c["name"] = name
    return c


def _commit(name, batch, nodes, n_kv, d, caches, kind, cap, page=0):
    c = dict(op="commit", batch=batch, nodes=nodes, n_kv=n_kv, head_dim=d, caches=caches, kind=kind,
             cap=cap, page=page)
    if name:
        c["name"] = name
    return c


def _fork(name, batch, copies, page, n_kv, d, pools, hi, add):
    """batch sequences, each forked `copies` times, then `add` positions reserved for all."""
    c = dict(op="fork", batch=batch, copies=copies, page=page, n_kv=n_kv, head_dim=d, pools=pools,
             hi=hi, add=add)
    if name:
        c["name"] = name
    return c


def _compact(name, n_pages, batch, page, n_kv, d, pools, used):
    """used: share of the pool's pages that hold rows."""
    c = dict(op="compact", n_pages=n_pages, batch=batch, page=page, n_kv=n_kv, head_dim=d,
             pools=pools, used=used)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user, a small tree on the E4B-shaped sliding layer (latency)
        _attn("tree_e4b_sliding_b1", SLIDING, 512, 8, 2, 256, False, 1, 2048, 2048, 8),
        # one user, a usual tree on the 12B-shaped global layer at a long context, K read as V
        _attn("tree_12b_global_b1", GLOBAL, 0, 16, 1, 512, True, 1, 8192, 8192, 32),
        # a serving batch on the sliding layer, trees of different sizes, the cache a ring
        _attn("tree_12b_ring_b16", RING, 1024, 16, 8, 256, False, 16, 1100, 16385, 32, True),
        # the same batch on the global layer over pages: the largest step
        _attn("tree_12b_global_b16", GLOBAL, 0, 16, 1, 512, True, 16, 129, 16385, 32, False, 0.0,
              256),
        # an odd batch of large odd trees on the E4B-shaped global layer, soft-cap, small pages
        _attn("tree_e4b_paged_b7_cap", GLOBAL, 0, 8, 2, 256, False, 7, 700, 9001, 61, True, 50.0,
              128),
        # the fp32 path, as a user checks a model's numbers
        _attn("tree_fp32_b2", GLOBAL, 0, 4, 2, 128, False, 2, 300, 700, 17, False, 0.0, 0, "fp32"),
        # one user's step: the accepted path, and its rows in the caches of eight owner layers
        _commit("commit_e4b_b1", 1, 8, 2, 256, 16, GLOBAL, 2112),
        # a batch's step over twelve ring caches' K and V
        _commit("commit_12b_b16", 16, 32, 8, 256, 24, RING, 1152),
        # one prompt continued four ways (the earlier branches dropped first)
        _fork("fork_b1x4", 1, 4, 128, 2, 256, 8, 1000, 1),
        # a batch, every sequence continued two ways, a tree of 32 reserved for each
        _fork("fork_b32x2", 32, 2, 128, 8, 256, 8, 1500, 32),
        # a small pool put together again
        _compact("compact_64", 64, 4, 128, 2, 256, 8, 0.5),
        # a large pool after many requests have come and gone
        _compact("compact_512", 512, 48, 128, 8, 256, 8, 0.55),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    what = rng.choice(["attn", "attn", "attn", "attn", "commit", "fork", "compact"])
    if what == "commit":
        kind = rng.choice([SLIDING, GLOBAL, RING])
        nodes = _log_int(rng, 1, 128)
        batch = _log_int(rng, 1, 64)
        n_kv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256, 512])
        cap = 128 * rng.randint(2, 12)
        caches = max(1, min(rng.randint(1, 48), (1 << 29) // (batch * n_kv * cap * d)))
        return _commit(None, batch, nodes, n_kv, d, caches, kind, cap,
                       rng.choice([0, 128]) if kind != RING else 0)
    if what == "fork":
        batch, copies = _log_int(rng, 1, 32), rng.randint(1, 4)
        page, n_kv, d = rng.choice([128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([64, 256, 512])
        hi = _log_int(rng, 10, 2000)
        pages = batch * (1 + copies) * (hi // page + 3)
        pools = max(1, min(rng.randint(1, 16), (1 << 29) // (pages * page * n_kv * d)))
        return _fork(None, batch, copies, page, n_kv, d, pools, hi, _log_int(rng, 1, 300))
    if what == "compact":
        n_pages = _log_int(rng, 16, 2000)
        page, n_kv, d = rng.choice([128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([64, 256, 512])
        pools = max(1, min(rng.randint(1, 16), (1 << 29) // (n_pages * page * n_kv * d)))
        return _compact(None, n_pages, rng.randint(1, 64), page, n_kv, d, pools,
                        rng.uniform(0.1, 0.95))
    d = rng.choice([64, 128, 256, 256, 512])
    group = rng.choice([1, 2, 4, 8, 16])
    n_kv = rng.choice([1, 2, 4, 8]) if group <= 4 else rng.choice([1, 2])
    dtype = rng.choice(["bf16"] * 7 + ["fp32"])
    kind = rng.choice([SLIDING, GLOBAL, RING])
    window = 0 if kind == GLOBAL else rng.choice([100, 512, 1024])
    nodes = _log_int(rng, 1, 128)
    hi = _log_int(rng, max(nodes, 16), 16385 if dtype == "bf16" else 2000)
    lo = rng.randint(nodes, hi)
    reach = hi if kind == GLOBAL else min(hi, window + nodes)
    most = 6e10 if dtype == "bf16" else 5e8                  # multiply-adds
    batch = max(1, min(_log_int(rng, 1, 64), int(60e6 // (reach * n_kv * d)),
                       int(most // (2.0 * nodes * group * n_kv * reach * d))))
    page = rng.choice([0, 0, 128, 256]) if kind != RING else 0
    return _attn(None, kind, window, group * n_kv, n_kv, d, rng.random() < 0.4, batch, lo, hi, nodes,
                 rng.random() < 0.5, rng.choice([0.0, 0.0, 50.0]), page, dtype)


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _gen(seed, dev=None):
    return torch.Generator(device=dev or DEV).manual_seed(seed)


def _rows(g, shape, dtype):
    """Rows of unit-variance channels, a few of them larger, as projected keys and values are. One
    block of rows is drawn, and every block holds that block rolled by another amount."""
    d = shape[-1]
    gain = 1 + 2 * (torch.rand(d, generator=g, device=DEV) < 0.03).float()
    n = math.prod(shape[:-1])
    out = torch.empty(n, d, dtype=dtype, device=DEV)
    step = max(1, (1 << 25) // d)
    block = (torch.randn(min(n, step), d, generator=g, device=DEV) * gain).to(dtype)
    for i, a in enumerate(range(0, n, step)):
        out[a:a + step] = torch.roll(block, 37 * i, 0)[:min(n, a + step) - a]
    return out.reshape(shape)


def _tree(rng_cpu, n, nodes):
    """Parents of one sequence's n nodes (-1: the root; entries behind n are unused)."""
    u = torch.rand(nodes, generator=rng_cpu)
    p = (u.pow(0.7) * torch.arange(nodes)).long()
    p[0] = -1
    p[n:] = -1
    return p


def _counts(c, g):
    B, n = c["batch"], c["nodes"]
    lo = max(1, n // 2) if c.get("ragged", True) else n
    return torch.randint(lo, n + 1, (B,), generator=g)


def _table(g, batch, per, n_pages):
    return torch.randperm(n_pages, generator=g, device=DEV)[:batch * per].int().reshape(
        batch, per).contiguous()


def _prepare_attn(c, seed):
    g, h = _gen(seed), _gen(seed, "cpu")
    B, d, n_kv, nodes = c["batch"], c["head_dim"], c["n_kv"], c["nodes"]
    dtype = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device=DEV)
    lens[0] = c["hi"]
    real = _counts(c, h)
    st = dict(case=c, lens=lens.int(), real=real.int().to(DEV) if c["ragged"] else None)
    st["parents"] = torch.stack([_tree(h, int(n), nodes) for n in real]).int().to(DEV)
    st["q"] = torch.randn(B, nodes, c["n_q"], d, generator=g, device=DEV).to(dtype)
    st["table"] = None
    if c["page"]:
        per = -(-c["hi"] // c["page"])
        shape = (B * per + 3, n_kv, c["page"], d)
        st["table"] = _table(g, B, per, shape[0])
    elif c["kind"] == RING:
        shape = (B, n_kv, -(-(c["window"] + nodes - 1) // 128) * 128, d)
    else:
        shape = (B, n_kv, c["hi"], d)
    st["k"] = _rows(g, shape, dtype)
    st["v"] = None if c["k_eq_v"] else _rows(g, shape, dtype)
    st["out"] = torch.empty_like(st["q"])
    if own:
        import mixed_sliding_global_gb300 as m
        n = m.gemma_attn_workspace_size_tree(B, c["kind"], c["window"], c["n_q"], n_kv, d, c["hi"],
                                             nodes)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def _prepare_commit(c, seed):
    """Trees whose accepted path is the root and the last nodes, so that a pass may be repeated."""
    g, h = _gen(seed), _gen(seed, "cpu")
    B, nodes = c["batch"], c["nodes"]
    real = _counts(c, h)
    tokens = torch.randint(0, 262144, (B, nodes), generator=h)
    target = torch.randint(0, 262144, (B, nodes), generator=h)
    parents = []
    for b in range(B):
        n = int(real[b])
        k = int(torch.randint(1, max(1, n // 2) + 1, (1,), generator=h))
        p = _tree(h, n, nodes)
        path = [0] + list(range(n - k + 1, n))
        for a, i in zip(path, path[1:]):
            p[i] = a
            target[b, a] = tokens[b, i]
        target[b, path[-1]] = 262144                          # no draft has this token
        parents.append(p)
    st = dict(case=c, tokens=tokens.int().to(DEV), target=target.int().to(DEV),
              parents=torch.stack(parents).int().to(DEV), real=real.int().to(DEV))
    top = c["cap"] - nodes if c["kind"] != RING else 20000
    st["pos"] = torch.randint(0, top + 1, (B,), generator=g, device=DEV).int()
    st["lens"] = st["pos"] + st["real"]
    st["table"] = None
    shape = (B, c["n_kv"], c["cap"], c["head_dim"])
    if c["page"]:
        per = c["cap"] // c["page"]
        st["table"] = _table(g, B, per, B * per)
        shape = (B * per, c["n_kv"], c["page"], c["head_dim"])
    st["caches"] = [_rows(g, shape, torch.bfloat16) for _ in range(c["caches"])]
    i32 = dict(dtype=torch.int32, device=DEV)
    st["path"] = torch.empty(B, nodes, **i32)
    st["keep"], st["token"], st["new_lens"] = (torch.empty(B, **i32) for _ in range(3))
    st["err"] = torch.zeros(1, **i32)
    return st


def _prepare_fork(c, seed):
    g = _gen(seed)
    S, F, ps = c["batch"], c["copies"], c["page"]
    B = S * (1 + F)
    per = -(-(c["hi"] + c["add"]) // ps) + 1
    n_pages = B * per
    lens = torch.zeros(B, dtype=torch.int64, device=DEV)
    lens[:S] = torch.randint(max(1, c["hi"] // 2), c["hi"] + 1, (S,), generator=g, device=DEV)
    lens[0] = c["hi"]
    table = _table(g, B, per, n_pages)
    held = torch.arange(per, device=DEV) < ((lens + ps - 1) // ps)[:, None]
    table = torch.where(held, table, torch.full_like(table, -1))
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[table[held].long()] = 1
    st = dict(case=c, table=table, refs=refs, lens=lens.int())
    i32 = dict(dtype=torch.int32, device=DEV)
    st["src"] = torch.arange(S, **i32).repeat_interleave(F)
    st["dst"] = torch.arange(S, B, **i32)
    st["add"] = torch.full((B,), c["add"], **i32)
    # what the earlier branches keep: nothing; the other sequences: everything
    st["to"] = torch.full((B,), per * ps, **i32)
    st["to"][S:] = 0
    st["pools"] = [_rows(g, (n_pages, c["n_kv"], ps, c["head_dim"]), torch.bfloat16)
                   for _ in range(c["pools"])]
    st["err"] = torch.zeros(1, **i32)
    if own:
        import mixed_sliding_global_gb300 as m
        st["ws"] = torch.empty(m.gemma_pages_workspace_size(n_pages), dtype=torch.uint8, device=DEV)
    return st


def _prepare_compact(c, seed):
    g = _gen(seed)
    B, P = c["batch"], c["n_pages"]
    used = max(1, int(P * c["used"]))
    per = -(-used // B)
    pages = torch.randperm(P, generator=g, device=DEV)[:used].int()
    table = torch.full((B * per,), -1, dtype=torch.int32, device=DEV)
    table[torch.randperm(B * per, generator=g, device=DEV)[:used]] = pages
    table = table.reshape(B, per)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[pages.long()] = 1
    st = dict(case=c, table0=table, refs0=refs, table=table.clone(), refs=refs.clone())
    st["pools"] = [_rows(g, (P, c["n_kv"], c["page"], c["head_dim"]), torch.bfloat16)
                   for _ in range(c["pools"])]
    st["n_used"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        import mixed_sliding_global_gb300 as m
        st["ws"] = torch.empty(m.gemma_pages_workspace_size(P), dtype=torch.uint8, device=DEV)
    return st


def prepare(case, seed):
    return {"attn": _prepare_attn, "commit": _prepare_commit, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------
# one pass: the plain forms
# --------------------------------------------------------------------------------------------
def _gather(st, cache, pos):
    """Rows [B][n_kv][N][d] of positions pos [B][N]."""
    c = st["case"]
    if st["table"] is not None:
        page = torch.gather(st["table"].long(), 1,
                            (pos // c["page"]).clamp_max(st["table"].shape[1] - 1))
        x = cache[page, :, pos % c["page"]]
    else:
        b = torch.arange(pos.shape[0], device=DEV)[:, None]
        slot = pos % cache.shape[2] if c["kind"] == RING else pos.clamp_max(cache.shape[2] - 1)
        x = cache[b, :, slot]
    return x.transpose(1, 2)                                  # from [B][N][n_kv][d]


def _ancestors(parents):
    """[B][n][n] truth values: m is i or an ancestor of i."""
    B, n = parents.shape
    up = torch.eye(n, device=DEV).expand(B, n, n).clone()
    edge = (torch.arange(n, device=DEV) == parents.long()[:, :, None]).float()
    step = 1
    while step < n:       # closed over paths of up to 2 * step edges each time round
        up = ((up + edge @ up) > 0).float()
        edge = edge @ edge
        step *= 2
    return up > 0


def _plain_attn(st):
    c = st["case"]
    B, nodes, n_q, d = st["q"].shape
    n_kv, G = c["n_kv"], c["n_q"] // c["n_kv"]
    lens = st["lens"].long()
    real = st["real"].long() if c["ragged"] else torch.full_like(lens, nodes)
    base = lens - real
    see = _ancestors(st["parents"])                                           # [B][n][n]
    depth = see.sum(-1) - 1                                                   # [B][n]
    if c["kind"] == GLOBAL:
        first, N = torch.zeros_like(base), c["hi"]
    else:
        first, N = (base - c["window"] + 1).clamp_min(0), min(c["hi"], c["window"] + nodes)
    pos = first[:, None] + torch.arange(N, device=DEV)                        # [B][N]
    k = _gather(st, st["k"], pos).float()
    v = k if c["k_eq_v"] else _gather(st, st["v"], pos).float()
    q = st["q"].float().reshape(B, nodes, n_kv, G, d).permute(0, 2, 3, 1, 4).reshape(
        B, n_kv, G * nodes, d)
    s = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    node = pos - base[:, None]                                                # [B][N]
    at = node.clamp(0, nodes - 1)
    in_tree = ((node >= 0) & (node < real[:, None]))[:, None, :] & torch.gather(
        see, 2, at[:, None, :].expand(B, nodes, N))
    back = torch.where(node < 0, node, torch.gather(depth, 1, at))            # text position - base
    ok = (node < 0)[:, None, :] | in_tree
    if c["kind"] != GLOBAL:
        ok = ok & (depth[:, :, None] - back[:, None, :] < c["window"])
    live = torch.arange(nodes, device=DEV) < real[:, None]                    # [B][n]
    ok = ok | ~live[:, :, None]          # rows behind the tree: anything finite, zeroed below
    s = s.reshape(B, n_kv, G, nodes, N).masked_fill(~ok[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(B, n_kv, G * nodes, N)
    o = (p @ v).reshape(B, n_kv, G, nodes, d).permute(0, 3, 1, 2, 4).reshape(B, nodes, n_q, d)
    return torch.where(live[:, :, None, None], o, torch.zeros_like(o)).to(st["q"].dtype)


def _plain_commit(st):
    c = st["case"]
    B, n = st["tokens"].shape
    tokens, target, parents = st["tokens"], st["target"], st["parents"]
    node = torch.arange(n, device=DEV)
    real = st["real"].long()
    live = node < real[:, None]
    cur = torch.zeros(B, dtype=torch.int64, device=DEV)
    keep = torch.ones(B, dtype=torch.int64, device=DEV)
    path = torch.full((B, n), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    going = torch.ones(B, dtype=torch.bool, device=DEV)
    for _ in range(1, n):
        want = torch.gather(target, 1, cur[:, None])
        hit = (parents == cur[:, None]) & (tokens == want) & live
        going = going & hit.any(1)
        child = torch.where(hit, node, torch.full_like(node, n)).amin(1)
        cur = torch.where(going, child, cur)
        at = keep.clamp_max(n - 1)[:, None]
        path.scatter_(1, at, torch.where(going[:, None], cur[:, None], torch.gather(path, 1, at)))
        keep = keep + going.long()
    token = torch.gather(target, 1, cur[:, None])[:, 0]
    base = st["pos"].long()
    to = base[:, None] + node
    frm = base[:, None] + torch.where(node < keep[:, None], path, node)

    def place(pos):
        if st["table"] is not None:
            page = torch.gather(st["table"].long(), 1, pos // c["page"])
            return page, pos % c["page"]
        b = torch.arange(B, device=DEV)[:, None].expand(B, n)
        return b, pos % c["cap"] if c["kind"] == RING else pos

    (r0, s0), (r1, s1) = place(frm), place(to)
    for x in st["caches"]:
        x[r1, :, s1] = x[r0, :, s0]
    return [path.int(), keep.int(), token, (base + keep).int()] + [x.view(torch.int16)
                                                                   for x in st["caches"]]


def _plain_fork(st):
    c = st["case"]
    table, refs, lens, ps = st["table"], st["refs"], st["lens"], c["page"]
    B, per = table.shape
    blk = torch.arange(per, device=DEV)
    # the earlier branches' pages go back
    gone = (table >= 0) & (blk * ps >= st["to"][:, None])
    refs.index_add_(0, table.clamp_min(0).reshape(-1).long(), -gone.reshape(-1).int())
    table.masked_fill_(gone, -1)
    # new branches share their source's pages
    src, dst = st["src"].long(), st["dst"].long()
    held = blk < ((lens[src] + ps - 1) // ps)[:, None]
    row = torch.where(held, table[src], torch.full_like(table[src], -1))
    table[dst] = row
    lens[dst] = lens[src]
    refs.index_add_(0, row.clamp_min(0).reshape(-1).long(), (row >= 0).reshape(-1).int())
    # private pages for the positions len .. len + add - 1 of every sequence
    K = (c["add"] + ps - 2) // ps + 1
    first = (lens // ps).long()
    b = first[:, None] + torch.arange(K, device=DEV)
    wanted = b * ps < (lens + st["add"])[:, None]
    at = b.clamp_max(per - 1)
    have = torch.gather(table, 1, at).long()
    page, need = have.reshape(-1), wanted.reshape(-1)
    held = need & (page >= 0)
    same = (page[:, None] == page[None, :]) & held[None, :] & held[:, None]
    others = refs[page.clamp_min(0)] - same.sum(1)             # holders that do not write now
    cow = held & ((torch.tril(same, -1).sum(1) > 0) | (others > 0))
    new = (need & (page < 0)) | cow
    free = torch.sort((refs != 0).int(), stable=True).indices  # the free pages first, in order
    given = torch.where(new, free[(torch.cumsum(new, 0) - 1).clamp_min(0)], page)
    refs.index_add_(0, page.clamp_min(0), -cow.int())
    refs.index_add_(0, given.clamp_min(0), new.int())
    old = torch.gather(table, 1, at)
    table.scatter_(1, at, torch.where(wanted, given.reshape(B, K).int(), old))
    # rows below the length go along (only a sequence's first page can have any)
    is_cow = cow.reshape(B, K)[:, 0]
    frm = have[:, 0].clamp_min(0)
    to = torch.where(is_cow, given.reshape(B, K)[:, 0], frm)
    row = torch.arange(ps, device=DEV) < (lens.long() - first * ps)[:, None]
    pick = torch.nonzero(is_cow)[:, 0]
    for x in st["pools"]:
        x[to[pick]] = torch.where(row[pick, None, :, None], x[frm[pick]], x[to[pick]])
    return [table, refs, lens] + [x.view(torch.int16) for x in st["pools"]]


def _plain_compact(st):
    table, refs = st["table"], st["refs"]
    table.copy_(st["table0"])          # the pool as the requests left it
    refs.copy_(st["refs0"])
    P = refs.shape[0]
    i = torch.arange(P, device=DEV)
    used = refs > 0
    n = used.sum()
    hole, high = torch.nonzero(~used & (i < n))[:, 0], torch.nonzero(used & (i >= n))[:, 0]
    where = i.clone()
    where[high] = hole
    table.copy_(torch.where(table >= 0, where[table.clamp_min(0).long()].int(), table))
    refs[hole] = refs[high]
    refs[high] = 0
    for x in st["pools"]:
        x[hole] = x[high]
    st["n_used"].copy_(n)
    return [table, refs, st["n_used"]] + [x.view(torch.int16) for x in st["pools"]]


# --------------------------------------------------------------------------------------------
# one pass: the package's calls
# --------------------------------------------------------------------------------------------
def _own_attn(st):
    import mixed_sliding_global_gb300 as m
    c = st["case"]
    m.gemma_attn_tree(st["out"], st["q"], [st["k"]], [st["v"]], [0], 0, st["lens"], st["parents"],
                      c["hi"], kind=c["kind"], window=c["window"], n_kv=c["n_kv"],
                      k_eq_v=c["k_eq_v"], scale=1 / math.sqrt(c["head_dim"]), softcap=c["softcap"],
                      n_real=st["real"], block_table=st["table"], workspace=st["ws"],
                      device_error=st["err"])
    return st["out"]


def _own_commit(st):
    import mixed_sliding_global_gb300 as m
    c = st["case"]
    m.gemma_tree_accept(st["tokens"], st["parents"], st["target"], st["path"], st["keep"],
                        st["token"], n_real=st["real"], seq_lens=st["lens"],
                        lens_out=st["new_lens"], device_error=st["err"])
    m.gemma_kv_keep(st["caches"], st["pos"], st["path"], st["keep"], kind=c["kind"],
                    block_table=st["table"], device_error=st["err"])
    return [st["path"], st["keep"], st["token"], st["new_lens"]] + [x.view(torch.int16)
                                                                    for x in st["caches"]]


def _own_fork(st):
    import mixed_sliding_global_gb300 as m
    c = st["case"]
    m.gemma_pages_free(st["table"], st["refs"], page_size=c["page"], keep_to=st["to"],
                       device_error=st["err"])
    m.gemma_pages_fork(st["table"], st["refs"], st["lens"], st["src"], st["dst"],
                       page_size=c["page"], device_error=st["err"])
    m.gemma_pages_reserve(st["pools"], st["table"], st["refs"], st["lens"], st["add"],
                          workspace=st["ws"], device_error=st["err"])
    return [st["table"], st["refs"], st["lens"]] + [x.view(torch.int16) for x in st["pools"]]


def _own_compact(st):
    import mixed_sliding_global_gb300 as m
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    m.gemma_pages_compact(st["pools"], st["table"], st["refs"], n_used=st["n_used"],
                          workspace=st["ws"], device_error=st["err"])
    return [st["table"], st["refs"], st["n_used"]] + [x.view(torch.int16) for x in st["pools"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _own_attn, "commit": _own_commit, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"attn": _plain_attn, "commit": _plain_commit, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


# --------------------------------------------------------------------------------------------
# work and 64-bit results
# --------------------------------------------------------------------------------------------
def work(case):
    c = case
    row = 2.0 * c["n_kv"] * c["head_dim"]
    if c["op"] == "commit":
        # a quarter of a tree's nodes is kept on average, the root in its place; trees of a bucket
        # have three quarters of its nodes
        moved = max(0.0, 0.75 * c["nodes"] / 4 - 0.5) * c["batch"]
        return {"bytes": 2 * moved * row * c["caches"] + 16 * c["batch"] * c["nodes"],
                "flops": c["batch"] * c["nodes"]}
    if c["op"] == "fork":
        # all holders of a sequence's last page but one copy half a page of rows on average
        rows = c["batch"] * c["copies"] * c["page"] / 2
        per = -(-(c["hi"] + c["add"]) // c["page"]) + 1
        table = 4 * c["batch"] * (1 + c["copies"]) * per
        return {"bytes": 2 * rows * row * c["pools"] + 4 * table, "flops": table}
    if c["op"] == "compact":
        n = max(1, int(c["n_pages"] * c["used"]))
        moved = n * (1 - n / c["n_pages"])                    # used pages behind the first n
        return {"bytes": 2 * moved * c["page"] * row * c["pools"] + 16 * c["n_pages"],
                "flops": c["n_pages"]}
    d, lo, hi = c["head_dim"], c["lo"], c["hi"]
    nodes = c["nodes"] * (0.75 if c["ragged"] else 1.0)
    lens = [hi] + [lo + (hi - lo) * (i + 0.5) / 64 for i in range(64)] * (c["batch"] > 1)
    wts = [1.0] + [(c["batch"] - 1) / 64.0] * 64
    keys = pairs = 0.0
    for n, wt in zip(lens, wts):
        base = max(0.0, n - nodes)
        seen = base if c["kind"] == GLOBAL else min(base, c["window"] - 1)
        keys += wt * (seen + nodes)
        # a node attends its prefix and a few ancestors
        pairs += wt * nodes * (seen + math.log2(nodes + 1) + 1)
    size = 4 if c["dtype"] == "fp32" else 2
    return {"bytes": size * (keys * c["n_kv"] * d * (1 if c["k_eq_v"] else 2)
                             + 2.0 * c["batch"] * c["nodes"] * c["n_q"] * d),
            "flops": 4.0 * pairs * c["n_q"] * d}


def exact(case, seed):
    c = case
    if c["op"] != "attn":          # whole numbers and copies
        return None
    st = prepare(case, seed)
    B, nodes, n_q, d = st["q"].shape
    G = n_q // c["n_kv"]
    out = torch.zeros(B, nodes, n_q, d, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(st["real"][b]) if c["ragged"] else nodes
        end = int(st["lens"][b])
        base = end - n
        up = st["parents"][b].tolist()
        line = []                                             # a node's ancestors and itself
        for i in range(n):
            line.append((line[up[i]] if up[i] >= 0 else []) + [i])
        first = 0 if c["kind"] == GLOBAL else max(0, base - c["window"] + 1)
        see = torch.zeros(n, end - first, dtype=torch.bool)
        for i in range(n):
            at = base + len(line[i]) - 1
            start = first if c["kind"] == GLOBAL else max(first, at - c["window"] + 1)
            see[i, start - first:max(0, base - first)] = True
            for dep, m in enumerate(line[i]):
                if c["kind"] == GLOBAL or len(line[i]) - 1 - dep < c["window"]:
                    see[i, base + m - first] = True
        see = see.to(DEV)
        j = torch.arange(first, end, device=DEV)
        if st["table"] is not None:
            row, slot = st["table"][b].long()[j // c["page"]], j % c["page"]
        else:
            row, slot = torch.full_like(j, b), j % st["k"].shape[2]
        for h in range(c["n_kv"]):
            k = st["k"][row, h, slot].double()
            v = k if c["k_eq_v"] else st["v"][row, h, slot].double()
            s = st["q"][b, :n, h * G:h * G + G].double().transpose(0, 1) @ k.T / math.sqrt(d)
            if c["softcap"]:
                s = torch.tanh(s / c["softcap"]) * c["softcap"]
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            out[b, :n, h * G:h * G + G] = (torch.softmax(s, -1) @ v).transpose(0, 1)
    return out
