"""Drafted decoding as a server runs it: trees of drafts over a paged pool and a ring cache together,
pages reserved, shared, given back and moved, tokens accepted and kept rows moved, step after step and
captured in a graph. The caches are then, bit for bit, what the accepted tokens' rows would have
filled one after another, and the last outputs attention over them."""
import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref

pytestmark = pytest.mark.gpu

VOCAB, NODES, D, N_Q, N_KV, PAGE, WINDOW = 8, 12, 64, 4, 2, 128, 50


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Two layers: a global one over a pool, a sliding one over rings (K is V there). A token's rows are
    table entries, so that what a cache has to hold follows from the tokens alone."""

    def __init__(self, batch, per=6, seed=0):
        gen = torch.Generator().manual_seed(seed)
        table = lambda *s: torch.randn(VOCAB, *s, generator=gen).bfloat16().cuda()  # noqa: E731
        self.B, self.per, self.P = batch, per, batch * per
        self.q = [table(N_Q, D) for _ in range(2)]
        self.k = [table(N_KV, D) for _ in range(2)]
        self.v = table(N_KV, D)
        self.head = torch.randn(2 * N_Q * D, VOCAB, generator=gen).cuda()
        shape = (self.P, N_KV, PAGE, D)
        self.pool = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.ring = torch.zeros(batch, N_KV, 128, D, dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((batch, per), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(self.P, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")  # rows in the caches
        self.err = i32([0])
        self.pages_ws = torch.empty(g.gemma_pages_workspace_size(self.P), dtype=torch.uint8, device="cuda")
        need = max(g.gemma_attn_workspace_size_tree(batch, k, w, N_Q, N_KV, D, per * PAGE, NODES)
                   for k, w in ((g.GEMMA_GLOBAL, 0), (g.GEMMA_SLIDING_RING, WINDOW)))
        self.ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
        # a step's buffers
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tokens, self.parents, self.path = z(batch, NODES), z(batch, NODES), z(batch, NODES)
        self.real, self.keep, self.next_token, self.pos = z(batch), z(batch), z(batch), z(batch)
        self.drawn, self.all_lens = z(batch, NODES), z(batch)
        self.out = [torch.zeros(batch, NODES, N_Q, D, dtype=torch.bfloat16, device="cuda")
                    for _ in range(2)]

    def step(self):
        """One step of every sequence, from tokens, parents and real: no host work in between."""
        e = dict(device_error=self.err)
        g.gemma_pages_reserve(self.pool, self.table, self.refs, self.lens, self.real,
                              workspace=self.pages_ws, **e)
        self.pos.copy_(self.lens)
        self.all_lens.copy_(self.lens + self.real)
        t = self.tokens.long()
        rows = [k[t] for k in self.k] + [self.v[t]]
        # rows behind a sequence's own nodes are not part of the pool's pages: written one by one
        for n in range(NODES):
            one = (self.real > n).int()
            at = torch.where(one > 0, self.pos + n, torch.full_like(self.pos, -1))
            self._append(rows, n, at)
        q = [x[t] for x in self.q]
        kw = dict(n_kv=N_KV, scale=D ** -0.5, n_real=self.real, workspace=self.ws, **e)
        g.gemma_attn_tree(self.out[0], q[0], [self.pool[0]], [self.pool[1]], [0], 0, self.all_lens,
                          self.parents, self.per * PAGE, kind=g.GEMMA_GLOBAL, window=0, k_eq_v=False,
                          block_table=self.table, **kw)
        g.gemma_attn_tree(self.out[1], q[1], [self.ring], None, [0], 0, self.all_lens, self.parents,
                          self.per * PAGE, kind=g.GEMMA_SLIDING_RING, window=WINDOW, k_eq_v=True, **kw)
        x = torch.cat([o.float().reshape(self.B * NODES, -1) for o in self.out], 1)
        logits = (x @ self.head).contiguous()
        lw = torch.zeros(max(16, g.gemma_logit_workspace_size(self.B * NODES, VOCAB)), dtype=torch.uint8,
                         device="cuda")
        g.gemma_logit_softcap_argmax(logits, 0.0, self.drawn.view(-1), workspace=lw)
        g.gemma_tree_accept(self.tokens, self.parents, self.drawn, self.path, self.keep,
                            self.next_token, n_real=self.real, seq_lens=self.all_lens,
                            lens_out=self.lens, **e)
        g.gemma_kv_keep(self.pool, self.pos, self.path, self.keep, block_table=self.table, **e)
        g.gemma_kv_keep([self.ring], self.pos, self.path, self.keep, kind=g.GEMMA_SLIDING_RING, **e)
        g.gemma_pages_free(self.table, self.refs, page_size=PAGE, keep_to=self.lens, **e)

    def _append(self, rows, n, at):
        """Node n of the sequences that have it (a negative position writes nothing)."""
        err = torch.zeros(1, dtype=torch.int32, device="cuda")   # (the skipped ones are reported)
        g.gemma_kv_append_paged([self.pool[0]], [self.pool[1]], [0], 0, rows[0][:, n:n + 1].contiguous(),
                                rows[2][:, n:n + 1].contiguous(), at, self.table, k_eq_v=False,
                                device_error=err)
        g.gemma_kv_append_ring([self.ring], None, [0], 0, rows[1][:, n:n + 1].contiguous(), None, at,
                               k_eq_v=True, device_error=err)

    def check(self, text, last_path=None):
        """Caches against the sequences' tokens, and the kept nodes' outputs against attention."""
        torch.cuda.synchronize()
        assert self.err.item() == 0
        for b, tokens in enumerate(text):
            n = len(tokens)
            assert self.lens[b].item() == n
            if n == 0:
                continue
            t = torch.tensor(tokens, device="cuda")
            at = torch.arange(n, device="cuda")
            page = self.table[b].long()[at // PAGE]
            assert (page >= 0).all()
            assert torch.equal(self.pool[0][page, :, at % PAGE], self.k[0][t])
            assert torch.equal(self.pool[1][page, :, at % PAGE], self.v[t])
            recent = at[max(0, n - WINDOW):]
            assert torch.equal(self.ring[b][:, recent % 128].transpose(0, 1), self.k[1][t[recent]])
            if last_path and last_path[b]:
                path = last_path[b]
                first = n - len(path)
                for layer, (kind, window) in enumerate(((tree_ref.GLOBAL, 0), (tree_ref.SLIDING, WINDOW))):
                    see = tree_ref.keys_of([i - 1 for i in range(len(path))], len(path), first, kind,
                                           window)
                    k = self.k[layer][t]
                    ref, mass, _ = tree_ref.attention(self.q[layer][t[first:]], k,
                                                      self.v[t] if layer == 0 else k, see, D ** -0.5)
                    got = self.out[layer][b, path].double()
                    # the output's rounding and P's, and 2^-14 for fp32 scores of 64 products
                    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -14) * (mass + ref.abs())
                    assert ((got - ref).abs() <= bound).all()


def prompt(server, text):
    """The sequences' first tokens into the caches."""
    add = i32([len(t) for t in text])
    g.gemma_pages_reserve(server.pool, server.table, server.refs, server.lens, add,
                          workspace=server.pages_ws, device_error=server.err)
    top = max(len(t) for t in text)
    t = torch.tensor([x + [0] * (top - len(x)) for x in text], device="cuda")
    rows = [k[t] for k in server.k] + [server.v[t]]
    for n in range(top):
        server._append(rows, n, torch.where(add > n, torch.full_like(add, n), torch.full_like(add, -1)))
    server.lens.copy_(add)


def drafts(server, text, pending, gen, real):
    """A tree per sequence: the pending token, a guess that continues it, and random branches."""
    tokens, parents = [], []
    for b in range(server.B):
        tk, pa = [pending[b]], [-1]
        for i in range(1, NODES):
            pa.append(int(torch.randint(0, i, (1,), generator=gen)))
            tk.append(int(torch.randint(0, VOCAB, (1,), generator=gen)))
        tokens.append(tk)
        parents.append(pa)
    server.tokens.copy_(i32(tokens))
    server.parents.copy_(i32(parents))
    server.real.copy_(i32(real))
    return tokens


def take(server, text, pending, tokens):
    """The step's result, on the host."""
    torch.cuda.synchronize()
    paths = []
    for b in range(server.B):
        n = server.keep[b].item()
        path = server.path[b].tolist()[:n]
        paths.append(path)
        text[b] += [tokens[b][i] for i in path]
        if n:
            pending[b] = server.next_token[b].item()
    return paths


@pytest.mark.parametrize("captured", [False, True])
def test_steps_forks_and_compaction(captured):
    B = 5
    s = Server(B)
    gen = torch.Generator().manual_seed(4)
    text = [torch.randint(0, VOCAB, (n,), generator=gen).tolist() for n in (100, 256, 127, 0, 0)]
    pending = [1, 2, 3, 4, 5]
    prompt(s, text)
    s.check(text)
    live = [True, True, True, False, False]
    graph = None
    kept = 0
    for step in range(30):
        real = [(1 + int(torch.randint(0, NODES, (1,), generator=gen))) if x else 0 for x in live]
        tokens = drafts(s, text, pending, gen, real)
        if captured and step == 0:
            side = torch.cuda.Stream()
            state = [x.clone() for x in (s.table, s.refs, s.lens, *s.pool, s.ring)]
            with torch.cuda.stream(side):
                side.wait_stream(torch.cuda.default_stream())
                s.step()                                  # a warm-up, taken back
            torch.cuda.synchronize()
            for x, y in zip((s.table, s.refs, s.lens, *s.pool, s.ring), state):
                x.copy_(y)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.step()
        if graph is not None:
            graph.replay()
        else:
            s.step()
        paths = take(s, text, pending, tokens)
        kept += sum(len(p) for p in paths)
        s.check(text, paths)
        if step == 12:      # sequence 0 goes on three ways, its last page shared
            assert len(text[0]) % PAGE
            g.gemma_pages_fork(s.table, s.refs, s.lens, i32([0, 0]), i32([3, 4]), page_size=PAGE,
                               device_error=s.err)
            s.ring[3], s.ring[4] = s.ring[0], s.ring[0]
            for b in (3, 4):
                text[b], live[b] = list(text[0]), True
                pending[b] = (pending[0] + b) % VOCAB
            s.check(text)
        if step == 22:      # sequence 1 ends, and the pool is put together
            live[1] = False
            g.gemma_pages_free(s.table, s.refs, page_size=PAGE,
                               keep_to=torch.where(i32([0, 1, 0, 0, 0]) > 0, i32([0] * 5), s.lens),
                               device_error=s.err)
            text[1] = []
            s.lens[1] = 0
            n_used = i32([0])
            g.gemma_pages_compact(s.pool, s.table, s.refs, n_used=n_used, workspace=s.pages_ws,
                                  device_error=s.err)
            torch.cuda.synchronize()
            used = int((s.refs > 0).sum())
            assert n_used.item() == used and (s.refs[:used] > 0).all()
            s.check(text)
    assert (s.table[2] >= 0).sum() > 1
    assert kept >= 30 * 3 * 1.25      # some drafts were accepted
    assert int(s.refs.sum()) == int((s.table >= 0).sum())
