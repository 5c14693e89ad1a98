"""The documented step over drafted tokens with a pool that runs out of pages: the sequences that get no
page of their own sit the step out, no row of another sequence is written over, and the same step goes on
once there are pages."""
import os
import re

import pytest
import torch

import mixed_sliding_global_gb300 as g

pytestmark = pytest.mark.gpu

PAGE, N_KV, N_Q, D, NODES, PER = 128, 2, 4, 64, 6, 3


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def documented_step():
    """The code block for users that reserves pages, compiled as it stands."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    step = [b for b in blocks if "gemma_pages_reserve" in b]
    assert len(step) == 1
    return compile(step[0], "README.md", "exec")


class Branches:
    """Sequence 0 of 130 positions, shared by its branches 1 and 2, and sequence 3 of 100; `n_pages` in all."""

    def __init__(self, n_pages):
        gen = torch.Generator().manual_seed(n_pages)
        self.table = torch.full((4, PER), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.lens, self.err = i32([0] * 4), i32([0])
        self.pool = [torch.zeros(n_pages, N_KV, PAGE, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.pages_ws = torch.empty(g.gemma_pages_workspace_size(n_pages), dtype=torch.uint8, device="cuda")
        self.rows = [torch.randn(4, 130, N_KV, D, generator=gen).bfloat16().cuda() for _ in range(2)]
        self.grow([130, 0, 0, 100])
        self.fork()
        self.held = [130, 130, 130, 100]
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        ws = g.gemma_attn_workspace_size_tree(4, g.GEMMA_GLOBAL, 0, N_Q, N_KV, D, PER * PAGE, NODES)
        q = torch.randn(4, NODES, N_Q, D, generator=gen).bfloat16().cuda()
        tokens = i32([[1, 2, 3, 4, 5, 6]] * 4)
        # every node's token is drawn behind the one before it: the whole chain holds
        self.names = dict(
            torch=torch, g=g, tokens=tokens, parents=i32([[-1, 0, 1, 2, 3, 4]] * 4),
            drawn=i32([[2, 3, 4, 5, 6, 7]] * 4), pool=self.pool, table=self.table, refs=self.refs,
            lens=self.lens, n_kv=N_KV, d=D, max_len=PER * PAGE, q=q, out=torch.empty_like(q),
            k_rows=torch.randn(4, NODES, N_KV, D, generator=gen).bfloat16().cuda(),
            v_rows=torch.randn(4, NODES, N_KV, D, generator=gen).bfloat16().cuda(),
            ws=torch.empty(max(16, ws), dtype=torch.uint8, device="cuda"),
            path=z(4, NODES), n_keep=z(4), next_token=z(4), err=self.err)

    def grow(self, add):
        g.gemma_pages_reserve(self.pool, self.table, self.refs, self.lens, i32(add), workspace=self.pages_ws,
                              device_error=self.err)
        for b, n in enumerate(add):
            if n:
                j = torch.arange(n, device="cuda")
                page = self.table[b].long()[j // PAGE]
                for x, rows in zip(self.pool, self.rows):
                    x[page, :, j % PAGE] = rows[b, :n]
        self.lens.copy_(i32(add))

    def fork(self):
        g.gemma_pages_fork(self.table, self.refs, self.lens, i32([0, 0]), i32([1, 2]), page_size=PAGE,
                           device_error=self.err)
        torch.cuda.synchronize()
        assert self.err.item() == 0

    def check(self, steps):
        """What each sequence holds: its first rows (a branch: its source's), then `steps[b]` times the
        drafted ones."""
        torch.cuda.synchronize()
        assert self.lens.tolist() == [n + NODES * s for n, s in zip(self.held, steps)]
        for b, s in enumerate(steps):
            for x, rows, new in zip(self.pool, self.rows, (self.names["k_rows"], self.names["v_rows"])):
                want = torch.cat([rows[0 if b < 3 else 3][:self.held[b]]] + [new[b]] * s)
                j = torch.arange(len(want), device="cuda")
                page = self.table[b].long()[j // PAGE]
                assert (page >= 0).all()
                assert torch.equal(x[page, :, j % PAGE], want)


@pytest.mark.parametrize("captured", [False, True])
def test_a_full_pool_in_the_documented_step(captured):
    """Four pages: two shared ones, one of sequence 3's, one free. The first branch that writes keeps the
    page only when all others have one of their own; with one free page of the two that are wanted, one
    branch gets it and two wait."""
    code = documented_step()
    s = Branches(4)
    names = dict(s.names)
    if captured:
        state = [x.clone() for x in (s.table, s.refs, s.lens, *s.pool)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            exec(code, names)                        # a warm-up, taken back
        torch.cuda.synchronize()
        for x, y in zip((s.table, s.refs, s.lens, *s.pool), state):
            x.copy_(y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            exec(code, names)
        go = graph.replay
    else:
        def go():
            exec(code, names)
    go()
    torch.cuda.synchronize()
    # branch 1 got the free page; 0 and 2 still share theirs, and neither may write
    assert s.refs.tolist() == [3, 2, 1, 1]
    s.check([0, 1, 0, 1])
    keep = names["n_keep"].tolist()
    assert keep == [0, NODES, 0, NODES]
    # branch 2 ends: 0 has the page for itself
    g.gemma_pages_free(s.table, s.refs, page_size=PAGE, keep_to=torch.where(i32([0, 0, 1, 0]) > 0, 0, s.lens).int())
    s.lens[2] = 0
    s.held[2] = 0
    # (an empty sequence has no page either, and none is free)
    go()
    s.check([1, 2, 0, 2])
    assert names["n_keep"].tolist() == [NODES, NODES, 0, NODES]
