"""Pages of a pool on the GPU: fork, reserve, free and compact against a model that takes one
sequence and one position at a time (tests/tree_ref.py)."""
import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """A pool on the device beside its model."""

    def __init__(self, batch, per, n_pages, page=128, seed=0, kinds=((2, (64,), torch.bfloat16),)):
        self.gen = torch.Generator().manual_seed(seed)
        self.B, self.per, self.P, self.ps = batch, per, n_pages, page
        host = [torch.randint(0, 100, (n_pages, n_kv, page) + tail, generator=self.gen).to(dt)
                for n_kv, tail, dt in kinds]
        self.pools = [x.cuda() for x in host]
        self.table = torch.full((batch, per), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.err = i32([0])
        self.ws = torch.full((g.gemma_pages_workspace_size(n_pages),), 255, dtype=torch.uint8,
                             device="cuda")
        self.model = tree_ref.Pages(self.table.tolist(), self.refs.tolist(), self.lens.tolist(), host,
                                    page)

    def reserve(self, add, full=False):
        g.gemma_pages_reserve(self.pools, self.table, self.refs, self.lens, i32(add),
                              workspace=self.ws, device_error=self.err)
        assert self.model.reserve(add) == full
        self.check(g.GEMMA_DEVERR_POOL_FULL if full else 0)

    def grow(self, add):
        """Reserve, and the rows written."""
        self.reserve(add)
        self.lens += i32(add)
        self.model.lens = [n + a for n, a in zip(self.model.lens, add)]

    def fork(self, src, dst, bits=0):
        g.gemma_pages_fork(self.table, self.refs, self.lens, i32(src), i32(dst), page_size=self.ps,
                           device_error=self.err)
        refused = self.model.fork(src, dst)
        self.check(bits)
        return refused

    def free(self, lo=None, hi=None, bits=0):
        g.gemma_pages_free(self.table, self.refs, page_size=self.ps,
                           keep_from=None if lo is None else i32(lo),
                           keep_to=None if hi is None else i32(hi), device_error=self.err)
        self.model.free(lo or [0] * self.B, hi or [1 << 40] * self.B)
        self.check(bits)

    def compact(self):
        used = i32([-5])
        g.gemma_pages_compact(self.pools, self.table, self.refs, n_used=used, workspace=self.ws,
                              device_error=self.err)
        assert used.item() == self.model.compact()
        self.check()

    def check(self, bits=0):
        torch.cuda.synchronize()
        assert self.err.item() == bits
        self.err.zero_()
        m = self.model
        assert self.table.tolist() == m.table
        assert self.refs.tolist() == m.refs
        assert self.lens.tolist() == m.lens
        for x, y in zip(self.pools, m.pools):
            assert torch.equal(x.cpu(), y)


KINDS = ((2, (64,), torch.bfloat16), (1, (128,), torch.float32), (3, (32,), torch.uint8),
         (3, (1,), torch.bfloat16), (3, (5,), torch.bfloat16))


@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("seed", range(4))
def test_random_use(seed, page):
    """Random growth, forks, releases and compaction over pools of every row width."""
    r = torch.Generator().manual_seed(seed)

    def rnd(n):
        return int(torch.randint(0, n, (1,), generator=r))

    B, per = 7, 6
    p = Pool(B, per, 40, page, seed, KINDS)
    p.grow([rnd(3 * page) for _ in range(3)] + [0] * 4)
    for step in range(14):
        what = rnd(5)
        if what == 0:
            add = [rnd(page) if 0 < n < 4 * page and rnd(2) else 0 for n in p.model.lens]
            p.grow(add)
        elif what == 1:
            live = [b for b in range(B) if p.model.lens[b] > 0]
            empty = [b for b in range(B) if all(e < 0 for e in p.model.table[b])]
            n = min(len(empty), 1 + rnd(3))
            if live and n:
                p.fork([live[rnd(len(live))] for _ in range(n)], empty[:n])
        elif what == 2:
            lo = [n // 2 if rnd(3) == 0 else 0 for n in p.model.lens]
            p.free(lo, None)
        elif what == 3:
            gone = [rnd(4) == 0 for _ in range(B)]
            p.free(None, [0 if x else 1 << 20 for x in gone])
            for b in range(B):
                if gone[b]:
                    p.lens[b] = 0
                    p.model.lens[b] = 0
        else:
            p.compact()


def test_copy_on_write_rules():
    """All holders of a page in the call: the first keeps it. One outside: all in it copy. A page
    that ends where the sequence does is not touched. A sequence that adds nothing keeps sharing."""
    p = Pool(6, 4, 24, kinds=KINDS)
    p.grow([300, 128, 0, 0, 0, 0])
    p.fork([0, 0, 1], [2, 3, 4])
    p.reserve([0, 1, 1, 0, 5, 0])        # 0 and 3 stay outside
    p.reserve([10, 0, 0, 200, 0, 0])     # now all that still share
    p.fork([0], [5])
    p.reserve([1, 1, 1, 1, 1, 1])
    p.reserve([1, 1, 1, 1, 1, 1])        # nothing is left to do
    p.compact()


def test_pool_runs_out():
    p = Pool(4, 4, 5)
    p.grow([130, 0, 0, 0])
    p.fork([0, 0], [1, 2])
    p.reserve([300, 1, 1, 128], full=True)
    p.free(None, [1 << 20, 0, 1 << 20, 1 << 20])
    p.lens[1] = 0
    p.model.lens[1] = 0
    p.reserve([0, 0, 1, 1], full=True)
    p.free(None, [130, 0, 130, 0])
    p.reserve([0, 0, 1, 1])


@pytest.mark.parametrize("batch,per,n_pages", [(1, 1, 1), (1500, 2, 2500), (3, 70, 300), (40, 40, 9000)])
def test_sizes(batch, per, n_pages):
    """One page; more sequences than the plan has threads; long sequences; many pages."""
    kinds = ((1, (2,), torch.bfloat16),)
    p = Pool(batch, per, n_pages, 128, 1, kinds)
    live = (batch + 1) // 2
    each = min(per * 128, max(1, n_pages // (2 * live)) * 128 - 28)
    p.grow([each if b < live else 0 for b in range(batch)])
    src = list(range(batch - live))
    p.fork(src, [live + s for s in src])
    room = min(60, per * 128 - each)
    p.reserve([room if b % 3 else 0 for b in range(batch)])
    p.free(None, [0 if b % 4 == 0 else 1 << 20 for b in range(batch)])
    p.compact()


def test_empty_and_full_pools_compact():
    p = Pool(2, 3, 6)
    p.compact()
    p.grow([384, 384])
    p.compact()
    p.free(None, [0, 384])
    p.compact()


def test_bad_forks_change_nothing():
    p = Pool(5, 3, 15)
    p.grow([200, 100, 0, 0, 0])
    bit = g.GEMMA_DEVERR_FORK
    # out of range, itself, a holder of pages, a source of the call, the same twice
    assert p.fork([0, 0, 0, 0], [2, -1, 5, 2], bit) == [1, 2, 3]
    assert p.fork([1, 1, 7, -1], [1, 0, 3, 4], bit) == [0, 1, 2, 3]
    assert p.fork([2, 3], [3, 4], bit) == [0]            # 3 is a source; it holds nothing itself
    p.lens[1] = 385
    p.model.lens[1] = 385
    assert p.fork([1], [3], g.GEMMA_DEVERR_SEQ_LEN) == [0]


def test_bad_entries_and_lengths():
    """Entries that are no page, pages nobody holds, lengths beyond the table: reported, left alone."""
    p = Pool(4, 2, 8)
    p.grow([10, 10, 10, 10])
    ok = p.table[0, 0].item()
    for e in (8, 1 << 30):
        p.table[1, 0] = e
        p.model.table[1][0] = -1                         # (the model leaves it out)
        g.gemma_pages_reserve(p.pools, p.table, p.refs, p.lens, i32([1, 1, 1, 1]), workspace=p.ws,
                              device_error=p.err)
        g.gemma_pages_free(p.table, p.refs, page_size=128, keep_to=i32([128, 0, 128, 128]),
                           device_error=p.err)
        torch.cuda.synchronize()
        assert p.err.item() == g.GEMMA_DEVERR_PAGE and p.table[1, 0].item() == e
        assert p.table[0, 0].item() == ok and p.refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
        p.err.zero_()
    p.table[1, 0] = 7                                    # a free page
    g.gemma_pages_reserve(p.pools, p.table, p.refs, p.lens, i32([0, 1, 0, 0]), workspace=p.ws,
                          device_error=p.err)
    torch.cuda.synchronize()
    assert p.err.item() == g.GEMMA_DEVERR_PAGE and p.table[1, 0].item() == 7
    p.err.zero_()
    p.table[1, 0] = 1
    for lens, add in (([10, -1, 10, 10], [1, 1, 1, 1]), ([10, 10, 10, 10], [1, -1, 1, 1]),
                      ([10, 256, 10, 10], [1, 1, 1, 1]), ([10, 10, 10, 2 ** 31 - 1], [1, 1, 1, 2 ** 31 - 1])):
        g.gemma_pages_reserve(p.pools, p.table, p.refs, i32(lens), i32(add), workspace=p.ws,
                              device_error=p.err)
        torch.cuda.synchronize()
        assert p.err.item() == g.GEMMA_DEVERR_WRITE_POS
        assert p.table.tolist() == [[0, -1], [1, -1], [2, -1], [3, -1]]
        p.err.zero_()


def test_a_table_entry_of_a_free_page_survives_compaction():
    p = Pool(2, 3, 9)
    p.grow([384, 384])
    p.free(None, [0, 384])
    p.table[0, 0] = 8                                    # nobody holds page 8
    g.gemma_pages_compact(p.pools, p.table, p.refs, workspace=p.ws, device_error=p.err)
    torch.cuda.synchronize()
    assert p.err.item() == g.GEMMA_DEVERR_PAGE
    assert p.table.tolist() == [[8, -1, -1], [0, 1, 2]]


def test_captured_and_replayed():
    """A step of free, fork and reserve in a graph: every replay starts from the state before it."""
    p, q = (Pool(4, 4, 20, seed=3, kinds=KINDS) for _ in range(2))
    for x in (p, q):
        x.grow([200, 129, 0, 0])
    src, dst, add = i32([0, 1]), i32([2, 3]), i32([1, 1, 1, 1])
    to = i32([200, 129, 0, 0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.gemma_pages_free(p.table, p.refs, page_size=128, keep_to=to, device_error=p.err)
        g.gemma_pages_fork(p.table, p.refs, p.lens, src, dst, page_size=128, device_error=p.err)
        g.gemma_pages_reserve(p.pools, p.table, p.refs, p.lens, add, workspace=p.ws,
                              device_error=p.err)
    for _ in range(3):
        graph.replay()
        q.free(None, [200, 129, 0, 0])
        q.fork([0, 1], [2, 3])
        q.reserve([1, 1, 1, 1])
    torch.cuda.synchronize()
    assert p.err.item() == 0
    assert torch.equal(p.table, q.table) and torch.equal(p.refs, q.refs)
    assert all(torch.equal(a, b) for a, b in zip(p.pools, q.pools))


def test_more_pools_than_one_launch_takes():
    p = Pool(2, 2, 4, kinds=((1, (8,), torch.bfloat16),) * 150)
    p.grow([100, 0])
    p.fork([0], [1])
    p.reserve([1, 1])
    p.free(None, [0, 256])
    p.compact()


def test_large_pages():
    """Pages of many copy units, offsets in a pool beyond 32 bits."""
    n = 80
    x = torch.zeros(n, 8, 256, 16384, dtype=torch.bfloat16, device="cuda")    # 64 MB a page, 5.4 GB
    table = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    x[70] = torch.randn(8, 256, 16384, device="cuda").bfloat16()
    table[0, 0] = 70
    refs[70], refs[75] = 2, 0
    table[1, 0] = 70
    lens, err = i32([200, 200]), i32([0])
    ws = torch.empty(g.gemma_pages_workspace_size(n), dtype=torch.uint8, device="cuda")
    g.gemma_pages_reserve([x], table, refs, lens, i32([1, 1]), workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and table.tolist() == [[70, -1], [75, -1]]
    assert torch.equal(x[75][:, :200], x[70][:, :200]) and (x[75][:, 200:] == 0).all()
    refs[3] = 0
    g.gemma_pages_compact([x], table, refs, workspace=ws, device_error=err)   # page 79 to page 3
    refs[60] = 0
    refs[76:] = 0
    g.gemma_pages_compact([x], table, refs, workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and table.tolist() == [[70, -1], [60, -1]]
    assert torch.equal(x[60], x[75])
