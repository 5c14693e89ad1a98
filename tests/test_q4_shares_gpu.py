"""GPU: 4-bit attention dealt as equal shares of the launch's key tiles, with its merge launch.

A call takes that way where the workspace query asks for scratch although its rows attend straight over
the cache; every test here asserts that. The bound is test_q4_gpu.py's for such rows:
2^-8 |out| + (2^-10 + 2^-13) A, A = sum p |v|."""
import math

import pytest
import torch

import mixed_sliding_global_gb300 as g
import q4_ref as R

pytestmark = pytest.mark.gpu

SLIDING, GLOBAL, RING = R.SLIDING, R.GLOBAL, R.RING


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A cache of random 4-bit rows, plain, paged or a ring of `ring` slots; rows behind a sequence's
    end hold NaN."""

    def __init__(self, lens, n_q, n_kv, d, msl, *, k_eq_v=False, page=0, n=1, seed=0, ring=0):
        self.lens, self.msl, self.n, self.page, self.k_eq_v = lens, msl, n, page, k_eq_v
        self.n_kv, self.d = n_kv, d
        gen = torch.Generator().manual_seed(seed)
        B, unit = len(lens), page or 32
        slots = ring or -(-msl // unit) * unit
        self.table = None
        shape = (B, n_kv, slots)
        if page:
            per = slots // page
            self.table = torch.randperm(B * per + 2, generator=gen)[:B * per].int().reshape(B, per)
            shape = (B * per + 2, n_kv, page)
        self.shape = shape
        self.t = []
        for _ in range(1 if k_eq_v else 2):
            codes = torch.randint(0, 256, shape + (d // 2,), generator=gen, dtype=torch.uint8)
            # five significant bits; keys of about unit variance
            s = (16 + torch.randint(0, 16, shape + (d // 64,), generator=gen)).float() / 64
            self.t += [codes, s.bfloat16()]
        for b, L in enumerate(lens):
            at = torch.arange(slots if ring else max(0, L) if L <= msl else 0, slots)
            where, slot = R.locate(at, b, GLOBAL, slots, self.table, page)
            for s in self.t[1::2]:
                s[where, :, slot] = math.nan
        self.q = torch.randn(B, n, n_q, d, generator=gen).bfloat16()

    def attend(self, kind=GLOBAL, window=0, softcap=0.0, table=None):
        B, _, n_q, d = self.q.shape
        args = [[x.cuda()] for x in self.t] + ([[None], [None]] if self.k_eq_v else [])
        if table is None:
            table = self.table
        q, err = self.q.cuda(), i32([0])
        size = g.gemma_attn_workspace_size_q4(B, kind, window, n_q, self.n_kv, d, self.msl, self.n,
                                              k_eq_v=self.k_eq_v)
        assert self.n * n_q // self.n_kv <= 64 and size > 0     # straight over the cache, in shares
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, math.nan)
        g.gemma_attn_q4(out, q, *args, [0], 0, i32(self.lens), self.msl, kind=kind, window=window,
                        n_kv=self.n_kv, k_eq_v=self.k_eq_v, scale=0.5 * d ** -0.5, softcap=softcap,
                        block_table=None if table is None else table.cuda(), workspace=ws,
                        device_error=err)
        torch.cuda.synchronize()
        return out.cpu(), err.item()

    def check(self, out, kind=GLOBAL, window=0, softcap=0.0, lost=()):
        """Against 64 bits; pages in `lost` read as zeros; sequences of a bad length are zero."""
        good = [b for b, L in enumerate(self.lens) if self.n <= L <= self.msl]
        v = [R.values(self.t[i], self.t[i + 1]) for i in range(0, len(self.t), 2)]
        for x in v:
            for page in lost:
                x[page] = 0
        pick = slice(None) if self.page else good
        table = None if self.table is None else self.table[good]
        ref, mass = R.attention(self.q[good], v[0][pick], v[-1][pick], [self.lens[b] for b in good],
                                kind, window, 0.5 * self.d ** -0.5, softcap, table, self.page)
        err = (out[good].double() - ref).abs()
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -13) * mass + 1e-6
        assert torch.isfinite(out).all()
        assert (err <= bound).all(), (err / bound).max().item()
        bad = [b for b in range(len(self.lens)) if b not in good]
        assert (out[bad] == 0).all()


@pytest.mark.parametrize("n_q,n_kv,d,k_eq_v,n", [
    (8, 8, 256, False, 1), (16, 8, 128, False, 3), (16, 2, 512, False, 1), (16, 4, 512, True, 2)])
def test_runs_of_bad_lengths(n_q, n_kv, d, k_eq_v, n):
    """Runs of sequences whose length is out of range between valid ones: more units in a row than
    the ring has stages, none of which has a tile to wait for. The valid ones are as they are."""
    msl = 2048
    lens = [msl, 0, -3, msl + 1, 900, 2 ** 31 - 1] + [n - 1, 5000] * 3 + [1300, n] + [-1] * 6 + [2000]
    c = Case(lens, n_q, n_kv, d, msl, k_eq_v=k_eq_v, n=n, seed=d + n)
    out, err = c.attend()
    assert err == g.GEMMA_DEVERR_SEQ_LEN
    c.check(out)


@pytest.mark.parametrize("n_q,n_kv,d,k_eq_v,n", [(8, 2, 256, False, 1), (16, 1, 512, False, 1)])
def test_bad_pages_among_good_ones(n_q, n_kv, d, k_eq_v, n):
    """Pages that are none read as zeros, and the tiles that reuse their stages as what they hold."""
    lens = [8192, 2000, 8000, 100, 6500, 8192]
    c = Case(lens, n_q, n_kv, d, 8192, k_eq_v=k_eq_v, page=128, n=n, seed=d + 1)
    table, lost = c.table.clone(), []
    gen = torch.Generator().manual_seed(5)
    for b, L in enumerate(lens):
        pages = torch.randperm(-(-L // 128), generator=gen)[:9].tolist()
        for i, page in enumerate(pages[1:]):
            lost.append(int(table[b, page]))
            table[b, page] = (-1, c.shape[0], 2 ** 30, -2 ** 31)[i % 4]
    out, err = c.attend(table=table)
    assert err == g.GEMMA_DEVERR_PAGE
    c.check(out, lost=lost)


@pytest.mark.parametrize("lens,n_q,n_kv,d,msl,opt", [
    # one long sequence, K as V; a window far into a long one; a ring
    ([8192], 16, 1, 512, 8192, dict(k_eq_v=True)),
    ([9000, 6100], 16, 1, 128, 9000, dict(kind=SLIDING, window=5000)),
    ([4001, 7000, 20000], 4, 1, 256, 20000, dict(kind=RING, window=4000)),
    # ragged batches at each head_dim, rows per unit of 2, 8, 16 and more
    ([6000, 1, 333, 5888, 128, 4097, 2, 129, 700, 3000, 5999, 64], 16, 8, 64, 6000, {}),
    ([6000, 1, 333, 5888, 128, 4097, 2, 129, 700, 3000, 5999, 64], 64, 8, 64, 6000, dict(cap=20.0)),
    ([2900, 4000, 1300, 4096, 1, 2047, 3999, 130] + [500 + 11 * i for i in range(25)], 64, 4, 64, 4096,
     dict(k_eq_v=True)),
    ([5999, 2, 6000, 1025], 8, 2, 128, 6000, dict(n=2)),
    ([5999, 2, 6000, 1025], 16, 2, 128, 6000, dict(k_eq_v=True, page=128)),
    ([6000, 17, 4100], 16, 1, 128, 6000, dict(n=3)),
    ([4500, 700, 3210, 4, 2222, 1, 4400, 999, 129, 4096, 3333, 2048, 1500], 8, 2, 256, 4500,
     dict(cap=50.0, page=256)),
    ([2000, 6000, 100], 2, 1, 256, 6000, dict(k_eq_v=True)),
    ([2000, 6000, 100], 16, 2, 256, 6000, {}),
    ([2000, 5990, 100], 16, 1, 256, 6000, dict(n=4, cap=30.0)),
    ([3000, 40, 2500, 1], 4, 2, 512, 3000, {}),
    ([3000, 40, 2500, 5], 8, 1, 512, 3000, dict(page=128)),
    ([3000, 40, 2500, 5], 16, 1, 512, 3000, dict(n=4)),
    ([2999, 41, 2501, 1], 32, 2, 512, 3000, dict(k_eq_v=True, cap=20.0)),
])
def test_against_the_definition(lens, n_q, n_kv, d, msl, opt):
    """Whole units, parts of units and the merge, over every instantiation: rows per unit up to 4, up
    to 8 and more, with K as V and without, windows, rings, pages and caps."""
    o = dict(kind=GLOBAL, window=0, cap=0.0, n=1, k_eq_v=False, page=0)
    o.update(opt)
    if o["n"] > 1:
        lens = [max(x, o["n"]) for x in lens]
    ring = -(-(o["window"] + o["n"] - 1) // 128) * 128 if o["kind"] == RING else 0
    c = Case(lens, n_q, n_kv, d, msl, k_eq_v=o["k_eq_v"], page=o["page"], n=o["n"], seed=d + n_q,
             ring=ring)
    out, err = c.attend(o["kind"], o["window"], o["cap"])
    assert err == 0
    c.check(out, o["kind"], o["window"], o["cap"])
