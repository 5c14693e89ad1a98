"""Attention of a drafted tree on every way that its sizes can take (matrix instructions of a warp, of
an SM with equal shares or a cluster per unit, of a pair of SMs), with ragged batches, empty and bad
sequences among the others, all layouts and caps."""
import pytest
import torch

import mixed_sliding_global_gb300 as g
from test_tree_gpu import Problem, random_tree
from tree_ref import GLOBAL, RING, SLIDING

pytestmark = pytest.mark.gpu


def ragged(batch, top, nodes, seed):
    """Lengths and node counts of a batch: one of each extreme, the rest spread."""
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(nodes, top + 1, (batch,), generator=gen).tolist()
    reals = torch.randint(0, nodes + 1, (batch,), generator=gen).tolist()
    lens[0], reals[0] = top, nodes
    if batch > 3:
        lens[1], reals[1] = nodes, nodes                 # no prefix
        reals[2] = 0                                      # no tree
        lens[3], reals[3] = 1, 1                          # one key
    return lens, reals


LAYOUTS = [dict(), dict(page=128), dict(kind=SLIDING, window=77), dict(kind=SLIDING, window=200, page=256),
           dict(kind=RING, window=300), dict(softcap=15.0, q_gain=3.0)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n_q,n_kv,d,k_eq_v,batch,top,nodes", [
    (4, 2, 64, False, 45, 700, 9),        # one SM per unit: equal shares, more sequences than a warp has lanes
    (8, 4, 256, False, 40, 500, 33),      # 160 units, 66 rows
    (16, 1, 128, True, 4, 900, 20),       # three row tiles of 128
    (8, 4, 256, True, 8, 400, 8),         # a cluster of several CTAs per unit
    (2, 2, 64, False, 3, 300, 7),
    (4, 2, 128, False, 40, 130, 12),      # units of few tiles: one CTA each
    (16, 2, 256, False, 35, 400, 40),     # pairs: 320 rows, two row tiles
    (16, 1, 256, True, 2, 2000, 16),      # pairs: few units, many parts
    (16, 1, 512, True, 34, 350, 6),       # pairs at head_dim 512, in two halves
    (8, 2, 512, False, 5, 900, 100),
    (16, 1, 512, True, 45, 300, 6),       # more units than pairs, short ones: whole ones to each
    (4, 2, 64, False, 90, 300, 11),       # the same of SMs
    (16, 2, 256, False, 35, 1500, 40),    # many more units than pairs, cut
    (16, 1, 512, True, 60, 900, 6),
    (8, 4, 256, False, 60, 900, 10),      # the same of SMs
    (4, 2, 64, False, 120, 900, 9),
    (4, 2, 512, False, 20, 600, 15),      # head_dim 512, 30 rows
    (2, 2, 512, True, 20, 600, 16),
])
def test_ragged_batches(layout, n_q, n_kv, d, k_eq_v, batch, top, nodes):
    lens, reals = ragged(batch, top, nodes, d + nodes)
    p = Problem(lens, reals, nodes, n_q=n_q, n_kv=n_kv, d=d, k_eq_v=k_eq_v, seed=nodes + batch, **layout)
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", [dict(), dict(page=256), dict(kind=SLIDING, window=2900),
                                    dict(kind=RING, window=2800), dict(softcap=15.0, q_gain=3.0),
                                    dict(k_eq_v=True)])
@pytest.mark.parametrize("group,nodes", [(1, 1), (1, 16), (2, 7), (4, 4)])
def test_few_rows_over_many_keys(d, layout, group, nodes):
    """Over 100,000 keys in all (sequences x KV heads x positions): up to 16 rows per KV head."""
    lens, reals = ragged(5, 4100, nodes, nodes)
    lens[4], reals[4] = 3999, nodes
    p = Problem(lens, reals, nodes, n_q=8 * group, n_kv=8, d=d, seed=d + nodes, **layout)
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("n_q,n_kv,d,nodes,batch,top", [
    (4, 2, 64, 9, 40, 300), (4, 2, 64, 3, 2, 100), (16, 1, 256, 9, 36, 300), (16, 1, 512, 9, 9, 300),
    (2, 2, 512, 9, 9, 300), (8, 8, 128, 8, 9, 2100), (16, 2, 256, 9, 50, 300), (16, 1, 512, 9, 50, 300),
    (4, 2, 64, 9, 100, 300), (16, 2, 256, 9, 60, 1300), (4, 2, 64, 9, 120, 900), (16, 1, 512, 9, 3, 900)])
def test_bad_sequences_among_others(n_q, n_kv, d, nodes, batch, top):
    """Bad lengths, counts and trees are skipped and reported; every other sequence is what it is alone."""
    gen = torch.Generator().manual_seed(7)
    lens = torch.randint(nodes, top + 1, (batch,), generator=gen).tolist()
    reals = [nodes] * batch
    p = Problem(lens, reals, nodes, n_q=n_q, n_kv=n_kv, d=d, k_eq_v=True, seed=d)
    p.msl = top
    p.k = torch.cat([p.k, torch.zeros_like(p.k[:, :, :1]).expand(-1, -1, top - p.k.shape[2], -1)],
                    2).contiguous() if top > p.k.shape[2] else p.k
    bad = {0: g.GEMMA_DEVERR_SEQ_LEN, batch - 1: g.GEMMA_DEVERR_TREE}
    p.lens = list(lens)
    p.lens[0] = top + 1
    p.parents = [list(x) for x in p.parents]
    p.parents[-1][nodes - 1] = nodes
    if batch > 4:
        p.reals = list(reals)
        p.reals[batch // 2] = nodes + 1
        bad[batch // 2] = g.GEMMA_DEVERR_N_REAL
    out = p.run()
    want = 0
    for bit in bad.values():
        want |= bit
    assert p.err == want
    p.reals = reals
    p.check(out, skipped=tuple(bad))


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens", [
    (8, 2, 256, 8, [1500]), (8, 2, 256, 40, [1500, 90]), (16, 1, 512, 12, [1500, 90]),
    (2, 2, 512, 12, [1500, 90]), (8, 8, 64, 4, [4000] * 4)])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_nan_outside_of_a_sequence_and_in_pad_rows(n_q, n_kv, d, nodes, lens, bad):
    """Rows behind a sequence's own nodes are zeros whatever the values of the others: one tree's V holds
    NaN or infinities at its root, which all its nodes attend, and its pad rows stay zero."""
    p = Problem(lens, [nodes - 2] * len(lens), nodes, n_q=n_q, n_kv=n_kv, d=d, seed=1)
    for b, n in enumerate(lens):
        p.v[b, :, n - (nodes - 2)] = float(bad)
    out = p.run()
    assert p.err == 0
    assert (out[:, nodes - 2:] == 0).all()
    assert not torch.isfinite(out[:, 0]).any()


@pytest.mark.parametrize("n_q,n_kv,d,nodes", [(4, 2, 128, 20), (16, 1, 256, 20), (16, 1, 512, 20),
                                              (2, 2, 512, 5)])
def test_an_output_of_16_byte_alignment(n_q, n_kv, d, nodes):
    """Rows and outputs aligned to 16 bytes and no more."""
    p = Problem([300, 77], [nodes, nodes], nodes, n_q=n_q, n_kv=n_kv, d=d, seed=3)
    flat = torch.full((p.q.numel() + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = flat[8:].view(p.q.shape)
    q = torch.empty(p.q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(p.q.shape)
    q.copy_(p.q)
    p.q = q
    p.check(p.run(out=out))
    assert torch.isnan(flat[:8]).all()


def test_many_sequences_of_one_key():
    """3,000 sequences of a few keys: more than every CTA has threads."""
    B = 3000
    gen = torch.Generator().manual_seed(2)
    parents = [[-1, 0], [-1, -1]] * (B // 2)
    lens = torch.randint(2, 9, (B,), generator=gen).tolist()
    for n_q, n_kv, d in ((1, 1, 64), (16, 1, 512)):
        p = Problem(lens, [2, 1] * (B // 2), 2, n_q=n_q, n_kv=n_kv, d=d, k_eq_v=True, parents=parents)
        p.check(p.run())
        assert p.err == 0


@pytest.mark.parametrize("n_q,n_kv,d,nodes,top", [
    (16, 2, 256, 12, 4000), (16, 1, 512, 12, 3000), (4, 2, 64, 12, 4000), (8, 4, 128, 12, 2000),
    (16, 2, 256, 12, 300), (16, 1, 512, 12, 300), (4, 2, 64, 12, 300), (8, 4, 256, 12, 300)])
@pytest.mark.parametrize("live", [[0], [63], [7, 40], []])
def test_a_batch_with_few_live_sequences(n_q, n_kv, d, nodes, top, live):
    """A bucket of 64 sequences of which few have nodes: theirs is cut into many parts, and the rows of all
    others are zeros."""
    reals = [nodes if b in live else 0 for b in range(64)]
    lens = [top if b in live else 0 for b in range(64)]
    p = Problem(lens, reals, nodes, n_q=n_q, n_kv=n_kv, d=d, k_eq_v=True, seed=d, cap=top)
    p.msl = top
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("kind,window", [(SLIDING, 100), (SLIDING, 640), (GLOBAL, 0)])
@pytest.mark.parametrize("n_q,n_kv,d,nodes,dtype", [
    (4, 2, 64, 9, torch.bfloat16), (8, 8, 64, 8, torch.bfloat16), (4, 2, 128, 40, torch.bfloat16),
    (8, 2, 256, 8, torch.bfloat16), (16, 2, 256, 30, torch.bfloat16), (16, 1, 512, 9, torch.bfloat16),
    (2, 2, 512, 9, torch.bfloat16), (4, 2, 64, 5, torch.float32)])
def test_tables_of_the_pages_in_use(n_q, n_kv, d, nodes, dtype, kind, window):
    """Entries of pages that lie wholly below the window or behind the last key are -1, as the page
    bookkeeping leaves them: they are not read."""
    lens = [nodes, 128, 129, 256, 300, 320, 700, 1300, 2049, 2560]
    p = Problem(lens, [min(nodes, n) for n in lens], nodes, kind=kind, window=window, n_q=n_q, n_kv=n_kv,
                d=d, page=128, dtype=dtype, seed=d)
    for b, n in enumerate(lens):
        base = n - min(nodes, n)
        first = max(0, base - window + 1) if kind == SLIDING else 0
        p.table[b, :first // 128] = -1
        p.table[b, (n - 1) // 128 + 1:] = -1
    p.check(p.run())
    assert p.err == 0
