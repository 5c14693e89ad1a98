"""Refusals of the drafted-tree and page entry points: every check fails on the host, before any
launch, so no GPU is touched. And the plain models that the GPU tests compare with."""
import ctypes

import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref
from mixed_sliding_global_gb300 import binding

INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = -1, -2, -3, -4
FAKE = 1 << 20            # aligned, never dereferenced
BAD = FAKE + 8


def lib():
    return g.library()


def _ptrs(*xs):
    return (ctypes.c_void_p * len(xs))(*xs)


def _i32(*xs):
    return (ctypes.c_int32 * len(xs))(*xs)


def attn(out=FAKE, q=FAKE, kc=(FAKE,), vc=(FAKE,), owner=(0,), layer=0, lens=FAKE, parents=FAKE,
         real=None, table=None, max_pages=4, page=128, n_pages=9, msl=64, nodes=8, batch=1, kind=1,
         window=0, n_q=4, n_kv=2, d=64, k_eq_v=0, cap=64, scale=0.125, softcap=0.0, dtype=0,
         ws=FAKE, ws_bytes=1 << 40, err=None):
    return lib().gemma_attn_tree(out, q, _ptrs(*kc), _ptrs(*vc), _i32(*owner), len(owner), layer,
                                 lens, parents, real, table, max_pages, page, n_pages, msl, nodes,
                                 batch, kind, window, n_q, n_kv, d, k_eq_v, cap, scale, softcap,
                                 dtype, ws, ws_bytes, err, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(d=96), UNSUPPORTED),
    (dict(n_q=6, n_kv=2), UNSUPPORTED),                  # group of 3
    (dict(n_q=64, n_kv=2), UNSUPPORTED),                 # group of 32
    (dict(nodes=129), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED),
    (dict(nodes=-1), INVALID),
    (dict(batch=-1), INVALID),
    (dict(msl=0), INVALID),
    (dict(msl=65), CAPACITY),
    (dict(msl=(1 << 30) + 1, cap=(1 << 30) + 1), UNSUPPORTED),
    (dict(batch=64, n_kv=4, msl=1 << 28, cap=1 << 28), UNSUPPORTED),  # 2^30 key tiles and a few
    (dict(cap=0), INVALID),
    (dict(kind=3), INVALID),
    (dict(kind=0, window=0), INVALID),
    (dict(kind=2, window=100, cap=100), UNSUPPORTED),    # a ring of no multiple of 128
    (dict(kind=2, window=122, cap=128), CAPACITY),       # 122 + 8 - 1 slots
    (dict(kind=2, window=64, cap=128, table=FAKE), INVALID),
    (dict(table=FAKE, page=64), UNSUPPORTED),
    (dict(table=FAKE, page=192), UNSUPPORTED),
    (dict(table=FAKE, n_pages=0), INVALID),
    (dict(table=FAKE, max_pages=1, msl=129), CAPACITY),
    (dict(table=BAD + 2), INVALID),
    (dict(owner=(1,)), INVALID),
    (dict(layer=1), INVALID),
    (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(softcap=-1.0), INVALID),
    (dict(softcap=float("inf")), INVALID),
    (dict(dtype=2), INVALID),
    (dict(vc=(None,)), INVALID),
    (dict(kc=(None,)), INVALID),
    (dict(out=None), INVALID),
    (dict(q=BAD), INVALID),
    (dict(kc=(BAD,)), INVALID),
    (dict(parents=None), INVALID),
    (dict(parents=FAKE + 2), INVALID),
    (dict(lens=FAKE + 1), INVALID),
    (dict(real=FAKE + 2), INVALID),
    (dict(err=FAKE + 2), INVALID),
])
def test_attn_tree_refuses(kwargs, status):
    assert attn(**kwargs) == status


def test_attn_tree_empty_calls():
    assert attn(batch=0) == 0
    assert attn(nodes=0) == 0


@pytest.mark.parametrize("kwargs", [dict(batch=-1), dict(n_nodes=0), dict(n_nodes=129),
                                    dict(head_dim=48), dict(max_seq_len=0), dict(kind=7),
                                    dict(batch=65536), dict(n_q=5)])
def test_workspace_size_refuses_what_the_call_refuses(kwargs):
    args = dict(batch=1, kind=1, window=0, n_q=4, n_kv=2, head_dim=64, max_seq_len=64, n_nodes=8)
    args.update(kwargs)
    with pytest.raises(ValueError):
        g.gemma_attn_workspace_size_tree(**args)
    assert g.gemma_attn_workspace_size_tree(0, 1, 0, 4, 2, 64, 64, 8) == 0


def accept(tokens=FAKE, parents=FAKE, nxt=FAKE, real=None, lens=None, batch=1, nodes=4, path=FAKE,
           keep=FAKE, token=FAKE, lens_out=None, err=None):
    return lib().gemma_tree_accept(tokens, parents, nxt, real, lens, batch, nodes, path, keep, token,
                                   lens_out, err, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(nodes=0), INVALID), (dict(nodes=129), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(tokens=None), INVALID), (dict(parents=None), INVALID), (dict(nxt=FAKE + 2), INVALID),
    (dict(path=None), INVALID), (dict(keep=None), INVALID), (dict(token=FAKE + 1), INVALID),
    (dict(lens_out=FAKE), INVALID),                      # without seq_lens
    (dict(real=FAKE + 2), INVALID), (dict(err=FAKE + 2), INVALID), (dict(batch=0), 0),
])
def test_tree_accept_refuses(kwargs, status):
    assert accept(**kwargs) == status


def keep(caches=(FAKE,), pos=FAKE, path=FAKE, n=FAKE, table=None, max_pages=4, page=128, n_pages=9,
         batch=1, nodes=4, kind=1, n_kv=2, cap=64, row=128, err=None):
    return lib().gemma_kv_keep(_ptrs(*caches), len(caches), pos, path, n, table, max_pages, page,
                               n_pages, batch, nodes, kind, n_kv, cap, row, err, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(caches=()), 0), (dict(batch=0), 0),
    (dict(caches=(FAKE, None)), INVALID), (dict(caches=(BAD,)), INVALID),
    (dict(pos=None), INVALID), (dict(path=FAKE + 2), INVALID), (dict(n=None), INVALID),
    (dict(row=3), INVALID), (dict(row=0), INVALID), (dict(n_kv=0), INVALID),
    (dict(nodes=0), INVALID), (dict(nodes=129), UNSUPPORTED), (dict(kind=5), INVALID),
    (dict(cap=0), INVALID), (dict(kind=2, cap=3), CAPACITY), (dict(batch=65536), UNSUPPORTED),
    (dict(table=FAKE, page=100), UNSUPPORTED), (dict(table=FAKE, kind=2), INVALID),
    (dict(table=FAKE + 2), INVALID), (dict(err=FAKE + 1), INVALID),
    (dict(n_kv=1 << 20, row=1 << 12), UNSUPPORTED),
])
def test_kv_keep_refuses(kwargs, status):
    assert keep(**kwargs) == status


def free(table=FAKE, max_pages=4, page=128, n_pages=9, refs=FAKE, lo=None, hi=FAKE, batch=2,
         err=None):
    return lib().gemma_pages_free(table, max_pages, page, n_pages, refs, lo, hi, batch, err, None)


def fork(table=FAKE, max_pages=4, page=128, n_pages=9, refs=FAKE, lens=FAKE, src=FAKE, dst=FAKE, n=1,
         batch=2, err=None):
    return lib().gemma_pages_fork(table, max_pages, page, n_pages, refs, lens, src, dst, n, batch,
                                  err, None)


def reserve(pools=(FAKE,), n_kv=(2,), row=(128,), table=FAKE, max_pages=4, page=128, n_pages=9,
            refs=FAKE, lens=FAKE, add=FAKE, batch=2, ws=FAKE, ws_bytes=1 << 40, err=None):
    return lib().gemma_pages_reserve(_ptrs(*pools), _i32(*n_kv), _i32(*row), len(pools), table,
                                     max_pages, page, n_pages, refs, lens, add, batch, ws, ws_bytes,
                                     err, None)


def compact(pools=(FAKE,), n_kv=(2,), row=(128,), table=FAKE, max_pages=4, page=128, n_pages=9,
            refs=FAKE, used=None, batch=2, ws=FAKE, ws_bytes=1 << 40, err=None):
    return lib().gemma_pages_compact(_ptrs(*pools), _i32(*n_kv), _i32(*row), len(pools), table,
                                     max_pages, page, n_pages, refs, used, batch, ws, ws_bytes, err,
                                     None)


@pytest.mark.parametrize("call", [free, fork, reserve, compact])
@pytest.mark.parametrize("kwargs,status", [
    (dict(batch=0), 0), (dict(batch=-1), INVALID), (dict(table=None), INVALID),
    (dict(refs=None), INVALID), (dict(table=FAKE + 2), INVALID), (dict(refs=FAKE + 1), INVALID),
    (dict(err=FAKE + 2), INVALID), (dict(page=0), INVALID), (dict(page=130), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(n_pages=(1 << 29) + 1), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(batch=65535, max_pages=1 << 16), UNSUPPORTED),
])
def test_pages_refuse(call, kwargs, status):
    assert call(**kwargs) == status


@pytest.mark.parametrize("status,made", [
    (INVALID, lambda: free(hi=None)), (INVALID, lambda: free(hi=FAKE + 2)),
    (INVALID, lambda: free(lo=FAKE + 1)),
    (INVALID, lambda: fork(n=-1)), (0, lambda: fork(n=0)), (INVALID, lambda: fork(n=3)),
    (INVALID, lambda: fork(src=None)), (INVALID, lambda: fork(dst=FAKE + 2)),
    (INVALID, lambda: fork(lens=None)),
    (INVALID, lambda: reserve(lens=None)), (INVALID, lambda: reserve(add=FAKE + 2)),
    (INVALID, lambda: compact(used=FAKE + 2)),
] + [x for call in (reserve, compact) for x in [
    (INVALID, lambda call=call: call(pools=(), n_kv=(), row=())),
    (INVALID, lambda call=call: call(pools=(BAD,))),
    (INVALID, lambda call=call: call(pools=(FAKE, None), n_kv=(1, 1), row=(2, 2))),
    (INVALID, lambda call=call: call(n_kv=(0,))),
    (INVALID, lambda call=call: call(row=(3,))),
    (UNSUPPORTED, lambda call=call: call(n_kv=(1 << 14,), row=(1 << 10,))),   # 2 GB a page
    (WORKSPACE, lambda call=call: call(ws=None)),
    (WORKSPACE, lambda call=call: call(ws=BAD)),
    (WORKSPACE, lambda call=call: call(ws_bytes=g.gemma_pages_workspace_size(9) - 1)),
]])
def test_pages_refuse_their_own_arguments(status, made):
    assert made() == status


def test_pages_workspace_size():
    for n in (0, -1, (1 << 29) + 1):
        with pytest.raises(ValueError):
            g.gemma_pages_workspace_size(n)
    assert g.gemma_pages_workspace_size(1) > 0


def test_python_calls_check_shapes_and_types():
    """Bad shapes, types and devices are refused by the binding, with no launch (CPU tensors are
    refused as such before anything is read)."""
    i = torch.zeros(2, 4, dtype=torch.int32)
    q = torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 64, 64, dtype=torch.bfloat16)
    kw = dict(kind=1, window=0, n_kv=2, k_eq_v=False, scale=0.1)
    with pytest.raises(ValueError):                      # out of another shape
        g.gemma_attn_tree(q[:, :3], q, [k], [k], [0], 0, i[:, 0], i, 64, **kw)
    with pytest.raises(ValueError):                      # CPU tensors
        g.gemma_attn_tree(q, q, [k], [k], [0], 0, i[:, 0].contiguous(), i, 64, **kw)
    with pytest.raises(g.GemmaError):                    # an owner behind its layer
        g.gemma_attn_tree(q, q, [k], [k], [1], 0, i[:, 0].contiguous(), i, 64, **kw)
    with pytest.raises(ValueError):
        g.gemma_tree_accept(i[0], i, i, i, i[:, 0], i[:, 0])
    with pytest.raises(TypeError):
        g.gemma_tree_accept(None, i, i, i, i[:, 0], i[:, 0])
    with pytest.raises(ValueError):
        g.gemma_kv_keep([k[0]], i[:, 0], i, i[:, 0])
    with pytest.raises(ValueError):
        g.gemma_pages_free(i[0], i[0], page_size=128, keep_to=i[:, 0])
    with pytest.raises(ValueError):
        g.gemma_pages_fork(i, i[0], i[:, 0], i[0], i[0], page_size=128)
    with pytest.raises(ValueError):
        g.gemma_pages_reserve([k], i, i[0], i[:, 0], i[:, 0])
    with pytest.raises(ValueError):
        g.gemma_pages_compact([k], i, i[0])


# ---- the models that the GPU tests compare with ------------------------------------------------
def test_reference_chain_is_causal_attention():
    """A chain attends what causal attention attends, with and without a window."""
    n, base = 5, 7
    parents = [-1, 0, 1, 2, 3]
    for kind, window in ((tree_ref.GLOBAL, 0), (tree_ref.SLIDING, 4), (tree_ref.SLIDING, 1)):
        see = tree_ref.keys_of(parents, n, base, kind, window)
        for i in range(n):
            p = base + i
            want = [j <= p and (kind == tree_ref.GLOBAL or p - j < window) for j in range(base + n)]
            assert see[i].tolist() == want


def test_reference_siblings_do_not_see_each_other():
    #      0 -> 1 -> 3,  0 -> 2 -> 4, a second root 5
    see = tree_ref.keys_of([-1, 0, 0, 1, 2, -1], 6, 2, tree_ref.GLOBAL, 0).int().tolist()
    assert see[3] == [1, 1, 1, 1, 0, 1, 0, 0]
    assert see[4] == [1, 1, 1, 0, 1, 0, 1, 0]
    assert see[5] == [1, 1, 0, 0, 0, 0, 0, 1]
    # window 2: depth 2 sees its parent and itself; a root one prefix key
    see = tree_ref.keys_of([-1, 0, 0, 1, 2, -1], 6, 2, tree_ref.SLIDING, 2).int().tolist()
    assert see[3] == [0, 0, 0, 1, 0, 1, 0, 0]
    assert see[1] == [0, 0, 1, 1, 0, 0, 0, 0]
    assert see[5] == [0, 1, 0, 0, 0, 0, 0, 1]


def test_reference_accept():
    parents, tokens = [-1, 0, 0, 1, 1, 3], [9, 4, 5, 6, 6, 7]
    assert tree_ref.accept(tokens, parents, [4, 6, 0, 7, 0, 8], 6) == ([0, 1, 3, 5], 8)
    assert tree_ref.accept(tokens, parents, [5, 6, 1, 7, 0, 8], 6) == ([0, 2], 1)
    assert tree_ref.accept(tokens, parents, [-1, 6, 1, 7, 0, 8], 6) == ([0], -1)
    assert tree_ref.accept(tokens, parents, [4, 6, 0, 7, 0, 8], 5) == ([0, 1, 3], 7)


def test_reference_pages():
    pools = [torch.arange(6 * 2 * 4).reshape(6, 2, 4, 1).clone()]
    m = tree_ref.Pages([[5, 1, -1], [-1] * 3, [-1] * 3], [0, 1, 0, 0, 0, 1], [6, 0, 0], pools, 4)
    assert m.fork([0, 0, 0], [1, 2, 2]) == [2]
    assert m.table[2] == [5, 1, -1] and m.refs == [0, 3, 0, 0, 0, 3] and m.lens == [6, 6, 6]
    assert not m.reserve([1, 1, 3])                     # all three write to page 1
    assert m.table == [[5, 1, -1], [5, 0, -1], [5, 2, 3]] and m.refs == [1, 1, 1, 1, 0, 3]
    assert torch.equal(m.pools[0][0][:, :2], pools[0][1][:, :2])
    assert torch.equal(m.pools[0][0][:, 2:], pools[0][0][:, 2:])
    m.free([4, 0, 0], [12, 0, 12])
    assert m.table == [[-1, 1, -1], [-1, -1, -1], [5, 2, 3]] and m.refs == [0, 1, 1, 1, 0, 1]
    assert m.compact() == 4 and m.table == [[-1, 1, -1], [-1, -1, -1], [0, 2, 3]]


def test_binding_covers_the_tree_and_page_calls():
    for name in ("gemma_attn_tree", "gemma_tree_accept", "gemma_kv_keep", "gemma_pages_free",
                 "gemma_pages_fork", "gemma_pages_reserve", "gemma_pages_compact"):
        assert name in binding._SIGNATURES and hasattr(g, name)
