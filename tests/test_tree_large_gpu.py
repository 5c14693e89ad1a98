"""Drafted trees and pages in caches of more than 2^31 elements: rows, pages and moves behind offsets that
32 bits hold."""
import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref
from test_tree_gpu import random_tree

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n_q,n_kv,d,nodes,dtype", [
    (16, 8, 512, 6, torch.bfloat16),     # a warp's matrix instructions
    (16, 1, 512, 6, torch.bfloat16),     # pairs
    (16, 2, 256, 20, torch.bfloat16),
    (16, 8, 256, 6, torch.bfloat16),     # one SM
    (16, 4, 64, 10, torch.bfloat16),
    (4, 2, 512, 3, torch.float32)])
def test_rows_behind_32_bits(n_q, n_kv, d, nodes, dtype, paged):
    window, page = 100, 256
    cap = (1 << 31) // (n_kv * d) + 4 * page
    cap -= cap % page
    n = cap - 7 if not paged else 5 * page - 7          # the sequence's length
    gen = torch.Generator().manual_seed(d)
    near = 256                                          # rows before the tree that are filled
    rows = torch.randn(near + nodes, n_kv, d, generator=gen).to(dtype).cuda()
    q = torch.randn(1, nodes, n_q, d, generator=gen).to(dtype).cuda()
    parents = random_tree(gen, nodes, 1.0)
    at = torch.arange(n - nodes - near, n, device="cuda")
    table = None
    if paged:
        n_pages = cap // page
        pool = torch.empty(n_pages, n_kv, page, d, dtype=dtype, device="cuda")
        table = i32([list(range(n_pages - 5, n_pages))])
        pool[table[0].long()[at // page], :, at % page] = rows
        cache, take = pool, lambda p: pool[table[0].long()[p // page], :, p % page]  # noqa: E731
    else:
        cache = torch.empty(1, n_kv, cap, d, dtype=dtype, device="cuda")
        cache[0][:, at] = rows.transpose(0, 1)
        take = lambda p: cache[0][:, p].transpose(0, 1)  # noqa: E731
    assert cache.numel() > 1 << 31
    err, out = i32([0]), torch.empty_like(q)
    size = g.gemma_attn_workspace_size_tree(1, g.GEMMA_SLIDING, window, n_q, n_kv, d, n, nodes)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    g.gemma_attn_tree(out, q, [cache], None, [0], 0, i32([n]), i32([parents]), n, kind=g.GEMMA_SLIDING,
                      window=window, n_kv=n_kv, k_eq_v=True, scale=d ** -0.5, block_table=table,
                      workspace=ws, device_error=err)
    # the last two nodes' rows move to the first two places
    pos = n - nodes
    path = i32([[nodes - 2, nodes - 1] + [-1] * (nodes - 2)])
    want = take(torch.tensor([n - 2, n - 1], device="cuda")).clone()
    rest = take(torch.arange(pos + 2, n, device="cuda")).clone()
    g.gemma_kv_keep([cache], i32([pos]), path, i32([2]), block_table=table, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.equal(take(torch.tensor([pos, pos + 1], device="cuda")), want)
    assert torch.equal(take(torch.arange(pos + 2, n, device="cuda")), rest)
    see = tree_ref.keys_of(parents, nodes, near, g.GEMMA_SLIDING, window)
    ref, mass, size = tree_ref.attention(q[0], rows, rows, see, d ** -0.5)
    bits = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    # the output's rounding and P's; fp32 sums of d products and of up to 130 keys, exponentials 2^-21
    rel = bits + 2 * (d / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -20 + 130 * 2.0 ** -23
    bound = bits * ref.abs() + rel * (mass + ref.abs()) + 1e-12
    assert ((out[0].double() - ref).abs() <= bound).all()


def test_pages_behind_32_bits():
    """Pages at the end of a pool of more than 2^31 elements are shared, copied and moved."""
    n_kv, page, d = 2, 128, 512
    n_pages = (1 << 31) // (n_kv * page * d) + 50
    pool = torch.empty(n_pages, n_kv, page, d, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 31
    last = n_pages - 1
    pool[last - 1:] = torch.randn(2, n_kv, page, d, device="cuda").bfloat16()
    data = pool[last - 1:].clone()
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    refs, lens = i32([0] * n_pages), i32([200, 0, 0])
    refs[:] = 1                                     # all taken but three pages far behind
    refs[last - 5:last - 2] = 0
    table[0, :2] = i32([last - 1, last])
    err = i32([0])
    ws = torch.empty(g.gemma_pages_workspace_size(n_pages), dtype=torch.uint8, device="cuda")
    g.gemma_pages_fork(table, refs, lens, i32([0]), i32([1]), page_size=page, device_error=err)
    g.gemma_pages_reserve([pool], table, refs, lens, i32([0, 5, 0]), workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert table[1].tolist() == [last - 1, last - 5, -1, -1]
    assert torch.equal(pool[last - 5, :, :72], data[1, :, :72])
    refs[:last - 10] = 0                            # and now hardly any: the pages move to the front
    refs[last - 10:last - 5] = 0
    n_used = i32([-1])
    refs[last - 4:last - 1] = 0
    refs[last - 1] = 2
    g.gemma_pages_compact([pool], table, refs, n_used=n_used, workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0 and n_used.item() == 3
    assert table[:2].tolist() == [[1, 2, -1, -1], [1, 0, -1, -1]]
    assert refs[:4].tolist() == [1, 2, 1, 0]
    assert torch.equal(pool[1:3], data) and torch.equal(pool[0, :, :72], data[1, :, :72])
