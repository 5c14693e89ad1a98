"""Caches of gemma_kv_keep that share bytes: two movers of one row would run at once, so the call is
refused on the host, before any launch."""
import ctypes

import pytest
import torch

import mixed_sliding_global_gb300 as g
from mixed_sliding_global_gb300 import binding

INVALID = -1
A = 1 << 30                # aligned, never dereferenced
BATCH, N_KV, CAP, ROW = 2, 2, 64, 128
SIZE = BATCH * N_KV * CAP * ROW
N_PAGES, PAGE = 9, 128
POOL = N_PAGES * N_KV * PAGE * ROW


def keep(caches, table=None, batch=BATCH, kind=1, n_kv=N_KV, cap=CAP, row=ROW, n_pages=N_PAGES, path=A):
    return g.library().gemma_kv_keep((ctypes.c_void_p * len(caches))(*caches), len(caches), A, path, A, table,
                                     4, PAGE, n_pages, batch, 4, kind, n_kv, cap, row, None, None)


@pytest.mark.parametrize("caches,size,kw", [
    ([0, 0], SIZE, {}),                                      # the same cache twice
    ([0, SIZE, 2 * SIZE, SIZE], SIZE, {}),
    ([0, SIZE - 16], SIZE, {}), ([SIZE - 16, 0], SIZE, {}),  # one begins in another
    ([0, 16], SIZE, {}),
    ([0, 0], SIZE, dict(kind=2, cap=128)),
    ([0, POOL - 16], POOL, dict(table=A)),
    ([i * SIZE for i in range(200)] + [150 * SIZE], SIZE, {}),  # in another launch than its double
    ([0, 1 << 62], 0, dict(n_kv=1 << 10, row=1 << 20, cap=1 << 30, batch=65535)),  # sizes beyond 64 bits
])
def test_caches_that_share_bytes_are_refused(caches, size, kw):
    assert keep([A + c for c in caches], **kw) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("order", [[0, 1, 2], [2, 0, 1], [1]])
@pytest.mark.parametrize("paged", [False, True])
def test_neighbours_are_taken(order, paged):
    """Caches that touch each other, in any order; and one cache twice, refused through Python too."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(3, 3, N_KV, PAGE, 64, device="cuda").bfloat16()     # three caches of one allocation
    want = x.clone()
    table = i32([[2], [0]]) if paged else None
    pos, path, n = i32([7, 120]), i32([[0, 2, 3, -1], [1, 3, 4, 7]]), i32([3, 4])
    caches = list(x) if paged else [c[:2] for c in x]
    path = torch.cat([path, torch.full_like(path, -1)], 1)
    for c in order:
        for b, (p, keep_b) in enumerate(((7, [0, 2, 3]), (120, [1, 3, 4, 7]))):
            at = [2, 0][b] if paged else b
            want[c, at, :, p:p + len(keep_b)] = x[c, at][:, [p + m for m in keep_b]]
    g.gemma_kv_keep([caches[c] for c in order], pos, path, n, block_table=table)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    with pytest.raises(binding.GemmaError):
        g.gemma_kv_keep([caches[0], caches[1], caches[0]], pos, path, n, block_table=table)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
