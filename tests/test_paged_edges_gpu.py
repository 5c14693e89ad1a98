"""Paged attention of many rows over a table that names only the pages in use (entries behind the last
key, and of pages wholly below the window, are -1, as the page bookkeeping leaves them): no error, and
the definition's result, as over a plain cache."""
import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("kind,window", [(g.GEMMA_SLIDING, 100), (g.GEMMA_SLIDING, 64), (g.GEMMA_GLOBAL, 0)])
@pytest.mark.parametrize("d,n_q,n_kv", [(64, 4, 2), (128, 8, 4), (256, 8, 2), (512, 4, 1)])
def test_tables_of_the_pages_in_use(d, n_q, n_kv, kind, window, page):
    B, n_new, blocks = 8, 40, 512 // page
    lens = [40, 128, 129, 170, 256, 300, 320, 512]   # the last fills the table
    gen = torch.Generator().manual_seed(d)
    k = torch.randn(B, n_kv, 512, d, generator=gen).bfloat16().cuda()
    v = torch.randn(B, n_kv, 512, d, generator=gen).bfloat16().cuda()
    q = torch.randn(B, n_new, n_q, d, generator=gen).bfloat16().cuda()
    order = torch.randperm(B * blocks, generator=gen).reshape(B, blocks)
    table = torch.full((B, blocks), -1, dtype=torch.int32)
    pool = [torch.full((B * blocks, n_kv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
            for _ in range(2)]
    for b, n in enumerate(lens):
        first = max(0, n - n_new - window + 1) if kind == g.GEMMA_SLIDING else 0
        for j in range(first // page, (n - 1) // page + 1):
            table[b, j] = order[b, j]
            rows = slice(0, min(page, n - j * page))
            for x, c in zip(pool, (k, v)):
                x[order[b, j], :, rows] = c[b, :, j * page:j * page + rows.stop]
    table = table.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(kind=kind, window=window, n_kv=n_kv, k_eq_v=False, scale=d ** -0.5, device_error=err)
    outs = []
    for paged in (False, True):
        size = g.gemma_attn_workspace_size_paged if paged else g.gemma_attn_workspace_size
        n = size(B, kind, window, n_q, n_kv, d, 512, n_new)
        ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, float("nan"))
        if paged:
            g.gemma_attn_paged(out, q, [pool[0]], [pool[1]], [0], 0, seq, table, 512, workspace=ws, **kw)
        else:
            g.gemma_attn_prefill(out, q, [k], [v], [0], 0, seq, 512, workspace=ws, **kw)
        outs.append(out)
    torch.cuda.synchronize()
    assert err.item() == 0
    # (the two place their key tiles differently, so that P and the sums round differently)
    for b, n in enumerate(lens):
        see = tree_ref.keys_of([i - 1 for i in range(n_new)], n_new, n - n_new, kind, window)
        ref, mass, size = tree_ref.attention(q[b], k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1),
                                             see, d ** -0.5)
        # half a step of the output and of P (in the sum and its normaliser), fp32 sums of d products
        # in matrix instructions of 16 and of up to 512 keys, exponentials 2^-21
        rel = 2 * (d / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -20 + 96 * 2.0 ** -23
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel) * (mass + ref.abs())
        for out in outs:
            assert ((out[b].double() - ref).abs() <= bound).all()
