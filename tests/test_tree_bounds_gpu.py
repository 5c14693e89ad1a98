"""Tree attention whose max_seq_len lies far above the lengths, as a captured step of a server has it: how
the work is cut goes by the bound or by the lengths, the results by the lengths."""
import pytest
import torch

from test_tree_gpu import Problem
from tree_ref import GLOBAL, RING, SLIDING

pytestmark = pytest.mark.gpu

TOP = 131072


@pytest.mark.parametrize("kind,window", [(GLOBAL, 0), (SLIDING, 300), (RING, 300)])
@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens,dtype", [
    (8, 8, 64, 16, [2600, 900], torch.bfloat16), (8, 8, 128, 5, [1000, 30, 3900], torch.bfloat16),
    (4, 2, 64, 9, [900], torch.bfloat16), (8, 2, 256, 8, [900, 64], torch.bfloat16),
    (8, 2, 256, 40, [1500, 90, 700], torch.bfloat16), (4, 2, 128, 30, [500] * 90, torch.bfloat16),
    (16, 1, 512, 12, [1500, 90], torch.bfloat16), (16, 1, 512, 2, [8200], torch.bfloat16),
    (2, 2, 512, 12, [1500, 90], torch.bfloat16), (2, 2, 512, 30, [129], torch.bfloat16),
    (4, 2, 128, 9, [300, 40], torch.float32)])
def test_a_bound_far_above_the_lengths(n_q, n_kv, d, nodes, lens, dtype, kind, window):
    lens = lens + [nodes, 0]
    reals = [nodes] * (len(lens) - 2) + [nodes - 1, 0]
    p = Problem(lens, reals, nodes, kind=kind, window=window, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype,
                page=0 if kind == RING else 128, seed=d + nodes)
    p.msl = TOP
    if kind != RING:       # the pages in use, and a table for the whole bound
        for b, n in enumerate(lens):
            p.table[b, -(-n // 128):] = -1
        rest = torch.full((len(lens), TOP // 128 - p.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        p.table = torch.cat([p.table, rest], 1).contiguous()
    p.check(p.run())
    assert p.err == 0
