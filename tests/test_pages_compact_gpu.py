"""Compaction looks at every entry of the table, whether or not a page has to move."""
import pytest
import torch

import mixed_sliding_global_gb300 as g

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("moves", [False, True])
@pytest.mark.parametrize("entry,bit", [(9, g.GEMMA_DEVERR_PAGE), (1 << 30, g.GEMMA_DEVERR_PAGE),
                                       (2 ** 31 - 1, g.GEMMA_DEVERR_PAGE),
                                       (8, g.GEMMA_DEVERR_PAGE),      # nobody holds page 8
                                       (-1, 0), (-2 ** 31, 0), (1, 0)])
def test_every_entry_is_looked_at(entry, bit, moves):
    """Pages 0 to 4 are in use; with moves one of them lies at 6 before the call."""
    x = torch.randint(0, 100, (9, 2, 128, 8), device="cuda").bfloat16()
    before = x.clone()
    table, refs = i32([[0, 1, 6 if moves else 2], [3, 4, entry]]), i32([1, 1, 0, 1, 1, 0, 0, 0, 0])
    refs[6 if moves else 2] = 1
    if entry == 1:
        refs[1] = 2
    want = refs.tolist()
    want[2], want[6] = 1, 0
    err, used = i32([0]), i32([-1])
    ws = torch.full((g.gemma_pages_workspace_size(9),), 255, dtype=torch.uint8, device="cuda")
    g.gemma_pages_compact([x], table, refs, n_used=used, workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == bit
    assert table.tolist() == [[0, 1, 2], [3, 4, entry]]
    assert refs.tolist() == want and used.item() == 5
    if moves:
        before[2] = before[6]
    assert torch.equal(x, before)


def test_a_pool_without_pages_in_use():
    """Nothing is in use, and an entry names a page all the same."""
    x = torch.zeros(3, 1, 128, 8, dtype=torch.bfloat16, device="cuda")
    table, refs, err = i32([[2, -1]]), i32([0, 0, 0]), i32([0])
    ws = torch.full((g.gemma_pages_workspace_size(3),), 255, dtype=torch.uint8, device="cuda")
    g.gemma_pages_compact([x], table, refs, workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == g.GEMMA_DEVERR_PAGE and table.tolist() == [[2, -1]]
