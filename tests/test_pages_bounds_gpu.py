"""Pages given back with both bounds: exactly those that hold no position of the interval, also where it
is empty or its ends lie in one page."""
import pytest
import torch

import mixed_sliding_global_gb300 as g

pytestmark = pytest.mark.gpu

PAGE, PER = 128, 4
BOUNDS = [(50, 50), (100, 40), (0, 0), (128, 128), (127, 127), (130, 130), (200, 129),   # none
          (500, 3), (512, 512), (2 ** 31 - 1, 2 ** 31 - 1), (-5, -5), (-1, 0), (384, 0), (600, 700),
          (50, 51), (127, 128), (127, 129), (128, 129), (0, 1), (511, 512), (3, 500),    # some
          (-9, 1), (256, 384), (255, 385), (300, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1)]


def kept(page, lo, hi):
    """By the definition, a position at a time."""
    return any(lo <= j < hi for j in range(page * PAGE, (page + 1) * PAGE))


@pytest.mark.parametrize("bounds", [BOUNDS, BOUNDS[:1], [(50, 50), (0, 512)]])
def test_pages_without_a_position_of_the_interval(bounds):
    B = len(bounds)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(B * PER, dtype=torch.int32, device="cuda").view(B, PER)
    refs, err = torch.ones(B * PER + 3, dtype=torch.int32, device="cuda"), i32([0])
    g.gemma_pages_free(table, refs, page_size=PAGE, keep_from=i32([lo for lo, _ in bounds]),
                       keep_to=i32([hi for _, hi in bounds]), device_error=err)
    torch.cuda.synchronize()
    want = [[b * PER + k if kept(k, lo, hi) else -1 for k in range(PER)] for b, (lo, hi) in enumerate(bounds)]
    assert table.tolist() == want
    assert refs.tolist() == [int(e >= 0) for row in want for e in row] + [1, 1, 1]
    assert err.item() == 0


@pytest.mark.parametrize("bounds", BOUNDS)
def test_one_bound_alone(bounds):
    """Without the other bound the interval is open on its side."""
    lo, hi = bounds
    for kw, a, b in (("keep_from", lo, 2 ** 40), ("keep_to", -2 ** 40, hi)):
        table = torch.arange(PER, dtype=torch.int32, device="cuda").view(1, PER)
        refs = torch.ones(PER, dtype=torch.int32, device="cuda")
        g.gemma_pages_free(table, refs, page_size=PAGE,
                           **{kw: torch.tensor([lo if kw == "keep_from" else hi], dtype=torch.int32,
                                               device="cuda")})
        torch.cuda.synchronize()
        want = [k if kept(k, a, b) else -1 for k in range(PER)]
        assert table.tolist() == [want]
        assert refs.tolist() == [int(e >= 0) for e in want]
