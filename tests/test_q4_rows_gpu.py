"""GPU: 4-bit attention on both sides of the rows per KV head that decide between the codes themselves and
a dequantised copy (64; 128 at head_dim 128, 192 at 512), each with its own bound (test_q4_gpu.py):
2^-8 |out| and (2^-10 + 2^-13) A straight over the codes, 2^-7 A (2^-6 more at head_dim 512) over the
copy."""
import pytest

import mixed_sliding_global_gb300 as g
import q4_ref as R
from test_q4_gpu import GLOBAL, SLIDING, Cache, fill, rows

pytestmark = pytest.mark.gpu

LIMIT = {64: 64, 128: 128, 256: 64, 512: 192}


@pytest.mark.parametrize("kind,window", [(GLOBAL, 0), (SLIDING, 150)])
@pytest.mark.parametrize("d,n_q,n,k_eq_v", [
    (64, 16, 4, False), (64, 16, 5, False), (128, 2, 64, False), (128, 2, 65, True),
    (128, 16, 7, True), (256, 8, 8, False), (256, 8, 9, False), (512, 16, 5, False),
    (512, 16, 12, True), (512, 16, 13, True), (512, 8, 24, False), (512, 1, 192, True),
    (512, 1, 193, True)])
def test_both_sides(d, n_q, n, k_eq_v, kind, window):
    lens = [n, 430, 257]
    c = Cache(3, 1, 448, d, k_eq_v)
    fill(c, lens, kind)
    q = rows((3, n, n_q, d), 31)
    size = g.gemma_attn_workspace_size_q4(3, kind, window, n_q, 1, d, 430, n, k_eq_v=k_eq_v)
    direct = n * n_q <= LIMIT[d]
    reach = 430 if kind == GLOBAL else min(430, window + n - 1)
    assert direct == (size < 3 * reach * d * 2)      # (a copy of K alone is that large)
    got = c.attend(q, lens, kind, window)
    assert c.err.item() == 0
    k, v = c.values()
    out, mass = R.attention(q, k, v, lens, kind, window, d ** -0.5)
    rel = 2.0 ** -10 + 2.0 ** -13 if direct else 2.0 ** -7 + (2.0 ** -6 if d == 512 else 0)
    err = (got.double().cpu() - out).abs() / (2.0 ** -8 * out.abs() + rel * mass + 1e-6)
    assert err.max() <= 1, err.max().item()
