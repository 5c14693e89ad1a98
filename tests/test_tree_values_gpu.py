"""Attention of a drafted tree with values at the edges: soft-caps far above and far below the scores,
and NaN keys that nodes do attend."""
import pytest
import torch

from test_tree_gpu import Problem

pytestmark = pytest.mark.gpu

# every way a step can run: n_q, n_kv, head_dim, nodes, lengths, dtype
WAYS = [(8, 8, 64, 16, [2600] * 5, torch.bfloat16),       # a warp's matrix instructions, many keys
        (8, 8, 128, 5, [4000, 3000, 3900], torch.bfloat16),
        (4, 2, 64, 9, [900], torch.bfloat16),             # a cluster for each unit
        (8, 2, 256, 40, [1500, 90, 700], torch.bfloat16), # pairs
        (4, 2, 128, 30, [1700] * 9, torch.bfloat16),      # one SM, equal shares
        (16, 1, 512, 12, [1500, 90], torch.bfloat16),
        (2, 2, 512, 12, [1500, 90], torch.bfloat16),
        (4, 2, 128, 9, [300, 40], torch.float32)]


class Capped(Problem):
    def tolerance(self, ref, mass, size, d, n_keys):
        """The bound without a cap, and what the cap adds to a score: tanh's series is off by 0.0036 x^12
        < 2^-20 of itself up to |x| = 1/2; rows with larger scores take 1 - 2 / (1 + e^2x), off by r (an
        exponential of 2^-22.5, a reciprocal of 2^-23 and three roundings of 2^-24) = 2^-21.2 twice, or
        2^-20.2 of the cap at most, where the row's largest |x| is above 1/2 and so size above cap / 2:
        2^-19.2 of size. 2^-19 of size covers both (twice: the normaliser)."""
        cap, self.softcap = self.softcap, 0.0
        bound = super().tolerance(ref, mass, size, d, n_keys)
        self.softcap = cap
        return bound + 2 * 2.0 ** -19 * size * (mass + ref.abs())


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens,dtype", WAYS)
@pytest.mark.parametrize("softcap", [1e-3, 3.0, 50.0, 1e5, 1e30])
def test_soft_caps_of_all_sizes(n_q, n_kv, d, nodes, lens, dtype, softcap):
    p = Capped(lens, [nodes] * len(lens), nodes, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, softcap=softcap,
               q_gain=4.0, seed=d)
    p.check(p.run())
    assert p.err == 0


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens,dtype", WAYS)
@pytest.mark.parametrize("where", [slice(0, 600), slice(65, 66), slice(0, 4000)])
def test_nan_keys_reach_the_nodes_that_attend_them(n_q, n_kv, d, nodes, lens, dtype, where):
    """Also where all keys of a part are NaN and its maximum stays at minus infinity."""
    p = Problem(lens + [nodes], [nodes] * (len(lens) + 1), nodes, n_q=n_q, n_kv=n_kv, d=d, dtype=dtype, seed=3)
    p.k[:len(lens), :, where.start:where.stop] = float("nan")
    out = p.run()
    assert p.err == 0
    for b, n in enumerate(lens):
        if where.start < n - nodes:      # (else the tree's own keys, attended by some)
            assert torch.isnan(out[b]).all()
    err = (out[-1].double() - p.ref[-1]).abs()
    assert (err <= p.bound[-1]).all()
