"""Soft-capped tree attention where a row's scores lie far apart: a key far below the cap's zero beside
scores that are small against the cap, and rows of which every score is far below zero."""
import math

import pytest
import torch

import mixed_sliding_global_gb300 as g
import tree_ref
from test_tree_gpu import i32, random_tree
from test_tree_values_gpu import WAYS

pytestmark = pytest.mark.gpu


def problem(n_q, n_kv, d, nodes, lens, dtype, softcap, low, seed):
    """q and K whose first column adds -0.6 of the cap to the score of the keys `low` (a function of the
    positions), and nothing to the others."""
    gen = torch.Generator().manual_seed(seed)
    B, top = len(lens), max(lens)
    q = torch.randn(B, nodes, n_q, d, generator=gen)
    k, v = (torch.randn(B, n_kv, top, d, generator=gen) for _ in range(2))
    q[..., 0] = 64.0
    k[..., 0] = torch.where(low(torch.arange(top)), -0.6 * softcap * math.sqrt(d) / 64, 0.0)
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    return q, k, v, [random_tree(gen, nodes, [0.5, 1.0, 2.0][b % 3]) for b in range(B)]


def run(q, k, v, lens, parents, softcap):
    B, nodes, n_q, d = q.shape
    out, err = torch.full_like(q, float("nan")), i32([0])
    n = g.gemma_attn_workspace_size_tree(B, g.GEMMA_GLOBAL, 0, n_q, k.shape[1], d, max(lens), nodes)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    g.gemma_attn_tree(out, q, [k], [v], [0], 0, i32(lens), i32(parents), max(lens), kind=g.GEMMA_GLOBAL,
                      window=0, n_kv=k.shape[1], k_eq_v=False, scale=d ** -0.5, softcap=softcap,
                      workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out


def bound(ref, mass, size, d, n_keys, dtype, softcap=1e9):
    """As in test_tree_gpu.Problem, `size` the largest scale * sum_i |q_i k_i| of the keys that carry
    weight, and for the cap 2^-19 of it (test_tree_values_gpu.Capped), twice: the normaliser. A cap's
    error is one of the score it is taken of, or, up to a cap of 64, 2^-20 of the cap."""
    if softcap <= 64:
        size = size + softcap / 2
    if dtype == torch.float32:
        rel = 2 * (d / 32 + 8) * 2.0 ** -24 * size + 2.0 ** -20 + n_keys * 2.0 ** -23
        return (rel + 2 * 2.0 ** -19 * size) * (mass + ref.abs()) + 1e-12
    rel = 2 * (d / 16 + 16) * 2.0 ** -23 * size + 2.0 ** -20 + (n_keys / 16 + 64) * 2.0 ** -23
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + rel + 2 * 2.0 ** -19 * size) * (mass + ref.abs()) + 1e-12


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens,dtype", WAYS)
@pytest.mark.parametrize("softcap", [64.0, 1e4, 1e6, 1e20])
def test_keys_far_below_the_others(n_q, n_kv, d, nodes, lens, dtype, softcap):
    """Every 16th key lies 0.5 of the cap below the rest: hardly any weight (some e^-30 of the
    other keys' at most), and no effect on the scores of the rest, which are some 2^-6 to 2^-66 of the cap."""
    low = lambda j: j % 16 == 5  # noqa: E731
    q, k, v, parents = problem(n_q, n_kv, d, nodes, lens, dtype, softcap, low, d)
    out = run(q, k, v, lens, parents, softcap)
    for b, n in enumerate(lens):
        see = tree_ref.keys_of(parents[b], nodes, n - nodes, tree_ref.GLOBAL, 0)
        kb, vb = k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1)
        ref, mass, _ = tree_ref.attention(q[b], kb, vb, see, d ** -0.5, softcap)
        carry = see & ~low(torch.arange(n))
        assert carry.any(1).all()
        size = tree_ref.attention(q[b], torch.where(low(torch.arange(n, device="cuda"))[:, None, None], 0, kb),
                                  vb, see, d ** -0.5)[2]
        e = (out[b].double() - ref).abs()
        assert (e <= bound(ref, mass, size, d, n, dtype, softcap)).all()


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens,dtype", WAYS)
@pytest.mark.parametrize("softcap", [20.0, 400.0])
def test_all_keys_far_below_zero(n_q, n_kv, d, nodes, lens, dtype, softcap):
    """Every score is about -0.6 of the cap: the error is one of the scores' size."""
    q, k, v, parents = problem(n_q, n_kv, d, nodes, lens, dtype, softcap, lambda j: j >= 0, d)
    out = run(q, k, v, lens, parents, softcap)
    for b, n in enumerate(lens):
        see = tree_ref.keys_of(parents[b], nodes, n - nodes, tree_ref.GLOBAL, 0)
        kb, vb = k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1)
        ref, mass, size = tree_ref.attention(q[b], kb, vb, see, d ** -0.5, softcap)
        e = (out[b].double() - ref).abs()
        assert (e <= bound(ref, mass, size, d, n, dtype)).all()


@pytest.mark.parametrize("n_q,n_kv,d,nodes,lens,dtype", WAYS)
def test_a_cap_of_nothing(n_q, n_kv, d, nodes, lens, dtype):
    """A cap far below the smallest score makes every score the cap or its negative, so that all keys that a
    node attends weigh alike; scores of exactly zero and keys of other branches do not turn into NaN."""
    q, k, v, parents = problem(n_q, n_kv, d, nodes, lens, dtype, 1.0, lambda j: j < 0, d)
    k[:, :, 3] = 0.0
    out = run(q, k, v, lens, parents, 1e-40)
    for b, n in enumerate(lens):
        see = tree_ref.keys_of(parents[b], nodes, n - nodes, tree_ref.GLOBAL, 0)
        kb, vb = k[b, :, :n].transpose(0, 1), v[b, :, :n].transpose(0, 1)
        ref, mass, _ = tree_ref.attention(0 * q[b], kb, vb, see, d ** -0.5)
        e = (out[b].double() - ref).abs()
        assert (e <= bound(ref, mass, torch.zeros_like(mass[..., :1]), d, n, dtype)).all()
