"""GPU: the accuracy that sampling promises, at the boundaries between tokens.

Rows whose many small weights are equal, so that errors of the same kind add up; uniforms and top_p are
the fp32 numbers next to the boundaries of the running sums. A boundary is where the definition in 64
bits (weights by exp, sums by fsum) puts it; a number closer to it than 2^-33 of the sum is left out:
sums are promised to about 2^-35, a quarter of that, and the weights' own 2^-40 are nothing beside
it."""
import math

import numpy as np
import pytest
import torch

import mixed_sliding_global_gb300 as g

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -33


def sums(x, t, softcap, m, k):
    """Order of a row of fp32 or bf16 logits, the running weights of its first m tokens and the sum
    of all (of the first k with k), in 64 bits."""
    x = x.double().numpy()
    order = np.argsort(-x, kind="stable")[:k or None]
    z = x[order]
    if softcap:
        z = softcap * np.tanh(z / softcap)
    w = np.exp((z - z[0]) / t)
    run = np.array([math.fsum(w[:i + 1]) for i in range(m)])
    return order, run, math.fsum(w)


def near(run, total, n):
    """The n fp32 numbers closest to a boundary run[i] / total but more than MARGIN from all of them, and
    how many of the running sums each one times the total is short of (the place it draws)."""
    r = run / total
    near_r = r.astype(np.float32)
    c = np.unique(np.concatenate([near_r, np.nextafter(near_r, np.float32(0)),
                                  np.nextafter(near_r, np.float32(1))]))
    c = c[(c >= 0) & (c < 1)]
    d = np.abs(c.astype(np.float64)[:, None] - r[None]).min(1)
    c, d = c[d > MARGIN], d[d > MARGIN]
    c = c[np.argsort(d, kind="stable")[:n]]
    place = np.searchsorted(r, c.astype(np.float64), side="right")   # first i with run > u total
    return c, place


def draw(x, u, t=None, p=None, softcap=0.0, k=0):
    B, V = x.shape
    out = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = lambda v: None if v is None else torch.as_tensor(v, dtype=torch.float32).expand(B).contiguous().cuda()  # noqa: E731
    ws = torch.empty(max(16, g.gemma_logit_sample_workspace_size(B, V, x.dtype)), dtype=torch.uint8,
                     device="cuda")
    g.gemma_logit_sample(x, out, f(u), temperature=f(t), top_p=f(p), softcap=softcap, workspace=ws,
                         top_k=torch.full((B,), k, dtype=torch.int32, device="cuda") if k else None,
                         device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out.cpu().numpy()


def check(x, B, t=1.0, softcap=0.0, m=200, k=0):
    """Uniforms at the boundaries of the first m tokens, then top_p there with the last kept drawn."""
    t = float(np.float32(t))
    order, run, total = sums(x, t, softcap, m + 1, k)
    xs = x.cuda().expand(B, -1).contiguous()
    u, place = near(run[:m], total, B)
    assert len(u) == B
    got = draw(xs, u, t, None, softcap, k)
    assert (got == order[place]).all(), ((got != order[place]).sum(), B)
    # keep the shortest prefix with run >= p total; its last token weighs more than 2^-24 of it
    last = run[place] - np.where(place > 0, run[place - 1], 0)
    ok = last > 2.0 ** -22 * total
    assert ok.sum() > B // 2
    got = draw(xs, np.full(B, 1 - 2.0 ** -24), t, u, softcap, k)
    assert (got == order[place])[ok].all(), ((got != order[place])[ok].sum(), ok.sum())


def row(V, bulk, seed, heads=1200):
    """One leading logit at 0, `heads` distinct ones between -14 and -10 and the rest at `bulk`."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.full((V,), bulk)
    at = torch.randperm(V, generator=gen)[:heads + 1]
    x[at[0]] = 0.0
    x[at[1:]] = -10 - 4 * torch.rand(heads, generator=gen)
    return x


def half_unit(bulk):
    """The fp32 number near `bulk` whose weight lies nearest to the middle of two multiples of 2^-43."""
    c = np.float32(bulk) + np.arange(4000, dtype=np.float32) * np.float32(2.0 ** -19)
    f = np.exp(c.astype(np.float64)) * 2.0 ** 43 % 1
    return float(c[np.argmin(np.abs(f - 0.499))])


@pytest.mark.parametrize("V,B", [(20000, 40), (70001, 8), (262144, 8), (262144, 64), (1048560, 16)])
@pytest.mark.parametrize("bulk", [-16.9, -17.5, -19.0, -22.5, -25.0])
def test_equal_logits_behind_distinct_ones(V, B, bulk):
    """fp32 without top_k or cap: the sum of all weights next to a short list of the largest."""
    check(row(V, half_unit(bulk), int(V - bulk)), B)


@pytest.mark.parametrize("k", [0, 3000])
@pytest.mark.parametrize("V,B", [(20000, 40), (262144, 8), (262144, 64), (1048560, 16)])
@pytest.mark.parametrize("bulk", [-16.9, -12.0])
def test_equal_logits_within_one_upper_half(V, B, bulk, k):
    """fp32 by histogram (a top_k beyond the lists', of the whole row or of a part that ends among
    the equal ones or before) at a temperature so small that most of the row shares its upper half:
    the sum of one bin holds weights far apart."""
    t = 2.0 ** -11
    x = row(V, half_unit(bulk), int(V - bulk) + 7, heads=5000) * t + 2.0146
    check(x, B, t=t, k=k or V)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("softcap", [50.0, 1e5, 1e7, 1e12, 3e38])
def test_large_caps(softcap, dtype):
    """Caps far above the logits, to which z is x and a little less: with 2^-47 of the cap, or 2^-40 of
    z if that is less, a weight is good to 2^-42 and better here."""
    gen = torch.Generator().manual_seed(9)
    x = (torch.randn(30000, generator=gen) * 3).to(dtype)
    if dtype == torch.bfloat16:
        x = torch.unique(x)[-900:]      # (boundaries between single tokens)
    softcap = float(np.float32(softcap))
    check(x, 64, softcap=softcap, m=300)
    check(x, 64, softcap=softcap, m=300, k=250)


def test_logits_as_large_as_the_cap():
    """Logits, caps and temperatures of 1e38."""
    x = torch.tensor([3e38, 2.9e38, 1e38, 0.0, -1e38, -3.3e38])
    for c in (3e38, 1e38):
        c = float(np.float32(c))
        check(x, 4, t=8e37, softcap=c, m=5)
        check(x.bfloat16(), 4, t=8e37, softcap=c, m=5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_temperatures(dtype):
    """Temperatures of 1e20 to 3e38 with logits as large, up to the type's lowest number: their
    differences leave fp32's range, the weights are ordinary."""
    low = torch.finfo(dtype).min
    for t in (1e20, 1e31, 3e38):
        t = float(np.float32(t))
        x = torch.tensor([0.9, 0.8, 0.1, 0.0, -0.3, -0.7]).double() * t
        x = torch.cat([x.to(dtype), torch.tensor([low], dtype=dtype)])
        for k in (0, 6, 7, 300):
            check(x, 6, t=t, m=6, k=k)
