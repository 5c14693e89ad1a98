"""GPU: sampling against its 64-bit definition (tests/sample_ref.py). Tokens are compared exactly: both
sides cut and draw at real numbers, the kernel with weights good to about 2^-40 and sums to 2^-35, so
that a row falls on the other side of a boundary about once in 2^30 rows; the seeded rows here are a
few thousand."""
import numpy as np
import pytest
import torch

import mixed_sliding_global_gb300 as g
import synth
from sample_ref import sample_row

pytestmark = pytest.mark.gpu


def run(x, u, t=None, k=None, p=None, m=None, softcap=0.0, ws=None, stream=None):
    B, V = x.shape
    x = x.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    f = lambda v, dt: None if v is None else torch.as_tensor(v, dtype=dt).expand(B).contiguous().cuda()  # noqa: E731
    n = g.gemma_logit_sample_workspace_size(B, V, x.dtype)
    if ws is None:
        ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    g.gemma_logit_sample(x, out, f(u, torch.float32), temperature=f(t, torch.float32),
                         top_k=f(k, torch.int32), top_p=f(p, torch.float32),
                         min_p=f(m, torch.float32), softcap=softcap, workspace=ws,
                         device_error=err, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), err.item()


def want(x, u, t=1.0, k=0, p=1.0, m=0.0, softcap=0.0):
    B = x.shape[0]
    f32 = lambda v: np.broadcast_to(np.asarray(v, np.float32).astype(np.float64), (B,))  # noqa: E731
    u, t, p, m = f32(u), f32(t), f32(p), f32(m)
    k = np.broadcast_to(np.asarray(k), (B,))
    xs = x.double().numpy()
    return torch.tensor([sample_row(xs[b], float(u[b]), float(t[b]), int(k[b]), float(p[b]),
                                    float(m[b]), softcap) for b in range(B)], dtype=torch.int32)


def check(x, u, **kw):
    got, err = run(x, u, **kw)
    ref = want(x, u, **kw)
    assert torch.equal(got, ref), (got.tolist()[:16], ref.tolist()[:16])
    assert err == 0


def uniforms(B, seed):
    u = torch.rand(B, generator=torch.Generator().manual_seed(seed))
    u[0] = 0.0
    if B > 1:
        u[1] = 1 - 2.0 ** -24
    return u


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
@pytest.mark.parametrize("B,V", [(1, 1), (2, 2), (3, 7), (4, 31), (5, 1000), (3, 4096), (3, 4097),
                                 (2, 70001), (1, 262144)])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_shapes(dtype, B, V, softcap):
    x = synth.logits(B, V, seed=B * 5 + V, dtype=dtype)
    for i, kw in enumerate([dict(), dict(k=20), dict(p=0.9), dict(m=0.02), dict(t=0.3, k=50, p=0.8),
                            dict(t=2.0, k=1000, p=0.95, m=0.01), dict(t=1.3, p=0.3, m=0.2)]):
        check(x, uniforms(B, 100 * i + V), softcap=softcap, **kw)


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_many_draws(dtype):
    """Each request of a batch with its own filters; the uniforms walk over [0, 1)."""
    B, V = 192, 5000
    x = synth.logits(1, V, seed=3, dtype=dtype).expand(B, V).contiguous()
    gen = torch.Generator().manual_seed(4)
    pick = lambda vals: torch.tensor(vals)[torch.randint(0, len(vals), (B,), generator=gen)]  # noqa: E731
    check(x, torch.arange(B) / B, t=pick([0.5, 1.0, 1.7]), k=pick([0, 1, 7, 300]),
          p=pick([1.0, 0.9, 0.5, 0.01]), m=pick([0.0, 0.1, 0.5]), softcap=30.0)


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_equal_logits(dtype):
    """Every logit equal: the draw is the index u V, the cuts count tokens, over all slices."""
    for V in (5, 4096, 50000, 262144):
        x = torch.full((4, V), 2.5).to(torch.bfloat16 if dtype == synth.BF16 else torch.float32)
        u = torch.tensor([0.0, 0.25, 0.5, 1 - 2.0 ** -24])
        check(x, u)
        check(x, u, p=0.5)
        check(x, u, k=3)
        check(x, u, m=1.0)
        got, _ = run(x, u)
        assert got.tolist() == [int(v * V) if v < 0.9 else V - 1 for v in u.tolist()]


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_ties_at_the_cuts(dtype):
    """Many tokens share the value a cut falls into: the lowest indices of it are kept."""
    V = 60000
    gen = torch.Generator().manual_seed(9)
    x = torch.randint(-3, 4, (6, V), generator=gen).float()
    x = x.bfloat16() if dtype == synth.BF16 else x
    u = uniforms(6, 5)
    n3 = int((x[0].float() == 3).sum())
    for kw in (dict(k=n3 - 5), dict(k=n3), dict(k=n3 + 1), dict(k=n3 + 4000), dict(p=0.5), dict(p=0.7),
               dict(k=n3 + 4000, p=0.9), dict(m=0.2), dict(p=0.99, m=0.05)):
        check(x, u, **kw)


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_masked_rows(dtype):
    """-inf and NaN are never drawn; the type's lowest number is a candidate like any other; rows
    of +inf, with and without a cap; a row without candidates."""
    dt = torch.bfloat16 if dtype == synth.BF16 else torch.float32
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dt).min
    x = torch.full((8, 9000), -inf)
    x[0, 777] = -5.0
    x[1, [3, 8999]] = torch.tensor([1.0, 1.0])
    x[2] = nan
    x[2, 4000] = 0.0
    x[3] = low
    x[3, [5, 6]] = torch.tensor([2.0, 3.0])
    x[4] = low
    x[5, :] = 1.0
    x[5, [100, 8000]] = inf
    x[6, :] = -0.0
    x[6, ::2] = 0.0
    x = x.to(dt)
    u = torch.tensor([0.9, 0.6, 0.3, 0.99, 0.5, 0.7, 0.77, 0.1])
    for cap in (0.0, 30.0):
        for kw in (dict(), dict(k=2), dict(p=0.6), dict(t=0.01), dict(m=0.5)):
            got, err = run(x, u, softcap=cap, **kw)
            assert torch.equal(got, want(x, u, softcap=cap, **kw)), (cap, kw)
            assert got[7].item() == -1 and err == g.GEMMA_DEVERR_SAMPLE
    got, _ = run(x, u)
    assert got.tolist()[:3] == [777, 8999, 4000] and got[5].item() == 8000


def test_bad_parameters():
    x = synth.logits(9, 100, seed=1)
    nan, inf = float("nan"), float("inf")
    t = torch.tensor([1.0, -1.0, nan, inf, 1, 1, 1, 1, 0.0])
    p = torch.tensor([0.9, 1, 1, 1, nan, 1, 1, 1, 1])
    m = torch.tensor([0.1, 0, 0, 0, 0, nan, 0, 0, 0])
    u = torch.tensor([0.5, 0.5, 0.5, 0.5, 0.5, 0.5, 1.0, -0.1, 0.9])
    got, err = run(x, u, t=t, p=p, m=m)
    assert err == g.GEMMA_DEVERR_SAMPLE
    assert got.tolist()[1:8] == [-1] * 7
    assert torch.equal(got, want(x, u, t=t, p=p, m=m))
    assert got[8].item() == int(x[8].float().argmax())


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_extreme_temperatures(dtype):
    x = synth.logits(5, 20000, seed=8, dtype=dtype)
    u = uniforms(5, 6)
    for t in (1e-30, 1e-6, 0.01, 50.0, 1e6, 3e38):
        check(x, u, t=t)
        check(x, u, t=t, p=0.9)
        check(x, u, t=t, softcap=30.0, m=0.5)


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_top_values(dtype):
    """top_p 0 and below, top_k beyond the row, min_p above 1."""
    x = synth.logits(4, 3000, seed=12, dtype=dtype)
    u = uniforms(4, 7)
    for kw in (dict(p=0.0), dict(p=-1.0), dict(k=5000), dict(k=3000), dict(k=2999), dict(k=-1),
               dict(m=2.0), dict(m=1.0), dict(p=1e-9), dict(p=0.9999999)):
        check(x, u, **kw)


def test_full_size_batch():
    B, V = 64, synth.VOCAB
    x = synth.logits(B, V, seed=21)
    gen = torch.Generator().manual_seed(22)
    pick = lambda vals: torch.tensor(vals)[torch.randint(0, len(vals), (B,), generator=gen)]  # noqa: E731
    check(x, uniforms(B, 23), t=pick([0.6, 1.0, 1.2]), k=pick([0, 40, 200]),
          p=pick([1.0, 0.95, 0.5]), m=pick([0.0, 0.05]), softcap=30.0)


def test_largest_vocabulary():
    V = 1048560
    x = synth.logits(1, V, seed=2)
    check(x, torch.tensor([0.7]), p=0.9)
    with pytest.raises(ValueError):
        g.gemma_logit_sample_workspace_size(1, V + 1, torch.bfloat16)


def test_agrees_with_the_greedy_step():
    """temperature 0 and top_k 1 give gemma_logit_softcap_argmax's index."""
    x = synth.logits(16, 50000, seed=30)
    idx = torch.empty(16, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(16, g.gemma_logit_workspace_size(16, 50000)), dtype=torch.uint8,
                     device="cuda")
    g.gemma_logit_softcap_argmax(x.cuda(), 30.0, idx, None, ws)
    torch.cuda.synchronize()
    for kw in (dict(t=0.0), dict(k=1)):
        got, _ = run(x, uniforms(16, 31), softcap=30.0, **kw)
        assert torch.equal(got, idx.cpu())


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_captured_step(dtype):
    """A captured call replayed with new logits and uniforms on another stream, its workspace full
    of other values, gives what the definition gives."""
    B, V = 3, 30000
    x = synth.logits(B, V, seed=40, dtype=dtype).cuda()
    u = uniforms(B, 41).cuda()
    p = torch.full((B,), 0.9, device="cuda")
    out = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(16, g.gemma_logit_sample_workspace_size(B, V, x.dtype)),
                     dtype=torch.uint8, device="cuda")
    call = lambda: g.gemma_logit_sample(x, out, u, top_p=p, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call()
    for seed in (50, 60):
        x.copy_(synth.logits(B, V, seed=seed, dtype=dtype))
        u.copy_(uniforms(B, seed + 1))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want(x.cpu(), u.cpu().numpy(), p=0.9))


@pytest.mark.parametrize("dtype", [synth.BF16, synth.FP32])
def test_more_rows_than_threads(dtype):
    """1,500 rows of an odd vocabulary, each with its own filters, good and bad ones."""
    B, V = 1500, 333
    x = synth.logits(B, V, seed=77, dtype=dtype)
    gen = torch.Generator().manual_seed(78)
    pick = lambda vals: torch.tensor(vals)[torch.randint(0, len(vals), (B,), generator=gen)]  # noqa: E731
    kw = dict(t=pick([0.0, 0.5, 1.0, -1.0]), k=pick([0, 1, 7, 300]), p=pick([1.0, 0.9, 0.3]),
              m=pick([0.0, 0.1]))
    u = uniforms(B, 79)
    got, err = run(x, u, **kw)
    assert torch.equal(got, want(x, u, **kw))
    assert err == g.GEMMA_DEVERR_SAMPLE


@pytest.mark.parametrize("n", [1, 31, 1023, 1024, 1025, 40000])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_crowded_upper_halves(n, softcap):
    """fp32 logits of which n share their upper 16 bits, with equal ones among them: at, below and
    above the number that is put in order at once."""
    V = 50000
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(3, V, generator=gen)
    x[:, 2000:2000 + n] = 2.0 + torch.randint(0, 8000, (3, n), generator=gen) * 2.0 ** -20
    x = x[:, torch.randperm(V, generator=gen)].contiguous()
    u = uniforms(3, 6)
    for kw in (dict(), dict(p=0.5), dict(k=300), dict(k=1000, p=0.9), dict(m=0.3), dict(t=0.2, p=0.8),
               dict(p=0.9, m=0.999), dict(k=20000, m=0.02)):
        check(x, u, softcap=softcap, **kw)
