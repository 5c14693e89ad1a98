"""GPU: the 4-bit cache and sampling as a serving loop uses them, and at their ends: a run of prompt,
decode steps and sampled tokens over layers of every kind; thousands of sequences; caches beyond
2^32 bytes; two streams at once; NaN among the keys; numbers far from one.

The bounds are those of test_q4_gpu.py: 2^-8 |out| + (2^-10 + 2^-13) A for up to 64 rows per KV
head, 2^-8 |out| + 2^-7 A (and 2^-6 A more at head_dim 512) beyond, A = sum p |v|."""
import math

import numpy as np
import pytest
import torch

import mixed_sliding_global_gb300 as g
import q4_ref as R
from sample_ref import sample_row

pytestmark = pytest.mark.gpu

SLIDING, GLOBAL, RING = R.SLIDING, R.GLOBAL, R.RING


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bound(out, mass, rows, d):
    rel = 2.0 ** -10 + 2.0 ** -13 if rows <= 64 else 2.0 ** -7 + (2.0 ** -6 if d == 512 else 0)
    return 2.0 ** -8 * out.abs() + rel * mass + 1e-6


def empty_cache(shape, d, fill=None):
    """Codes and scales [*shape][...]; garbage unless `fill` gives a generator."""
    codes = torch.empty(shape + (d // 2,), dtype=torch.uint8, device="cuda")
    scales = torch.empty(shape + (d // 64,), dtype=torch.bfloat16, device="cuda")
    if fill is not None:
        codes.random_(0, 256, generator=fill)
        scales.fill_(math.nan)
    return codes, scales


# ---------------------------------------------------------------------------------------------
# a serving loop
# ---------------------------------------------------------------------------------------------
class Model:
    """Four layers of every kind (the third reads the first one's cache), an embedding and an
    output projection, all random; the attention and the tokens are the package's."""

    LAYERS = [dict(kind=SLIDING, window=70, n_q=8, n_kv=2, d=128, kv=False, cap=256),
              dict(kind=GLOBAL, window=0, n_q=8, n_kv=1, d=512, kv=True, cap=256),
              dict(kind=SLIDING, window=70, n_q=8, n_kv=2, d=128, kv=False, cap=256),
              dict(kind=RING, window=80, n_q=4, n_kv=4, d=64, kv=False, cap=128)]
    OWNER = [0, 1, 0, 3]
    H, V, MAX = 256, 5003, 256

    def __init__(self, B):
        gen = torch.Generator(device="cuda").manual_seed(5)
        w = lambda *s: (torch.randn(*s, generator=gen, device="cuda") / math.sqrt(s[0])).bfloat16()  # noqa: E731
        self.B = B
        self.embed = w(self.H, self.V).T.contiguous() * 16
        self.out = w(self.H, self.V)
        self.wq = [w(self.H, c["n_q"] * c["d"]) for c in self.LAYERS]
        self.wk = [w(self.H, c["n_kv"] * c["d"]) for c in self.LAYERS]
        self.wv = [w(self.H, c["n_kv"] * c["d"]) for c in self.LAYERS]
        self.wo = [w(c["n_q"] * c["d"], self.H) for c in self.LAYERS]
        self.caches = [[], [], [], []]
        for layer, c in enumerate(self.LAYERS):
            own = self.OWNER[layer] == layer
            for i in range(2):
                codes, scales = empty_cache((B, c["n_kv"], c["cap"]), c["d"], gen) if own and (
                    i == 0 or not c["kv"]) else (None, None)
                self.caches[2 * i].append(codes)
                self.caches[2 * i + 1].append(scales)
        self.err = i32([0])
        n = max(g.gemma_attn_workspace_size_q4(B, c["kind"], c["window"], c["n_q"], c["n_kv"],
                                               c["d"], self.MAX, n, k_eq_v=c["kv"])
                for c in self.LAYERS for n in (1, 40))
        self.ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")   # all layers share it
        self.sws = torch.empty(max(16, g.gemma_logit_sample_workspace_size(B, self.V,
                                                                           torch.bfloat16)),
                               dtype=torch.uint8, device="cuda")

    def tensors(self):
        return [t for x in self.caches for t in x if t is not None]

    def step(self, ids, pos, lens, u, token, seen=None):
        """Tokens ids [B][n] at positions pos [B] on: writes the sampled next token."""
        B, n = ids.shape
        h = self.embed[ids.long()]
        for layer, c in enumerate(self.LAYERS):
            q = (h @ self.wq[layer]).reshape(B, n, c["n_q"], c["d"])
            k = (h @ self.wk[layer]).reshape(B, n, c["n_kv"], c["d"])
            v = None if c["kv"] else (h @ self.wv[layer]).reshape(B, n, c["n_kv"], c["d"])
            kw = dict(k_eq_v=c["kv"], device_error=self.err)
            g.gemma_kv_append_q4(*self.caches, self.OWNER, layer, k, v, pos, kind=c["kind"], **kw)
            o = torch.empty_like(q)
            g.gemma_attn_q4(o, q, *self.caches, self.OWNER, layer, lens, self.MAX, kind=c["kind"],
                            window=c["window"], n_kv=c["n_kv"], scale=c["d"] ** -0.5,
                            workspace=self.ws, **kw)
            if seen is not None:
                own = self.OWNER[layer]
                seen.append((layer, q.cpu(), o.cpu(), lens.cpu().tolist(),
                             [None if x[own] is None else x[own].cpu() for x in self.caches]))
            h = h + o.reshape(B, n, -1) @ self.wo[layer]
        logits = (h[:, -1] @ self.out).contiguous()
        g.gemma_logit_sample(logits, token, u, temperature=self.t, top_k=self.k, top_p=self.p,
                             softcap=30.0, workspace=self.sws, device_error=self.err)
        return logits


def test_prompt_decode_and_sampling_together():
    """A prompt of 40 tokens and eight decode steps: every layer's attention against 64 bits over
    its owner's cache as it then is, every token against the definition on its logits; then the
    same steps from a captured graph, bit for bit."""
    B, n = 3, 40
    m = Model(B)
    m.t = torch.tensor([0.8, 1.0, 0.0], device="cuda")
    m.k = i32([20, 0, 5])
    m.p = torch.tensor([0.9, 0.95, 1.0], device="cuda")
    gen = torch.Generator().manual_seed(8)
    prompt = torch.randint(0, m.V, (B, n), generator=gen).int().cuda()
    us = torch.rand(9, B, generator=gen)
    seen = []

    def verify(logits, u, token):
        for layer, q, o, lens, cache in seen:
            c = m.LAYERS[layer]
            k = R.values(cache[0], cache[1])
            v = k if c["kv"] else R.values(cache[2], cache[3])
            out, mass = R.attention(q, k, v, lens, c["kind"], c["window"], c["d"] ** -0.5)
            rows = q.shape[1] * c["n_q"] // c["n_kv"]
            assert ((o.double() - out).abs() <= bound(out, mass, rows, c["d"])).all(), (layer, lens)
        x = logits.cpu().double().numpy()
        f = lambda t: t.cpu().double().tolist()  # noqa: E731
        want = [sample_row(x[b], float(np.float32(u[b])), f(m.t)[b], int(m.k[b]), f(m.p)[b], 0.0,
                           30.0) for b in range(B)]
        assert token.tolist() == want
        seen.clear()

    pos, lens = i32([0] * B), i32([n] * B)
    token = i32([-7] * B)
    u = us[0].cuda()
    verify(m.step(prompt, pos, lens, u, token, seen), us[0], token.cpu())
    ids = token[:, None].clone()
    pos += n
    lens += 1
    start = [t.clone() for t in m.tensors()], ids.clone()
    eager = []
    for i in range(8):
        u.copy_(us[i + 1])
        verify(m.step(ids, pos, lens, u, token, seen), us[i + 1], token.cpu())
        eager.append(token.cpu().tolist())
        ids.copy_(token[:, None])
        pos += 1
        lens += 1
    assert m.err.item() == 0
    final = [t.clone() for t in m.tensors()]

    for t, t0 in zip(m.tensors(), start[0]):
        t.copy_(t0)
    ids.copy_(start[1])
    pos.fill_(n)
    lens.fill_(n + 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        m.step(ids, pos, lens, u, token)
        ids.copy_(token[:, None])
        pos.add_(1)
        lens.add_(1)
    for i in range(8):
        u.copy_(us[i + 1])
        m.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert token.cpu().tolist() == eager[i]
    for t, t1 in zip(m.tensors(), final):
        assert torch.equal(t.view(torch.uint8), t1.view(torch.uint8))
    assert m.err.item() == 0


# ---------------------------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------------------------
def attend(q, cache, lens, kind, window, msl, n_kv, k_eq_v, table=None, scale=None):
    d = q.shape[-1]
    out = torch.full_like(q, math.nan)
    err = i32([0])
    n = g.gemma_attn_workspace_size_q4(q.shape[0], kind, window, q.shape[2], n_kv, d, msl,
                                       q.shape[1], k_eq_v=k_eq_v)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    g.gemma_attn_q4(out, q, *[[x] for x in cache], [0], 0, i32(lens), msl, kind=kind,
                    window=window, n_kv=n_kv, k_eq_v=k_eq_v, scale=scale or d ** -0.5,
                    block_table=table, workspace=ws, device_error=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out.cpu()


@pytest.mark.parametrize("B,n_q,n_kv,d,cap", [(4200, 2, 1, 64, 96), (700, 4, 4, 64, 480)])
def test_thousands_of_sequences(B, n_q, n_kv, d, cap):
    """More sequences than shares are laid out for, of every length up to the capacity."""
    gen = torch.Generator().manual_seed(B)
    cache = [*empty_cache((B, n_kv, cap), d), *empty_cache((B, n_kv, cap), d)]
    new = [torch.randn(B, cap, n_kv, d, generator=gen).bfloat16().cuda() for _ in range(2)]
    g.gemma_kv_append_q4(*[[x] for x in cache], [0], 0, *new, i32([0] * B),
                         k_eq_v=False)
    lens = torch.randint(1, cap + 1, (B,), generator=gen).tolist()
    q = torch.randn(B, 1, n_q, d, generator=gen).bfloat16().cuda()
    got = attend(q, cache, lens, GLOBAL, 0, cap, n_kv, False)
    pick = torch.randperm(B, generator=gen)[:300].tolist() + [0, B - 1]
    k, v = (R.values(cache[i][pick].cpu(), cache[i + 1][pick].cpu()) for i in (0, 2))
    out, mass = R.attention(q[pick].cpu(), k, v, [lens[b] for b in pick], GLOBAL, 0, d ** -0.5)
    assert ((got[pick].double() - out).abs() <= bound(out, mass, 1, d)).all()


@pytest.mark.parametrize("n", [1, 5, 60])
@pytest.mark.parametrize("paged", [False, True])
def test_cache_beyond_32_bit_offsets(paged, n):
    """Rows whose codes lie beyond 2^32 bytes: written, read back and attended to."""
    d, n_q, window, B, tail = 512, 4, 300, 2, 512
    gen = torch.Generator().manual_seed(n)
    if paged:
        page, n_pages = 128, 150000                       # 4.9 GB of codes
        cache, per = empty_cache((n_pages, 1, page), d), 4
        ids = torch.arange(n_pages - B * per, n_pages).flip(0).reshape(B, per).int()
        table, lens, msl = ids.cuda(), [512, 433], 512
    else:
        cap = 10_000_000                                  # 2.56 GB of codes per sequence
        cap -= cap % 32
        cache, table, lens, msl = empty_cache((B, 1, cap), d), None, [cap, cap - 777], cap
    cache = [*cache, None, None]
    new = torch.randn(B, tail, 1, d, generator=gen).bfloat16()
    first = [max(0, L - tail) for L in lens]
    kw = dict(k_eq_v=True, block_table=table)
    new_pos = i32(first)
    g.gemma_kv_append_q4(*[[x] for x in cache], [0], 0, new[:, :min(tail, min(lens))].cuda(), None,
                         new_pos, **kw)
    m = min(tail, min(lens))
    back = torch.empty(B, m, 1, d, dtype=torch.bfloat16, device="cuda")
    g.gemma_kv_read_q4(*[[x] for x in cache], [0], 0, back, None, new_pos, **kw)
    code, scale = R.quantise(new[:, :m])
    want = code.double() * scale.repeat_interleave(64, -1)
    assert torch.equal(back.cpu().double(), want)
    # the written rows as a cache of their own: sequence b's position first + m is its end
    ends = [f + m for f in first]
    q = torch.randn(B, n, n_q, d, generator=gen).bfloat16().cuda()
    got = attend(q, cache, ends, SLIDING, window, msl, 1, True, table)
    k = want.transpose(1, 2)
    out, mass = R.attention(q.cpu(), k, k, [m] * B, SLIDING, window, d ** -0.5)
    assert ((got.double() - out).abs() <= bound(out, mass, n * n_q, d)).all()


# ---------------------------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------------------------
def test_two_streams_at_once():
    """Calls on two streams with a workspace each give what they give alone."""
    B, n_q, d, cap = 16, 16, 512, 2048
    gen = torch.Generator(device="cuda").manual_seed(3)
    jobs = []
    for i in range(2):
        codes, _ = empty_cache((B, 1, cap), d, gen)
        scales = torch.rand(B, 1, cap, d // 64, generator=gen, device="cuda").bfloat16()
        lens = torch.randint(1, cap + 1, (B,), generator=gen, device="cuda").int()
        q = torch.randn(B, 1, n_q, d, generator=gen, device="cuda").bfloat16()
        ws = torch.empty(g.gemma_attn_workspace_size_q4(B, GLOBAL, 0, n_q, 1, d, cap, 1,
                                                        k_eq_v=True),
                         dtype=torch.uint8, device="cuda")
        x = torch.randn(9, 50001, generator=gen, device="cuda") * 4
        x = x.bfloat16() if i else x
        sws = torch.empty(g.gemma_logit_sample_workspace_size(9, 50001, x.dtype),
                          dtype=torch.uint8, device="cuda")
        jobs.append((codes, scales, lens, q, ws, x, torch.rand(9, generator=gen, device="cuda"),
                     sws, torch.full((9,), 0.9, device="cuda")))
    outs = [[torch.empty_like(j[3]) for _ in range(20)] for j in jobs]
    toks = [[i32([-7] * 9) for _ in range(20)] for j in jobs]

    def go(i, r):
        codes, scales, lens, q, ws, x, u, sws, p = jobs[i]
        g.gemma_attn_q4(outs[i][r], q, [codes], [scales], [None], [None], [0], 0, lens, cap,
                        kind=GLOBAL, window=0, n_kv=1, k_eq_v=True, scale=d ** -0.5, workspace=ws)
        g.gemma_logit_sample(x, toks[i][r], u, top_p=p, workspace=sws)

    for i in range(2):
        go(i, 0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(1, 20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                go(i, r)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
        assert all(torch.equal(t, toks[i][0]) for t in toks[i])
        assert (toks[i][0] >= 0).all()


# ---------------------------------------------------------------------------------------------
# numbers
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("d,n_q", [(128, 4), (256, 16)])
def test_nan_among_the_keys(d, n_q, n):
    """A NaN group of K makes every row that sees the key NaN, one of V its 64 columns."""
    L, cap = 300, 320
    gen = torch.Generator().manual_seed(d)
    x = [torch.randn(2, L, 1, d, generator=gen).bfloat16() for _ in range(2)]
    x[0][0, 7, 0, 3] = math.nan        # K of sequence 0
    x[1][1, 9, 0, 64] = -math.inf      # V's second group of sequence 1
    cache = [*empty_cache((2, 1, cap), d), *empty_cache((2, 1, cap), d)]
    g.gemma_kv_append_q4(*[[t] for t in cache], [0], 0, x[0].cuda(), x[1].cuda(), i32([0, 0]),
                         k_eq_v=False)
    q = torch.randn(2, n, n_q, d, generator=gen).bfloat16().cuda()
    got = attend(q, cache, [L, L], GLOBAL, 0, L, 1, False)
    assert torch.isnan(got[0]).all()
    assert torch.isnan(got[1, ..., 64:128]).all()
    k, v = (R.values(cache[i].cpu(), cache[i + 1].cpu()) for i in (0, 2))
    v[1, 0, 9, 64:128] = 0
    out, mass = R.attention(q.cpu(), k, v, [L, L], GLOBAL, 0, d ** -0.5)
    ok = (got.double() - out).abs() <= bound(out, mass, n * n_q, d)
    assert ok[1, ..., :64].all() and ok[1, ..., 128:].all()


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("e", [-60, 50])
def test_magnitudes_far_from_one(e, n):
    """Queries of 2^e with keys of 2^-e, values whose rows lie many binades apart, the largest
    values late: the scores are ordinary, and so are the bounds."""
    d, n_q, L = 256, 8, 400
    gen = torch.Generator().manual_seed(e + 100)
    k = torch.randn(1, L, 2, d, generator=gen) * 2.0 ** -e
    v = torch.randn(1, L, 2, d, generator=gen)
    v *= torch.exp2(torch.linspace(-8, 8, L)).reshape(1, L, 1, 1) * 2.0 ** e
    cache = [*empty_cache((1, 2, 416), d), *empty_cache((1, 2, 416), d)]
    g.gemma_kv_append_q4(*[[t] for t in cache], [0], 0, k.bfloat16().cuda(), v.bfloat16().cuda(),
                         i32([0]), k_eq_v=False)
    q = (torch.randn(1, n, n_q, d, generator=gen) * 2.0 ** e).bfloat16().cuda()
    got = attend(q, cache, [L], GLOBAL, 0, L, 2, False)
    kk, vv = (R.values(cache[i].cpu(), cache[i + 1].cpu()) for i in (0, 2))
    out, mass = R.attention(q.cpu(), kk, vv, [L], GLOBAL, 0, d ** -0.5)
    rel = 2.0 ** -10 + 2.0 ** -13
    assert ((got.double() - out).abs() <= 2.0 ** -8 * out.abs() + rel * mass).all()


def test_tensors_of_other_devices_are_refused():
    """Every tensor of a call has to be on the current device."""
    cache = [*empty_cache((1, 1, 64), 64), None, None]
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    kw = dict(kind=GLOBAL, window=0, n_kv=1, k_eq_v=True, scale=1.0)

    def call(q=q, cache=cache, lens=i32([1]), **more):
        g.gemma_attn_q4(torch.empty_like(q), q, *[[x] for x in cache], [0], 0, lens, 64, **kw,
                        **more)

    call()
    torch.cuda.synchronize()
    for bad in (dict(q=q.cpu()), dict(cache=[cache[0].cpu(), *cache[1:]]), dict(lens=i32([1]).cpu()),
                dict(workspace=torch.empty(64)), dict(device_error=torch.zeros(1).int())):
        with pytest.raises(ValueError):
            call(**bad)
    x, u = torch.zeros(1, 8, device="cuda").bfloat16(), torch.zeros(1, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    for bad in (dict(uniform=u.cpu()), dict(top_p=u.cpu()), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            g.gemma_logit_sample(x, i32([0]), **{**dict(uniform=u, workspace=ws), **bad})


@pytest.mark.parametrize("gap", [8.0, 12.0])
@pytest.mark.parametrize("d,n_q", [(128, 8), (512, 16)])
def test_small_weights_behind_a_large_one(d, n_q, gap):
    """One key with nearly all the weight and a value of zero: what is left are weights of about
    e^-gap. Each is off by 2^-11 of itself twice, or, below fp16's normal range, by at most 2^-31
    of the largest weight as such and 2^-30 of it times V's largest scale as a product."""
    L = 260
    gen = torch.Generator().manual_seed(d)
    q = torch.randn(1, 1, n_q, d, generator=gen)
    q[..., :64] = 1.0                       # the first group sets the score, the others add noise
    k = torch.randn(1, L, 1, d, generator=gen) * 0.05
    k[..., :64] = 0.0
    k[:, 17, :, :64] = gap * math.sqrt(d) / 64
    v = torch.randn(1, L, 1, d, generator=gen)
    v[:, 17] = 0.0
    cache = [*empty_cache((1, 1, 288), d), *empty_cache((1, 1, 288), d)]
    g.gemma_kv_append_q4(*[[t] for t in cache], [0], 0, k.bfloat16().cuda(), v.bfloat16().cuda(),
                         i32([0]), k_eq_v=False)
    got = attend(q.bfloat16().cuda(), cache, [L], GLOBAL, 0, L, 1, False)
    kk, vv = (R.values(cache[i].cpu(), cache[i + 1].cpu()) for i in (0, 2))
    out, mass = R.attention(q.bfloat16(), kk, vv, [L], GLOBAL, 0, d ** -0.5)
    small = L * (2.0 ** -31 + 2.0 ** -30) * vv[:, :, :L].abs().max()
    assert mass.max() < 260 * math.exp(-gap) * 3      # the large weight carries nothing
    assert ((got.double() - out).abs() <= 2.0 ** -8 * out.abs() +
            (2.0 ** -10 + 2.0 ** -13) * mass + small).all()


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("e", [-112, 112])
def test_queries_and_keys_at_the_ends_of_the_range(e, n, softcap):
    """Queries of 2^e with keys of 2^-e: scores of ordinary size from numbers whose products with the
    codes' 2^24 leave fp32's range."""
    d, n_q, L = 256, 8, 300
    gen = torch.Generator().manual_seed(e + 500)
    k = torch.randn(1, L, 2, d, generator=gen) * 2.0 ** -e
    v = torch.randn(1, L, 2, d, generator=gen)
    cache = [*empty_cache((1, 2, 320), d), *empty_cache((1, 2, 320), d)]
    g.gemma_kv_append_q4(*[[t] for t in cache], [0], 0, k.bfloat16().cuda(), v.bfloat16().cuda(),
                         i32([0]), k_eq_v=False)
    q = (torch.randn(1, n, n_q, d, generator=gen) * 2.0 ** e).bfloat16().cuda()
    out = torch.full_like(q, math.nan)
    size = g.gemma_attn_workspace_size_q4(1, GLOBAL, 0, n_q, 2, d, L, n, k_eq_v=False)
    g.gemma_attn_q4(out, q, *[[t] for t in cache], [0], 0, i32([L]), L, kind=GLOBAL, window=0,
                    n_kv=2, k_eq_v=False, scale=d ** -0.5, softcap=softcap,
                    workspace=torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    kk, vv = (R.values(cache[i].cpu(), cache[i + 1].cpu()) for i in (0, 2))
    ref, mass = R.attention(q.cpu(), kk, vv, [L], GLOBAL, 0, d ** -0.5, softcap)
    assert ((out.cpu().double() - ref).abs() <= bound(ref, mass, n * n_q // 2, d)).all()
