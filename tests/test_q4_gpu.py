"""GPU: the 4-bit KV cache (append, read-back, attention) against its 64-bit definition.

Codes, scales and read-back values are compared exactly: the quantiser is exact arithmetic. The
attention's bound is derived from its roundings (tests/q4_ref.py gives out = sum p v and
A = sum p |v|). A rounding to bf16 (eight significant bits) is off by at most 2^-8 of the value
(half of torch.finfo's eps 2^-7), one to fp16 by 2^-11, so the output's is at most 2^-8 |out|, and
the weights carry
  - up to 64 rows (token, query head) per KV head, straight over the cache: the roundings to fp16
    of p and of p times V's scale, 2^-10 A together, and fp32 sums: 2^-13 A covers scores up to 16
    whose exponents are off by 16 log2(e) 2^-24 per addition of eight groups, and the like;
  - more rows, over a dequantised bf16 copy (at head_dim 128 and 512 up to 128 and 192 still
    directly, well within this): the rounding of p to bf16 (2^-8) and that of the normaliser's
    terms (2^-8), together 2^-7 A; and at head_dim 512 that of half of each score to
    fp16: scores below 16 move exponents by at most 16 * 2^-11 = 2^-7 and weights by twice that
    with the normaliser, 2^-6 A.
"""
import math

import pytest
import torch

import mixed_sliding_global_gb300 as g
import q4_ref as R

pytestmark = pytest.mark.gpu

SLIDING, GLOBAL, RING = R.SLIDING, R.GLOBAL, R.RING


def rows(shape, seed, dtype=torch.bfloat16, spread=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    if spread:   # group magnitudes over many binades, zeros among them
        e = torch.randint(-30, 30, shape[:-1] + (shape[-1] // 64, 1), generator=gen).float()
        x = (x.reshape(*shape[:-1], -1, 64) * torch.exp2(e)).reshape(shape)
        x[..., ::7] = 0
    return x.to(dtype)


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


class Cache:
    """A 4-bit cache on the GPU, filled with garbage (NaN scales) until rows are written."""

    def __init__(self, B, n_kv, cap, d, k_eq_v=False, page=0, seed=0):
        self.kind_shape = (B, n_kv, cap, d)
        gen = torch.Generator().manual_seed(seed)
        if page:
            per = -(-cap // page)
            self.n_pages = B * per + 2
            self.table = torch.randperm(self.n_pages, generator=gen)[:B * per].int().reshape(B, per)
            shape = (self.n_pages, n_kv, page)
        else:
            self.table, shape = None, (B, n_kv, cap)
        self.page, self.k_eq_v = page, k_eq_v
        self.t = []
        for _ in range(1 if k_eq_v else 2):
            codes = torch.randint(0, 256, shape + (d // 2,), generator=gen, dtype=torch.uint8)
            scales = torch.full(shape + (d // 64,), math.nan, dtype=torch.bfloat16)
            self.t += [codes.cuda(), scales.cuda()]
        if k_eq_v:
            self.t += [None, None]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self):
        return [[x] for x in self.t]

    def kw(self):
        return dict(block_table=None if self.table is None else self.table.cuda(),
                    device_error=self.err, k_eq_v=self.k_eq_v)

    def append(self, k, v, pos, kind=GLOBAL):
        g.gemma_kv_append_q4(*self.args(), [0], 0, k.cuda(), None if v is None else v.cuda(),
                             torch.tensor(pos, dtype=torch.int32, device="cuda"), kind=kind,
                             **self.kw())

    def read(self, n, pos, kind=GLOBAL, dtype=torch.bfloat16):
        B, n_kv, _, d = self.kind_shape
        out = [torch.full((B, n, n_kv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        g.gemma_kv_read_q4(*self.args(), [0], 0, out[0], None if self.k_eq_v else out[1],
                           torch.tensor(pos, dtype=torch.int32, device="cuda"), kind=kind,
                           **self.kw())
        return out[0].cpu(), out[1].cpu()

    def values(self):
        k = R.values(self.t[0].cpu(), self.t[1].cpu())
        return k, (k if self.k_eq_v else R.values(self.t[2].cpu(), self.t[3].cpu()))

    def attend(self, q, lens, kind, window, softcap=0.0, max_len=None, scale=None, ws=None):
        B, n_kv, _, d = self.kind_shape
        q = q.cuda()
        out = torch.full_like(q, math.nan)
        msl = max_len or max(max(lens), q.shape[1])
        n = g.gemma_attn_workspace_size_q4(q.shape[0], kind, window, q.shape[2], n_kv, d, msl,
                                           q.shape[1], k_eq_v=self.k_eq_v)
        if ws is None:   # contents on entry must not matter
            ws = torch.full((max(n // 4, 4),), math.nan, dtype=torch.float32, device="cuda")
        g.gemma_attn_q4(out, q, *self.args(), [0], 0,
                        torch.tensor(lens, dtype=torch.int32, device="cuda"), msl, kind=kind,
                        window=window, n_kv=n_kv, scale=scale or d ** -0.5, softcap=softcap,
                        workspace=ws, **self.kw())
        torch.cuda.synchronize()
        return out


# ---------------------------------------------------------------------------------------------
# append and read-back
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n_kv,n,d,k_eq_v", [(1, 1, 1, 64, False), (3, 2, 5, 128, True),
                                               (2, 8, 1, 256, False), (1, 1, 37, 512, True),
                                               (5, 3, 9, 64, True), (2, 4, 70, 256, False)])
def test_append_codes_and_scales_are_exact(dtype, B, n_kv, n, d, k_eq_v):
    """Every code and scale equals the definition's, rows behind and before the new ones keep
    their bits, and the read-back gives code * scale exactly in both types."""
    cap, pos = 96, [(17 * b) % 20 for b in range(B)]
    c = Cache(B, n_kv, cap, d, k_eq_v, seed=n)
    before = [None if x is None else x.clone() for x in c.t]
    new = [rows((B, n, n_kv, d), 3 + i, dtype, spread=True) for i in range(1 if k_eq_v else 2)]
    c.append(new[0], None if k_eq_v else new[1], pos)
    assert c.err.item() == 0
    for i, x in enumerate(new):
        code, scale = R.quantise(x)
        sign = torch.signbit(x) & (scale > 0).repeat_interleave(64, -1)
        want_c = before[2 * i].cpu().clone()
        want_s = before[2 * i + 1].cpu().clone()
        for b in range(B):
            sl = slice(pos[b], pos[b] + n)
            want_c[b, :, sl] = R.pack(code[b], sign[b]).transpose(0, 1)
            want_s[b, :, sl] = scale[b].bfloat16().transpose(0, 1)
        assert torch.equal(c.t[2 * i].cpu(), want_c)
        assert torch.equal(bits(c.t[2 * i + 1].cpu()), bits(want_s))
        for dt in (torch.bfloat16, torch.float32):
            got = c.read(n, pos, dtype=dt)[i]
            want = code.double() * scale.repeat_interleave(64, -1)
            assert torch.equal(got.double(), want)
            assert torch.equal(want.bfloat16().double(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_special_values(dtype):
    """Zeros, ties, subnormals, the type's largest values, NaN and infinities."""
    d = 512
    x = torch.zeros(1, 1, 1, d)
    x[..., 0:64] = 0
    x[..., 64:128] = torch.arange(64).float() / 64 * 7          # ties among them at scale 1
    x[..., 127] = 7
    x[..., 128:192] = 2.0 ** -130
    x[..., 192:256] = torch.finfo(dtype).max
    x[..., 200] = -torch.finfo(dtype).max
    x[..., 256:320] = 1.0
    x[..., 300] = math.nan
    x[..., 320:384] = 2.0
    x[..., 350] = -math.inf
    x[..., 384:448] = -torch.arange(64).float() * 0.5
    x[..., 448:512] = 1e-30
    x = x.to(dtype)
    c = Cache(1, 1, 32, d, True)
    c.append(x, None, [3])
    got = c.read(1, [3], dtype=torch.float32)[0].double()
    code, scale = R.quantise(x)
    want = code.double() * scale.repeat_interleave(64, -1)
    assert torch.isnan(got[..., 256:384]).all()
    keep = torch.ones(d, dtype=torch.bool)
    keep[256:384] = False
    assert torch.equal(got[..., keep], want[..., keep])
    assert c.err.item() == 0


def test_append_ring_paged_and_errors():
    """Ring slots wrap; paged rows land in their pages; bad positions and pages are reported and
    write nothing; a shared layer writes nothing."""
    d, n_kv = 128, 2
    x = rows((2, 7, n_kv, d), 5)
    c = Cache(2, n_kv, 128, d, True)
    c.append(x, None, [125, 1000], kind=RING)
    k, _ = c.values()
    code, scale = R.quantise(x)
    want = code.double() * scale.repeat_interleave(64, -1)
    for b, p in enumerate((125, 1000)):
        for t in range(7):
            assert torch.equal(k[b, :, (p + t) % 128], want[b, t])
    assert torch.equal(c.read(7, [125, 1000], kind=RING)[0].double(), want)
    assert c.err.item() == 0

    c = Cache(2, n_kv, 512, d, True, page=128, seed=2)
    c.append(x, None, [125, 380])
    assert torch.equal(c.read(7, [125, 380])[0].double(), want) and c.err.item() == 0
    c.table[1, 3] = c.n_pages
    before = [t.clone() for t in c.t[:2]]
    c.append(rows((2, 7, n_kv, d), 6), None, [10, 384])
    assert c.err.item() == g.GEMMA_DEVERR_PAGE
    k0, k1 = R.values(before[0].cpu(), before[1].cpu()), c.values()[0]
    page = int(c.table[1, 2])
    assert torch.equal(torch.nan_to_num(k0[page]), torch.nan_to_num(k1[page]))
    assert torch.equal(c.read(1, [10, 384])[0][1], torch.zeros(1, n_kv, d, dtype=torch.bfloat16))

    c = Cache(2, n_kv, 64, d, True)
    before = [t.clone() for t in c.t[:2]]
    c.append(x, None, [58, -1])
    assert c.err.item() == g.GEMMA_DEVERR_WRITE_POS
    assert torch.equal(c.t[0], before[0]) and torch.equal(bits(c.t[1]), bits(before[1]))
    assert (c.read(7, [58, -1])[0] == 0).all()
    g.gemma_kv_append_q4([c.t[0], None], [c.t[1], None], None, None, [0, 0], 1, x.cuda(), None,
                         torch.zeros(2, dtype=torch.int32, device="cuda"), k_eq_v=True)
    assert torch.equal(c.t[0], before[0])


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def fill(c, lens, kind, spread=1.0, seed=11):
    """Append every position that a step may read (the last cap ones on a ring)."""
    B, n_kv, cap, d = c.kind_shape
    gen = torch.Generator().manual_seed(seed)
    for b, L in enumerate(lens):
        n = min(L, cap) if kind == RING else L
        if n < 1:
            continue
        x = [(torch.randn(1, n, n_kv, d, generator=gen) * spread).bfloat16() for _ in range(2)]
        one = Cache.__new__(Cache)
        one.__dict__.update(c.__dict__)
        if c.table is None:
            one.t = [None if t is None else t[b:b + 1] for t in c.t]
        else:
            one.table = c.table[b:b + 1]
        one.append(x[0], None if c.k_eq_v else x[1], [L - n], kind=kind)


def check(c, q, lens, kind, window, softcap=0.0, **kw):
    got = c.attend(q, lens, kind, window, softcap, **kw)
    assert c.err.item() == 0
    k, v = c.values()
    out, mass = R.attention(q, k, v, lens, kind, window, q.shape[-1] ** -0.5, softcap, c.table,
                            c.page)
    err = (got.double().cpu() - out).abs()
    d, n = q.shape[-1], q.shape[1]
    direct = n * (q.shape[2] // c.kind_shape[1]) <= 64
    rel = 2.0 ** -10 + 2.0 ** -13 if direct else 2.0 ** -7 + (2.0 ** -6 if d == 512 else 0)
    bound = 2.0 ** -8 * out.abs() + rel * mass + 1e-6
    assert torch.isfinite(got).all()
    worst = (err / bound).max().item()
    assert worst <= 1, f"error {worst:.2f} of the bound, {err.max().item():.3e}"
    return got


DECODE = [
    # kind, window, n_q, n_kv, d, k_eq_v, lens, page, softcap
    (GLOBAL, 0, 1, 1, 64, False, [1], 0, 0.0),
    (GLOBAL, 0, 16, 1, 512, True, [1, 2, 127, 128, 129, 1000], 0, 0.0),
    (GLOBAL, 0, 16, 1, 512, False, [300, 31], 0, 0.0),
    (GLOBAL, 0, 8, 1, 512, True, [513, 5], 0, 50.0),
    (SLIDING, 100, 16, 8, 256, False, [99, 100, 101, 333], 0, 0.0),
    (SLIDING, 1, 4, 2, 128, False, [1, 40, 129], 0, 0.0),
    (SLIDING, 1024, 8, 2, 256, False, [2048], 0, 0.0),
    (SLIDING, 65, 16, 1, 256, True, [64, 65, 66, 500], 0, 0.0),
    (GLOBAL, 0, 4, 1, 64, True, [700, 33], 0, 0.0),
    (GLOBAL, 0, 16, 1, 128, False, [257, 3, 640], 0, 30.0),
    (GLOBAL, 0, 6, 3, 128, False, [90, 260], 0, 0.0),
    (RING, 100, 8, 2, 256, False, [50, 128, 129, 900], 0, 0.0),
    (RING, 128, 16, 1, 512, True, [1, 1000], 0, 0.0),
    (RING, 300, 2, 2, 64, False, [383, 385], 0, 0.0),
    (GLOBAL, 0, 8, 2, 256, False, [1, 128, 129, 700], 128, 0.0),
    (SLIDING, 200, 16, 8, 64, True, [256, 257, 700], 256, 50.0),
    (GLOBAL, 0, 32, 2, 512, False, [400, 130], 128, 0.0),
]


@pytest.mark.parametrize("kind,window,n_q,n_kv,d,k_eq_v,lens,page,softcap", DECODE)
def test_decode(kind, window, n_q, n_kv, d, k_eq_v, lens, page, softcap):
    cap = -(-(window if kind == RING else max(lens)) // 128) * 128
    c = Cache(len(lens), n_kv, cap, d, k_eq_v, page)
    fill(c, lens, kind)
    q = rows((len(lens), 1, n_q, d), 21)
    check(c, q, lens, kind, window, softcap)


MULTI = [
    (GLOBAL, 0, 16, 1, 512, True, [40, 700], 9, 0, 0.0),
    (GLOBAL, 0, 2, 1, 64, False, [5, 129], 5, 0, 0.0),
    (SLIDING, 100, 16, 8, 256, False, [300, 33], 33, 0, 0.0),
    (SLIDING, 7, 4, 2, 128, False, [64, 200], 64, 128, 0.0),
    (RING, 100, 8, 2, 256, False, [120, 800], 20, 0, 50.0),
    (GLOBAL, 0, 8, 4, 128, True, [260, 131], 2, 0, 0.0),
    (SLIDING, 64, 8, 1, 512, False, [150, 90], 3, 0, 0.0),
    (GLOBAL, 0, 8, 2, 256, False, [150, 390], 70, 128, 0.0),
    (GLOBAL, 0, 16, 1, 64, True, [500], 4, 0, 0.0),
]


@pytest.mark.parametrize("kind,window,n_q,n_kv,d,k_eq_v,lens,n,page,softcap", MULTI)
def test_several_tokens(kind, window, n_q, n_kv, d, k_eq_v, lens, n, page, softcap):
    cap = -(-(window + n - 1 if kind == RING else max(lens)) // 128) * 128
    c = Cache(len(lens), n_kv, cap, d, k_eq_v, page)
    fill(c, lens, kind)
    q = rows((len(lens), n, n_q, d), 22)
    check(c, q, lens, kind, window, softcap)


def test_invalid_lengths_are_reported_and_zeroed():
    for n in (1, 3, 40):
        c = Cache(4, 2, 128, 128)
        fill(c, [100] * 4, GLOBAL)
        q = rows((4, n, 4, 128), 5)
        got = c.attend(q, [100, n - 1, 129, 60], GLOBAL, 0, max_len=128)
        assert c.err.item() == g.GEMMA_DEVERR_SEQ_LEN
        assert (got[1] == 0).all() and (got[2] == 0).all()
        k, v = c.values()
        out, mass = R.attention(q[::3], k[::3], v[::3], [100, 60], GLOBAL, 0, 128 ** -0.5)
        assert ((got[::3].double().cpu() - out).abs() <= 2.0 ** -8 * out.abs() + 2.0 ** -7 * mass +
                1e-6).all()


@pytest.mark.parametrize("d,n", [(64, 1), (256, 1), (256, 5), (512, 1)])
def test_units_shared_by_clusters(d, n):
    """Few sequences, whose key tiles are shared out within clusters: of one tile and of all, with
    bad lengths among them, and two pages that are none."""
    lens = [1000, n - 1, n, 1025, 129, 777]
    c = Cache(6, 1, 1024, d)
    fill(c, [min(max(x, 0), 1024) for x in lens], GLOBAL)
    q = rows((6, n, 4, d), 15)
    got = c.attend(q, lens, GLOBAL, 0, max_len=1024)
    assert c.err.item() == g.GEMMA_DEVERR_SEQ_LEN
    assert (got[1] == 0).all() and (got[3] == 0).all()
    ok = [0, 2, 4, 5]
    k, v = c.values()
    out, mass = R.attention(q[ok], k[ok], v[ok], [lens[i] for i in ok], GLOBAL, 0, d ** -0.5)
    assert ((got[ok].double().cpu() - out).abs() <= 2.0 ** -8 * out.abs() +
            (2.0 ** -10 + 2.0 ** -13) * mass + 1e-6).all()

    c = Cache(2, 1, 1024, d, page=128)
    fill(c, [900, 1024], GLOBAL)
    lost = [int(c.table[0, 3]), int(c.table[1, 7])]
    c.table[0, 3], c.table[1, 7] = c.n_pages, -1
    got = c.attend(q[:2], [900, 1024], GLOBAL, 0, max_len=1024)
    assert c.err.item() == g.GEMMA_DEVERR_PAGE
    k, v = c.values()
    c.table[0, 3], c.table[1, 7] = lost
    for p in lost:
        k[p], v[p] = 0, 0
    out, mass = R.attention(q[:2], k, v, [900, 1024], GLOBAL, 0, d ** -0.5, 0.0, c.table, 128)
    assert ((got.double().cpu() - out).abs() <= 2.0 ** -8 * out.abs() +
            (2.0 ** -10 + 2.0 ** -13) * mass + 1e-6).all()


def test_bad_page_reads_as_zeros():
    for n in (1, 40):
        c = Cache(1, 1, 512, 256, False, page=128)
        fill(c, [400], GLOBAL)
        good = [t.clone() for t in c.t]
        page = int(c.table[0, 1])
        c.table[0, 1] = -5
        q = rows((1, n, 4, 256), 6)
        got = c.attend(q, [400], GLOBAL, 0)
        assert c.err.item() == g.GEMMA_DEVERR_PAGE
        c.t = good
        c.table[0, 1] = page
        k, v = c.values()
        k[page], v[page] = 0, 0
        out, mass = R.attention(q, k, v, [400], GLOBAL, 0, 256 ** -0.5, 0.0, c.table, 128)
        assert ((got.double().cpu() - out).abs() <= 2.0 ** -8 * out.abs() + 2.0 ** -7 * mass +
                1e-6).all()


@pytest.mark.parametrize("d,k_eq_v,n", [(512, True, 1), (256, False, 1), (256, False, 40)])
def test_captured_step(d, k_eq_v, n):
    """Append and attention captured together on a side stream and replayed with new rows give
    what eager calls give, with a workspace that held other values."""
    n_q, n_kv = (16, 1) if k_eq_v else (8, 4)
    L0, cap = 300, 512
    c = Cache(2, n_kv, cap, d, k_eq_v)
    fill(c, [L0, 150], GLOBAL)
    start = [None if t is None else t.clone() for t in c.t]
    new = [rows((2, n, n_kv, d), 30 + i).cuda() for i in range(2)]
    q = rows((2, n, n_q, d), 33).cuda()
    pos = torch.tensor([L0, 150], dtype=torch.int32, device="cuda")
    lens = pos + n
    ws = torch.empty(max(16, g.gemma_attn_workspace_size_q4(2, GLOBAL, 0, n_q, n_kv, d, cap, n,
                                                            k_eq_v=k_eq_v)),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        g.gemma_kv_append_q4(*c.args(), [0], 0, new[0], None if k_eq_v else new[1], pos, **c.kw())
        g.gemma_attn_q4(out, q, *c.args(), [0], 0, lens, cap, kind=GLOBAL, window=0, n_kv=n_kv,
                        scale=d ** -0.5, workspace=ws, **c.kw())

    step()
    torch.cuda.synchronize()
    eager = out.clone()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for t, t0 in zip(c.t, start):
        if t is not None:
            t.copy_(t0)
    out.fill_(math.nan)
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    # another step through the same graph: new rows, new queries, one position on
    new[0].copy_(rows((2, n, n_kv, d), 40))
    new[1].copy_(rows((2, n, n_kv, d), 41))
    q.copy_(rows((2, n, n_q, d), 43))
    pos += n
    lens += n
    graph.replay()
    torch.cuda.synchronize()
    k, v = c.values()
    o, m = R.attention(q.cpu(), k, v, lens.tolist(), GLOBAL, 0, d ** -0.5)
    assert ((out.double().cpu() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -7 * m + 1e-6).all()
    assert c.err.item() == 0


def test_decode_step_follows_prompt():
    """A prompt attended through the prefill path and the tokens after it one by one: the last
    query of a prompt of n tokens gives what a decode step gives at the same length."""
    d, n_kv, n_q, n = 256, 2, 4, 50
    c = Cache(1, n_kv, 256, d)
    x = [rows((1, n, n_kv, d), 60 + i) for i in range(2)]
    c.append(x[0], x[1], [100])
    pre = [rows((1, 100, n_kv, d), 70 + i) for i in range(2)]
    c.append(pre[0], pre[1], [0])
    q = rows((1, n, n_q, d), 80)
    a = check(c, q, [150], SLIDING, 90)
    for i in (0, 17, 49):
        b = check(c, q[:, i:i + 1], [101 + i], SLIDING, 90)
        k, v = c.values()
        o, m = R.attention(q[:, i:i + 1], k, v, [101 + i], SLIDING, 90, d ** -0.5)
        diff = (a[:, i:i + 1].double() - b.double()).abs().cpu()
        # the two bounds of check() added up
        assert (diff <= 2.0 ** -7 * o.abs() + 2.0 ** -6 * m + 2e-6).all()
