"""Cases of the 4-bit KV cache (append, read-back, attention) and of the sampling step.

Each case is a dict of plain values. ``run`` computes the operator from elementary torch
operations while ``own`` is false, and through the package's entry points while it is true.

4-bit format: a row of head_dim elements has a scale per 64 elements (bf16 with at most five
significant bits, the smallest with 7 * scale >= max |x|) and codes rint(x / scale) in [-7, 7],
sign-magnitude, eight to a 32-bit little-endian word: element 2j of the eight has its magnitude
in bits 4j..4j+2 and its sign in bit (15 + 4j) % 32, element 2j + 1 in bits 16+4j..16+4j+2 and
bit (31 + 4j) % 32. code * scale is exact in bf16.
"""
import math

import torch

own = False

SLIDING, GLOBAL, RING = 0, 1, 2
GROUP = 64
DEV = "cuda"


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def _attn(name, kind, window, n_q, n_kv, d, k_eq_v, batch, lo, hi, n_new=1, softcap=0.0, page=0):
    """lo..hi: range of the sequences' lengths (after the step's append)."""
    c = dict(op="attn", kind=kind, window=window, n_q=n_q, n_kv=n_kv, head_dim=d, k_eq_v=k_eq_v,
             batch=batch, lo=lo, hi=hi, n_new=n_new, softcap=softcap, page=page)
    if name:
        c["name"] = name
    return c


def _append(name, n_kv, d, batch, n_new, k_eq_v, start):
    c = dict(op="append", n_kv=n_kv, head_dim=d, batch=batch, n_new=n_new, k_eq_v=k_eq_v,
             start=start)
    if name:
        c["name"] = name
    return c


def _sample(name, batch, vocab, dtype, softcap, top_k, top_p, min_p, temperature, mixed=False):
    c = dict(op="sample", batch=batch, vocab=vocab, dtype=dtype, softcap=softcap, top_k=top_k,
             top_p=top_p, min_p=min_p, temperature=temperature, mixed=mixed)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user, a short context: the sliding layer of the E4B-shaped decode (latency)
        _attn("decode_e4b_sliding_b1", SLIDING, 512, 8, 2, 256, False, 1, 2048, 2048),
        # one user, the 12B-shaped global layer at its full context, K read as V
        _attn("decode_12b_global_b1", GLOBAL, 0, 16, 1, 512, True, 1, 8192, 8192),
        # a full ragged serving batch: a sliding layer whose cache is a ring of the window
        _attn("decode_ring_b64", RING, 1024, 16, 8, 256, False, 64, 129, 16385),
        # the same batch's global layer: the long contexts that the 4-bit cache is for
        _attn("decode_global_b64", GLOBAL, 0, 16, 1, 512, True, 64, 129, 16385),
        # an E4B-shaped batch over a paged pool, odd lengths, attention soft-cap
        _attn("decode_paged_b13_cap", GLOBAL, 0, 8, 2, 256, False, 13, 700, 9001, 1, 50.0, 256),
        # a prompt of 512 tokens onto a cached prefix, both layer kinds of the 12B shape
        _attn("prefill_12b_sliding", SLIDING, 1024, 16, 8, 256, False, 4, 4096, 4096, 512),
        _attn("prefill_12b_global", GLOBAL, 0, 16, 1, 512, True, 4, 4096, 4096, 512),
        # the new rows of a decode step, and of a prompt chunk, quantised into the cache
        _append("append_decode_b64", 8, 256, 64, 1, False, 1000),
        _append("append_prompt_b4", 8, 256, 4, 512, False, 1601),
        # the next token of one user from the whole vocabulary, the usual filters
        _sample("sample_b1", 1, 262144, "bf16", 30.0, 64, 0.95, 0.0, 1.0),
        # a serving batch whose requests each bring their own filters
        _sample("sample_b64_mixed", 64, 262144, "bf16", 30.0, 0, 1.0, 0.0, 1.0, True),
        # fp32 logits, an odd vocabulary, nucleus sampling alone
        _sample("sample_fp32_b9", 9, 70001, "fp32", 0.0, 0, 0.9, 0.0, 0.8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    what = rng.choice(["attn", "attn", "attn", "append", "sample", "sample"])
    if what == "append":
        d = rng.choice([64, 128, 256, 512])
        n_kv = rng.choice([1, 2, 4, 8])
        batch = _log_int(rng, 1, 64)
        n_new = _log_int(rng, 1, max(1, min(700, 4096 * 256 // (batch * n_kv * d // 8 + 1))))
        return _append(None, n_kv, d, batch, n_new, rng.random() < 0.3, _log_int(rng, 1, 4000))
    if what == "sample":
        batch = _log_int(rng, 1, 64)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        vocab = _log_int(rng, 50, 262144 if dtype == "bf16" else max(51, 1 << 21) // batch)
        return _sample(None, batch, min(vocab, 262144), dtype, rng.choice([0.0, 30.0]),
                       rng.choice([0, 1, 20, 64, 1000]), rng.choice([1.0, 0.95, 0.8, 0.3]),
                       rng.choice([0.0, 0.0, 0.02, 0.1]), rng.choice([0.3, 0.7, 1.0, 1.5]),
                       rng.random() < 0.4)
    d = rng.choice([64, 128, 256, 256, 512])
    group = rng.choice([1, 2, 4, 8, 16])
    n_kv = rng.choice([1, 2, 4, 8]) if group <= 4 else rng.choice([1, 2])
    kind = rng.choice([SLIDING, GLOBAL, RING])
    window = 0 if kind == GLOBAL else rng.choice([100, 512, 1024])
    n_new = rng.choice([1, 1, 1, 1, rng.randint(2, 9), _log_int(rng, 10, 400)])
    hi = _log_int(rng, max(n_new, 16), 16385 if n_new == 1 else 4096)
    lo = rng.randint(n_new, hi)
    n_read = hi if kind == GLOBAL else min(hi, window + n_new)
    top = 60e6 if n_new == 1 else 12e6
    batch = max(1, min(_log_int(rng, 1, 64), int(top // (n_read * n_kv * d))))
    if n_new > 1:
        batch = max(1, min(batch, int(4 * 512 * 16 // (n_new * group * n_kv))))
    page = rng.choice([0, 0, 128, 256]) if kind != RING else 0
    return _attn(None, kind, window, group * n_kv, n_kv, d, rng.random() < 0.4, batch, lo, hi,
                 n_new, rng.choice([0.0, 0.0, 50.0]), page)


# --------------------------------------------------------------------------------------------
# the 4-bit format in elementary operations
# --------------------------------------------------------------------------------------------
def _quantise(x):
    """x [..., d] -> (codes uint8 [..., d/2], scales bf16 [..., d/64])."""
    d = x.shape[-1]
    g = x.float().reshape(*x.shape[:-1], d // GROUP, GROUP)
    amax = g.abs().amax(-1)
    finite = torch.isfinite(g).all(-1)
    man, ex = torch.frexp(torch.where(finite, amax, torch.ones_like(amax)).double() / 7)
    s = torch.ldexp(torch.ceil(man * 32) / 32, ex)           # up to five significant bits
    s = torch.where(amax > 0, s.clamp_min(2.0 ** -126), torch.zeros_like(s))
    live = finite & (amax > 0)
    code = torch.round(g.double() / torch.where(live, s, torch.ones_like(s)).unsqueeze(-1))
    code = torch.where(live.unsqueeze(-1), code, torch.zeros_like(code))
    scale = torch.where(finite, s, torch.full_like(s, float("nan"))).bfloat16()
    mag = code.abs().long().reshape(*x.shape[:-1], d // 8, 8)
    neg = (live.unsqueeze(-1) & torch.signbit(g)).long().reshape(*x.shape[:-1], d // 8, 8)
    word = torch.zeros_like(mag[..., 0])
    for e in range(8):
        j, h = e // 2, e % 2
        word |= mag[..., e] << (16 * h + 4 * j)
        word |= neg[..., e] << ((15 + 16 * h + 4 * j) % 32)
    byte = torch.stack([(word >> (8 * i)) & 255 for i in range(4)], -1)
    return byte.to(torch.uint8).reshape(*x.shape[:-1], d // 2).contiguous(), scale.contiguous()


def _values(codes, scales):
    """codes [..., d/2], scales [..., d/64] -> fp32 values [..., d]."""
    d = codes.shape[-1] * 2
    word = codes.contiguous().view(torch.int32)
    out = torch.empty(*word.shape, 8, dtype=torch.float32, device=codes.device)
    for e in range(8):
        j, h = e // 2, e % 2
        mag = (word >> (16 * h + 4 * j)) & 7
        neg = (word >> ((15 + 16 * h + 4 * j) % 32)) & 1
        out[..., e] = (mag * (1 - 2 * neg)).float()
    out = out.reshape(*codes.shape[:-1], d // GROUP, GROUP) * scales.float().unsqueeze(-1)
    return out.reshape(*codes.shape[:-1], d)


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _cache(g, rows, d):
    """A quantised cache of `rows` rows: unit-variance channels, a few of them larger, as
    projected keys and values have."""
    codes = torch.empty(rows, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, d // GROUP, dtype=torch.bfloat16, device=DEV)
    gain = 1 + 2 * (torch.rand(d, generator=g, device=DEV) < 0.03).float()
    step = max(1, (1 << 25) // d)
    # one block of rows is drawn, and every block of the cache is that block with its rows
    # rolled by another amount: distinct content at the cost of one draw
    n = min(rows, step)
    c0, s0 = _quantise((torch.randn(n, d, generator=g, device=DEV) * gain).bfloat16())
    for i, a in enumerate(range(0, rows, step)):
        b = min(rows, a + step)
        codes[a:b] = torch.roll(c0, 1 + 37 * i, 0)[:b - a]
        scales[a:b] = torch.roll(s0, 1 + 37 * i, 0)[:b - a]
    return codes, scales


def _prepare_attn(c, seed):
    g = _gen(seed)
    B, d, n_kv, n_new = c["batch"], c["head_dim"], c["n_kv"], c["n_new"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g, device=DEV)
    lens[0] = c["hi"]
    lens = lens.int()
    st = dict(case=c, lens=lens)
    st["q"] = torch.randn(B, n_new, c["n_q"], d, generator=g, device=DEV).bfloat16()
    if c["page"]:
        per = -(-c["hi"] // c["page"])
        n_pages = B * per + 3
        st["table"] = torch.randperm(n_pages, generator=g, device=DEV)[:B * per].int().reshape(
            B, per).contiguous()
        shape = (n_pages, n_kv, c["page"])
    else:
        st["table"] = None
        cap = -(-(c["window"] + n_new - 1) // 128) * 128 if c["kind"] == RING else \
            -(-c["hi"] // 64) * 64
        shape = (B, n_kv, cap)
    rows = shape[0] * shape[1] * shape[2]
    for n in ("k",) if c["k_eq_v"] else ("k", "v"):
        codes, scales = _cache(g, rows, d)
        st[n + "c"], st[n + "s"] = codes.reshape(*shape, -1), scales.reshape(*shape, -1)
    if c["k_eq_v"]:
        st["vc"] = st["vs"] = None
    st["out"] = torch.empty_like(st["q"])
    if own:
        import mixed_sliding_global_gb300 as m
        n = m.gemma_attn_workspace_size_q4(B, c["kind"], c["window"], c["n_q"], n_kv, d, c["hi"],
                                           n_new, k_eq_v=c["k_eq_v"])
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def _prepare_append(c, seed):
    g = _gen(seed)
    B, d, n_kv, n_new = c["batch"], c["head_dim"], c["n_kv"], c["n_new"]
    cap = -(-(c["start"] + 64 + n_new) // 64) * 64
    st = dict(case=c)
    gain = 1 + 2 * (torch.rand(d, generator=g, device=DEV) < 0.03).float()
    for n in ("k",) if c["k_eq_v"] else ("k", "v"):
        st[n] = (torch.randn(B, n_new, n_kv, d, generator=g, device=DEV) * gain).bfloat16()
        st[n + "c"] = torch.zeros(B, n_kv, cap, d // 2, dtype=torch.uint8, device=DEV)
        st[n + "s"] = torch.zeros(B, n_kv, cap, d // GROUP, dtype=torch.bfloat16, device=DEV)
        st[n + "o"] = torch.empty_like(st[n])
    if c["k_eq_v"]:
        st["v"] = st["vc"] = st["vs"] = st["vo"] = None
    st["pos"] = (c["start"] + torch.randint(0, 64, (B,), generator=g, device=DEV)).int()
    if own:
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def _prepare_sample(c, seed):
    g = _gen(seed)
    B, V = c["batch"], c["vocab"]
    x = 8 * torch.randn(B, V, generator=g, device=DEV)       # most inside the cap of 30
    if c["dtype"] == "bf16":
        x = x.bfloat16()
    f = dict(dtype=torch.float32, device=DEV)
    st = dict(case=c, x=x, u=torch.rand(B, generator=g, **f))
    if c["mixed"]:    # every request of the batch brings its own filters
        def pick(vals):
            return torch.tensor(vals, **f)[torch.randint(0, len(vals), (B,), generator=g,
                                                         device=DEV)]
        st["t"] = pick([0.6, 0.8, 1.0, 1.2])
        st["k"] = pick([0, 40, 64, 200]).int()
        st["p"] = pick([1.0, 0.95, 0.9, 0.5])
        st["m"] = pick([0.0, 0.0, 0.05])
    else:
        st["t"] = torch.full((B,), c["temperature"], **f)
        st["k"] = torch.full((B,), c["top_k"], dtype=torch.int32, device=DEV)
        st["p"] = torch.full((B,), c["top_p"], **f)
        st["m"] = torch.full((B,), c["min_p"], **f)
    st["out"] = torch.empty(B, dtype=torch.int32, device=DEV)
    if own:
        import mixed_sliding_global_gb300 as m
        n = m.gemma_logit_sample_workspace_size(B, V, x.dtype)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


def prepare(case, seed):
    return {"attn": _prepare_attn, "append": _prepare_append,
            "sample": _prepare_sample}[case["op"]](case, seed)


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def _positions(c, lens):
    """First position that each sequence's step may read, and how many positions are laid out."""
    if c["kind"] == GLOBAL:
        return torch.zeros_like(lens), c["hi"]
    first = (lens - c["n_new"] - c["window"] + 1).clamp_min(0)
    return first, min(c["hi"], c["window"] + c["n_new"] - 1)


def _rows(st, codes, scales, pos):
    """Values [B][n_kv][N][d] of positions pos [B][N]."""
    c = st["case"]
    B = pos.shape[0]
    if st["table"] is not None:
        page = torch.gather(st["table"].long(), 1, (pos // c["page"]).clamp_max(
            st["table"].shape[1] - 1))
        a, s = codes[page, :, pos % c["page"]], scales[page, :, pos % c["page"]]
    else:
        b = torch.arange(B, device=pos.device)[:, None]
        slot = pos % codes.shape[2] if c["kind"] == RING else pos.clamp_max(codes.shape[2] - 1)
        a, s = codes[b, :, slot], scales[b, :, slot]
    return _values(a, s).transpose(1, 2)                     # from [B][N][n_kv][d]


def _plain_attn(st):
    c = st["case"]
    B, n_new, n_q, d = st["q"].shape
    n_kv, G = c["n_kv"], c["n_q"] // c["n_kv"]
    lens = st["lens"].long()
    first, N = _positions(c, lens)
    pos = first[:, None] + torch.arange(N, device=DEV)                        # [B][N]
    k = _rows(st, st["kc"], st["ks"], pos)
    v = k if c["k_eq_v"] else _rows(st, st["vc"], st["vs"], pos)
    q = st["q"].float().reshape(B, n_new, n_kv, G, d).permute(0, 2, 3, 1, 4).reshape(
        B, n_kv, G * n_new, d)
    s = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    at = lens[:, None] - n_new + torch.arange(n_new, device=DEV)              # [B][n_new]
    ok = pos[:, None, :] <= at[:, :, None]
    if c["kind"] != GLOBAL:
        ok &= at[:, :, None] - pos[:, None, :] < c["window"]
    s = s.reshape(B, n_kv, G, n_new, N).masked_fill(~ok[:, None, None], -math.inf)
    s = s - s.amax(-1, keepdim=True)
    p = torch.exp(s)
    p = (p / p.sum(-1, keepdim=True)).reshape(B, n_kv, G * n_new, N)
    o = (p @ v).reshape(B, n_kv, G, n_new, d).permute(0, 3, 1, 2, 4).reshape(B, n_new, n_q, d)
    return o.bfloat16()


def _own_attn(st):
    import mixed_sliding_global_gb300 as m
    c = st["case"]
    m.gemma_attn_q4(st["out"], st["q"], [st["kc"]], [st["ks"]], [st["vc"]], [st["vs"]], [0], 0,
                    st["lens"], c["hi"], kind=c["kind"], window=c["window"], n_kv=c["n_kv"],
                    k_eq_v=c["k_eq_v"], scale=1 / math.sqrt(c["head_dim"]), softcap=c["softcap"],
                    block_table=st["table"], workspace=st["ws"], device_error=st["err"])
    return st["out"]


def _plain_append(st):
    """Quantise the new rows, place them, and read them back as bf16 values."""
    c = st["case"]
    out = {}
    B, n_kv = c["batch"], c["n_kv"]
    b = torch.arange(B, device=DEV)[:, None, None]
    h = torch.arange(n_kv, device=DEV)[None, None, :]
    slot = (st["pos"].long()[:, None] + torch.arange(c["n_new"], device=DEV))[:, :, None]
    for n in ("k",) if c["k_eq_v"] else ("k", "v"):
        codes, scales = _quantise(st[n])
        st[n + "c"][b, h, slot] = codes
        st[n + "s"][b, h, slot] = scales
        out[n] = _values(st[n + "c"][b, h, slot], st[n + "s"][b, h, slot]).bfloat16()
    return out


def _own_append(st):
    import mixed_sliding_global_gb300 as m
    c = st["case"]
    kw = dict(k_eq_v=c["k_eq_v"], device_error=st["err"])
    m.gemma_kv_append_q4([st["kc"]], [st["ks"]], [st["vc"]], [st["vs"]], [0], 0, st["k"], st["v"],
                         st["pos"], **kw)
    m.gemma_kv_read_q4([st["kc"]], [st["ks"]], [st["vc"]], [st["vs"]], [0], 0, st["ko"], st["vo"],
                       st["pos"], **kw)
    return {"k": st["ko"]} if c["k_eq_v"] else {"k": st["ko"], "v": st["vo"]}


def _plain_sample(st):
    """In 64 bits: cumulative weights next to u and top_p decide whole numbers."""
    c = st["case"]
    B, V = st["x"].shape
    z = st["x"].double()
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    _, order = torch.sort(st["x"].float(), dim=-1, descending=True, stable=True)
    zs = torch.gather(z, 1, order)
    rank = torch.arange(V, device=DEV)
    k = torch.where(st["k"] > 0, st["k"], V).long()[:, None]
    w = torch.exp((zs - zs[:, :1]) / st["t"].double()[:, None])
    w = w * (rank < k)
    cum = torch.cumsum(w, -1)
    reach = cum < st["p"].double()[:, None] * cum[:, -1:]
    keep = torch.ones_like(reach)
    keep[:, 1:] = reach[:, :-1]                # kept while the mass before it is short of top_p
    keep |= st["p"][:, None] >= 1
    keep &= (w >= st["m"].double()[:, None]) & (rank < k)
    cum = torch.cumsum(w * keep, -1)
    hit = (cum > st["u"].double()[:, None] * cum[:, -1:]) & keep
    return torch.gather(order, 1, hit.int().argmax(-1, keepdim=True))[:, 0].int()


def _own_sample(st):
    import mixed_sliding_global_gb300 as m
    m.gemma_logit_sample(st["x"], st["out"], st["u"], temperature=st["t"], top_k=st["k"],
                         top_p=st["p"], min_p=st["m"], softcap=st["case"]["softcap"],
                         workspace=st["ws"], device_error=st["err"])
    return st["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _own_attn, "append": _own_append, "sample": _own_sample}[op](state)
    return {"attn": _plain_attn, "append": _plain_append, "sample": _plain_sample}[op](state)


# --------------------------------------------------------------------------------------------
# work and 64-bit results
# --------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "append":   # rows in, 4-bit rows out, 4-bit rows in, values out
        rows = c["batch"] * c["n_new"] * c["n_kv"] * (1 if c["k_eq_v"] else 2)
        d = c["head_dim"]
        return {"bytes": rows * (4 * d + 2 * (d // 2 + d // 32)), "flops": rows * 3 * d}
    if c["op"] == "sample":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["batch"] * (c["vocab"] * size + 24), "flops": c["batch"] * c["vocab"]}
    d, n_new, lo, hi = c["head_dim"], c["n_new"], c["lo"], c["hi"]
    # the mean over the lengths of one sequence's keys read, and of its (query, key) pairs
    lens = [hi] + [lo + (hi - lo) * (i + 0.5) / 64 for i in range(64)] * (c["batch"] > 1)
    wts = [1.0] + [(c["batch"] - 1) / 64.0] * 64
    keys = pairs = 0.0
    for n, wt in zip(lens, wts):
        if c["kind"] == GLOBAL:
            kn, pn = n, n_new * (n - (n_new - 1) / 2)
        else:
            kn = min(n, c["window"] + n_new - 1)
            # position p of the n_new last ones attends min(p + 1, window) keys
            short = min(max(c["window"] - (n - n_new), 0), n_new)
            pn = (n_new - short) * c["window"] + short * (n - n_new) + short * (short + 1) / 2
        keys += wt * kn
        pairs += wt * pn
    row = (d // 2 + d // 32) * (1 if c["k_eq_v"] else 2)
    return {"bytes": keys * c["n_kv"] * row + 4 * c["batch"] * n_new * c["n_q"] * d,
            "flops": 4.0 * pairs * c["n_q"] * d}


def _unpack64(codes, scales):
    """fp64 values of code rows [R][d/2], one byte at a time."""
    b = codes.to(torch.int64)
    bit = torch.stack([(b >> i) & 1 for i in range(8)], -1).reshape(b.shape[0], -1, 32)
    val = []
    for e in range(8):
        m0 = 4 * (e // 2) + (16 if e % 2 else 0)
        sg = (m0 + 15) % 32
        mag = bit[..., m0] + 2 * bit[..., m0 + 1] + 4 * bit[..., m0 + 2]
        val.append(torch.where(bit[..., sg] == 1, -mag, mag))
    val = torch.stack(val, -1).reshape(b.shape[0], -1, GROUP).double()
    return (val * scales.double()[..., None]).reshape(b.shape[0], -1)


def _exact_attn(c, st):
    B, n_new, n_q, d = st["q"].shape
    G = n_q // c["n_kv"]
    out = torch.zeros(B, n_new, n_q, d, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(st["lens"][b])
        first = 0 if c["kind"] == GLOBAL else max(0, n - n_new - c["window"] + 1)
        j = torch.arange(first, n, device=DEV)
        i = torch.arange(n - n_new, n, device=DEV)[:, None]
        see = (j <= i) if c["kind"] == GLOBAL else (j <= i) & (i - j < c["window"])
        if st["table"] is not None:
            where = (st["table"][b].long()[j // c["page"]], j % c["page"])
        else:
            where = (torch.full_like(j, b), j % st["kc"].shape[2])
        for h in range(c["n_kv"]):
            k = _unpack64(st["kc"][where[0], h, where[1]], st["ks"][where[0], h, where[1]])
            v = k if c["k_eq_v"] else _unpack64(st["vc"][where[0], h, where[1]],
                                                st["vs"][where[0], h, where[1]])
            for r in range(h * G, h * G + G):
                s = st["q"][b, :, r].double() @ k.T / math.sqrt(d)
                if c["softcap"]:
                    s = torch.tanh(s / c["softcap"]) * c["softcap"]
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                out[b, :, r] = torch.softmax(s, -1) @ v
    return out


def _exact_append(c, st):
    out = {}
    for n in ("k",) if c["k_eq_v"] else ("k", "v"):
        x = st[n].double().reshape(-1, GROUP)
        top = x.abs().max(-1).values
        # the smallest j * 2^e (16 <= j < 32) that is at least top / 7
        e = torch.floor(torch.log2(top / 7)) - 4
        s = torch.full_like(top, math.inf)
        for de in (-1, 0, 1):
            unit = torch.exp2(e + de)
            j = torch.ceil(top / 7 / unit).clamp_min(16)
            s = torch.where((j <= 32) & (j * unit * 7 >= top), torch.minimum(s, j * unit), s)
        s = torch.where(top > 0, s, torch.ones_like(s))[:, None]
        out[n] = (torch.round(x / s) * s).reshape(st[n].shape)
    return out


def _exact_sample(c, st):
    import numpy as np
    B, V = st["x"].shape
    x = st["x"].double().cpu().numpy()
    par = {n: st[n].double().cpu().numpy() for n in ("u", "t", "k", "p", "m")}
    out = []
    for b in range(B):
        order = np.lexsort((np.arange(V), -x[b]))
        if par["k"][b] > 0:
            order = order[:int(par["k"][b])]
        z = x[b][order]
        if c["softcap"]:
            z = c["softcap"] * np.tanh(z / c["softcap"])
        w = np.exp((z - z[0]) / par["t"][b])
        n = len(w)
        if par["p"][b] < 1:
            total = math.fsum(w)
            n = min(n, int(np.searchsorted(np.cumsum(w), par["p"][b] * total)) + 1)
        n = min(n, int(np.count_nonzero(w >= par["m"][b])))
        cum = np.cumsum(w[:n])
        i = min(int(np.searchsorted(cum, par["u"][b] * cum[-1], side="right")), n - 1)
        out.append(int(order[i]))
    return torch.tensor(out, dtype=torch.int32)


def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append,
            "sample": _exact_sample}[case["op"]](case, st)
