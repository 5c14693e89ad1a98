"""Host checks of the 4-bit cache entry points (no GPU): every refusal before any launch."""
import ctypes

import pytest
import torch

import mixed_sliding_global_gb300 as g
import q4_ref as R
from test_abi import CAPACITY, FAKE, INVALID, UNSUPPORTED, _i32, _ptrs, lib


def attn(owner=(0,), layer=0, msl=64, n=1, batch=1, kind=1, window=0, n_q=4, n_kv=1, d=64,
         k_eq_v=1, cap=64, scale=0.125, softcap=0.0, dtype=0, kc=(FAKE,), ks=(FAKE,), vc=(None,),
         vs=(None,), table=None, max_pages=0, page=0, n_pages=0, out=FAKE, q=FAKE, lens=FAKE):
    return lib().gemma_attn_q4(out, q, _ptrs(*kc), _ptrs(*ks), _ptrs(*vc), _ptrs(*vs),
                               _i32(*owner), len(owner), layer, lens, table, max_pages, page,
                               n_pages, msl, n, batch, kind, window, n_q, n_kv, d, k_eq_v, cap,
                               scale, softcap, dtype, None, 0, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(owner=(1,)), INVALID), (dict(layer=3), INVALID), (dict(n_q=6, n_kv=4), INVALID),
    (dict(n_q=32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
    (dict(kind=0, window=0), INVALID), (dict(kind=5), INVALID), (dict(msl=65), CAPACITY),
    (dict(msl=3, n=4), INVALID), (dict(n=-1), INVALID), (dict(k_eq_v=0), INVALID),
    (dict(ks=(None,)), INVALID), (dict(kc=(None,)), INVALID), (dict(kc=(FAKE + 8,)), INVALID),
    (dict(ks=(FAKE + 8,)), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(dtype=7), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=70000), UNSUPPORTED), (dict(cap=72), UNSUPPORTED),
    (dict(cap=0), INVALID), (dict(kind=2, window=64, cap=96), UNSUPPORTED),
    (dict(kind=2, window=129, cap=128), CAPACITY),
    (dict(table=FAKE, max_pages=4, page=64, n_pages=8), UNSUPPORTED),
    (dict(table=FAKE, max_pages=0, page=128, n_pages=8), INVALID),
    (dict(table=FAKE, max_pages=4, page=128, n_pages=8, kind=2, window=64), INVALID),
    (dict(table=FAKE, max_pages=1, page=128, n_pages=8, msl=129), CAPACITY),
    (dict(out=None), INVALID), (dict(q=FAKE + 4), INVALID), (dict(lens=None), INVALID),
    (dict(batch=0), 0), (dict(n=0), 0),
])
def test_attention_argument_errors(kw, status):
    assert attn(**kw) == status


def rows_call(fn, owner=(0,), layer=0, batch=1, n=1, kind=1, n_kv=1, d=64, cap=64, k_eq_v=1,
              dtype=0, kc=(FAKE,), ks=(FAKE,), vc=(None,), vs=(None,), k=FAKE, v=None, pos=FAKE,
              table=None, max_pages=0, page=0, n_pages=0):
    return getattr(lib(), fn)(_ptrs(*kc), _ptrs(*ks), _ptrs(*vc), _ptrs(*vs), _i32(*owner),
                              len(owner), layer, k, v, pos, table, max_pages, page, n_pages, batch,
                              n, kind, n_kv, d, cap, k_eq_v, dtype, None, None)


@pytest.mark.parametrize("fn", ["gemma_kv_append_q4", "gemma_kv_read_q4"])
@pytest.mark.parametrize("kw,status", [
    (dict(owner=(1,)), INVALID), (dict(batch=-1), INVALID), (dict(n=-1), INVALID),
    (dict(n=65), CAPACITY), (dict(d=80), UNSUPPORTED), (dict(cap=40), UNSUPPORTED),
    (dict(kind=2, cap=96), UNSUPPORTED), (dict(kind=9), INVALID), (dict(n_kv=0), INVALID),
    (dict(dtype=2), INVALID), (dict(k=None), INVALID), (dict(k=FAKE + 2), INVALID),
    (dict(pos=None), INVALID), (dict(k_eq_v=0), INVALID),
    (dict(k_eq_v=0, vc=(FAKE,), vs=(FAKE,)), INVALID), (dict(ks=(None,)), INVALID),
    (dict(batch=70000), UNSUPPORTED), (dict(table=FAKE, page=100, max_pages=1, n_pages=1),
                                       UNSUPPORTED),
    (dict(n=1 << 29, cap=1 << 30), UNSUPPORTED),
    (dict(batch=0), 0), (dict(n=0), 0),
])
def test_row_argument_errors(fn, kw, status):
    assert rows_call(fn, **kw) == status


def test_shared_layer_appends_nothing():
    assert rows_call("gemma_kv_append_q4", owner=(0, 0), layer=1, kc=(FAKE, None),
                     ks=(FAKE, None), vc=(None, None), vs=(None, None)) == 0


def test_workspace_size_rejects_bad_arguments():
    bad = ctypes.c_size_t(-1).value
    f = lib().gemma_attn_workspace_size_q4
    assert f(1, 1, 0, 6, 4, 64, 64, 1, 1) == bad
    assert f(1, 1, 0, 4, 1, 96, 64, 1, 1) == bad
    assert f(1, 1, 0, 4, 1, 64, 3, 4, 1) == bad
    assert f(-1, 1, 0, 4, 1, 64, 64, 1, 1) == bad
    assert f(0, 1, 0, 4, 1, 64, 64, 1, 1) == 0


def test_binding_checks_shapes_and_types():
    """The binding refuses mismatched caches before it takes a pointer."""
    codes, scales = torch.zeros(1, 1, 64, 32, dtype=torch.uint8), torch.zeros(1, 1, 64, 1).bfloat16()
    q = torch.zeros(1, 1, 4, 64).bfloat16()
    lens = torch.ones(1, dtype=torch.int32)
    kw = dict(kind=1, window=0, n_kv=1, k_eq_v=True, scale=1.0)
    with pytest.raises(TypeError):
        g.gemma_attn_q4(q, q, [codes.int()], [scales], None, None, [0], 0, lens, 64, **kw)
    with pytest.raises(ValueError):
        g.gemma_attn_q4(q, q, [codes], [scales[:, :, :32]], None, None, [0], 0, lens, 64, **kw)
    with pytest.raises(ValueError):
        g.gemma_attn_q4(q, q, [codes], [scales], None, None, [0], 0, lens.repeat(2), 64, **kw)
    with pytest.raises(ValueError):   # K and V caches missing
        g.gemma_attn_q4(q, q, [codes], [scales], None, None, [0], 0, lens, 64,
                        **{**kw, "k_eq_v": False})
    x = torch.zeros(2, 1, 1, 64).bfloat16()
    with pytest.raises(ValueError):   # two sequences, a cache of one
        g.gemma_kv_append_q4([codes], [scales], None, None, [0], 0, x, None,
                             torch.zeros(2, dtype=torch.int32), k_eq_v=True)
    with pytest.raises(ValueError):   # CPU tensors
        g.gemma_attn_q4(q, q, [codes], [scales], None, None, [0], 0, lens, 64, **kw)


@pytest.mark.parametrize("owner,layer", [([1, 1], 0), ([0, 0, 1], 2), ([0], 1), ([0], -1), ([-1], 0)])
def test_binding_refuses_bad_owner_maps(owner, layer):
    """As the C entry points do, whatever the caches hold."""
    codes, scales = torch.zeros(1, 1, 64, 32, dtype=torch.uint8), torch.zeros(1, 1, 64, 1).bfloat16()
    q = torch.zeros(1, 1, 4, 64).bfloat16()
    n = len(owner)
    with pytest.raises(g.GemmaError) as e:
        g.gemma_attn_q4(q, q, [codes] * n, [scales] * n, None, None, owner, layer,
                        torch.ones(1, dtype=torch.int32), 64, kind=1, window=0, n_kv=1,
                        k_eq_v=True, scale=1.0)
    assert e.value.status == INVALID
    with pytest.raises(g.GemmaError) as e:
        g.gemma_kv_read_q4([codes] * n, [scales] * n, None, None, owner, layer, q[:, :, :1], None,
                           torch.zeros(1, dtype=torch.int32), k_eq_v=True)
    assert e.value.status == INVALID


def test_reference_format():
    """The tests' quantiser: 7 s >= max > 7 (s minus a step), codes in range, values exact in
    bf16, and packing round-trips."""
    gen = torch.Generator().manual_seed(1)
    x = (torch.randn(20, 256, generator=gen) *
         torch.exp2(torch.randint(-40, 40, (20, 1), generator=gen).float())).bfloat16()
    code, s = R.quantise(x)
    assert code.abs().max() == 7
    top = x.double().abs().reshape(20, 4, 64).amax(-1)
    assert (7 * s >= top).all() and (7 * s * 15 / 16 <= top).all()
    val = code.double() * s.repeat_interleave(64, -1)
    assert torch.equal(val.bfloat16().double(), val)
    assert (val - x.double()).abs().le(s.repeat_interleave(64, -1) / 2).all()
    assert torch.equal(R.values(R.pack(code, torch.signbit(x)), s.bfloat16()), val)


def test_misaligned_words_are_refused():
    """Positions, lengths, block tables and the error word are read and added to as 32-bit words."""
    args = lambda **kw: {**dict(batch=1, table=None, pos=FAKE, err=FAKE), **kw}  # noqa: E731
    paged = dict(max_pages=4, page=128, n_pages=8)

    def rows(fn, batch, table, pos, err):
        p = paged if table else dict(max_pages=0, page=0, n_pages=0)
        return getattr(lib(), fn)(_ptrs(FAKE), _ptrs(FAKE), _ptrs(None), _ptrs(None), _i32(0), 1, 0,
                                  FAKE, None, pos, table, *p.values(), batch, 1, 1, 1, 64, 64, 1, 0,
                                  err, None)

    def attention(batch, table, pos, err):
        p = paged if table else dict(max_pages=0, page=0, n_pages=0)
        return lib().gemma_attn_q4(FAKE, FAKE, _ptrs(FAKE), _ptrs(FAKE), _ptrs(None), _ptrs(None),
                                   _i32(0), 1, 0, pos, table, *p.values(), 64, 1, batch, 1, 0, 4, 1,
                                   64, 1, 64, 0.125, 0.0, 0, None, 0, err, None)

    for bad in (dict(pos=FAKE + 2), dict(table=FAKE + 1), dict(err=FAKE + 3), dict(err=FAKE + 2)):
        assert attention(**args(**bad)) == INVALID, bad
        for fn in ("gemma_kv_append_q4", "gemma_kv_read_q4"):
            assert rows(fn, **args(**bad)) == INVALID, (fn, bad)


@pytest.mark.parametrize("owner,layer", [([1, 1], 0), ([0, 0, 1], 2), ([0], 1), ([0, 1], -1), ([-1], 0)])
def test_binding_append_refuses_bad_owner_maps(owner, layer):
    """A layer that shares a cache writes nothing; one that no map describes is refused, as by the C
    entry point."""
    codes, scales = torch.zeros(1, 1, 64, 32, dtype=torch.uint8), torch.zeros(1, 1, 64, 1).bfloat16()
    x, pos, n = torch.zeros(1, 1, 1, 64).bfloat16(), torch.zeros(1, dtype=torch.int32), len(owner)
    with pytest.raises(g.GemmaError) as e:
        g.gemma_kv_append_q4([codes] * n, [scales] * n, None, None, owner, layer, x, None, pos,
                             k_eq_v=True)
    assert e.value.status == INVALID
    g.gemma_kv_append_q4([codes, None], [scales, None], None, None, [0, 0], 1, x, None, pos,
                         k_eq_v=True)
    g.gemma_kv_append_q4([codes, None], [scales, None], None, None, [0, 0], 1, None, None, None,
                         k_eq_v=True)


@pytest.mark.parametrize("kw", [dict(batch=65536), dict(n_q=32768, n_kv=32768),
                                dict(msl=(1 << 30) + 64, cap=1 << 30),
                                dict(n=100, msl=1 << 27, cap=1 << 30),
                                dict(n=100, kind=0, window=1 << 27, msl=1 << 28, cap=1 << 30)])
def test_workspace_size_refuses_what_the_call_refuses(kw):
    a = {**dict(batch=1, kind=1, window=0, n_q=4, n_kv=2, d=512, msl=64, n=1, cap=64), **kw}
    assert attn(**a) in (UNSUPPORTED, CAPACITY, INVALID)
    size = lib().gemma_attn_workspace_size_q4
    shape = [a[k] for k in ("batch", "kind", "window", "n_q", "n_kv", "d", "msl", "n")]
    assert size(*shape, 1) == ctypes.c_size_t(-1).value
    shape[0] = 0      # (the limits of a call without sequences are the same)
    if "batch" not in kw:
        assert size(*shape, 1) == ctypes.c_size_t(-1).value
