"""Host checks of the sampling entry point (no GPU), and pins of the tests' own definition."""
import ctypes

import numpy as np
import pytest
import torch

import mixed_sliding_global_gb300 as g
from sample_ref import sample_row
from test_abi import FAKE, INVALID, UNSUPPORTED, lib

WORKSPACE = -4


def call(x=FAKE, batch=1, vocab=8, dtype=0, cap=30.0, u=FAKE, out=FAKE, ws=None, ws_bytes=0):
    return lib().gemma_logit_sample(x, batch, vocab, dtype, cap, None, None, None, None, u, out, ws,
                                    ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(vocab=0), INVALID), (dict(dtype=3), INVALID),
    (dict(cap=-1.0), INVALID), (dict(cap=float("nan")), INVALID), (dict(cap=float("inf")), INVALID),
    (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(u=None), INVALID),
    (dict(out=None), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(vocab=1048561), UNSUPPORTED),
    (dict(), WORKSPACE), (dict(dtype=1), WORKSPACE), (dict(dtype=1, ws=FAKE, ws_bytes=100), WORKSPACE),
    (dict(dtype=1, ws=FAKE + 8, ws_bytes=1 << 20), WORKSPACE), (dict(batch=0), 0),
])
def test_argument_errors(kw, status):
    assert call(**kw) == status


def test_workspace_size():
    f, bad = lib().gemma_logit_sample_workspace_size, ctypes.c_size_t(-1).value
    assert f(-1, 8, 0) == bad and f(1, 0, 0) == bad and f(1, 8, 5) == bad and f(1, 1 << 21, 0) == bad
    assert f(5, 262144, 0) == 32 and f(0, 8, 1) == 0
    assert f(4, 1000, 1) == 16 + (4 << 19)
    with pytest.raises(ValueError):
        g.gemma_logit_sample_workspace_size(1, 8, torch.float16)


def test_binding_checks_types():
    x, i, f = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    with pytest.raises(ValueError):
        g.gemma_logit_sample(x[0], i, f)
    with pytest.raises(TypeError):
        g.gemma_logit_sample(x, f, f)
    with pytest.raises(TypeError):
        g.gemma_logit_sample(x, i, f[:1])
    with pytest.raises(TypeError):
        g.gemma_logit_sample(x, i, f, top_k=f)
    with pytest.raises(TypeError):
        g.gemma_logit_sample(x, i, f, temperature=i)


def test_reference_definition():
    """Closed forms: weights 8, 4, 2, 1, 1 over fifteen... sixteenths; each cut by hand."""
    x = np.log(np.array([1.0, 8.0, 2.0, 4.0, 1.0]))
    order = [1, 3, 2, 0, 4]
    for i, edge in enumerate([0.0, 8, 12, 14, 15]):
        assert sample_row(x, (edge + 0.01) / 16) == order[i]
        assert sample_row(x, (edge - 0.01) / 16 % 1) == order[i - 1]
    assert sample_row(x, 0.999, k=2) == 3 and sample_row(x, 0.999, k=4) == 0
    assert sample_row(x, 0.999, p=0.5) == 1 and sample_row(x, 0.999, p=0.51) == 3
    assert sample_row(x, 0.999, p=0.76) == 2
    assert sample_row(x, 0.999, m=0.24) == 2 and sample_row(x, 0.999, m=0.26) == 3
    assert sample_row(x, 0.999, t=0.0) == 1
    # squared weights 64, 16, 4, 1, 1 at T = 1/2
    assert sample_row(x, 63.9 / 86, t=0.5) == 1 and sample_row(x, 64.1 / 86, t=0.5) == 3
    assert sample_row(np.full(3, -np.inf), 0.5) == -1
    assert sample_row(np.array([np.inf, 1, np.inf]), 0.6) == 2


@pytest.mark.parametrize("i", range(7))
def test_misaligned_words_are_refused(i):
    """Parameters, tokens and the error word are 32-bit words."""
    p = [FAKE + 2 if j == i else FAKE for j in range(7)]
    ws = 1 << 20
    assert lib().gemma_logit_sample(FAKE, 1, 8, 0, 30.0, p[0], p[1], p[2], p[3], p[4], p[5], FAKE, ws,
                                    p[6], None) == INVALID


def test_workspace_size_refuses_what_the_call_refuses():
    assert call(batch=65536) == UNSUPPORTED
    for dtype in (0, 1):
        assert lib().gemma_logit_sample_workspace_size(65536, 8, dtype) == ctypes.c_size_t(-1).value
        assert lib().gemma_logit_sample_workspace_size(65535, 8, dtype) >= 4 * 65535
