"""64-bit definition of the sampling step for the tests (numpy, no package code): one row at a time,
by sorting."""
from __future__ import annotations

import math

import numpy as np


def sample_row(x, u, t=1.0, k=0, p=1.0, m=0.0, softcap=0.0) -> int:
    """x: the row's logits as fp64 (NaN and -inf allowed)."""
    if not (t >= 0 and math.isfinite(t)) or p != p or m != m or not 0 <= u < 1:
        return -1
    idx = np.nonzero(~np.isnan(x) & (x != -np.inf))[0]
    if len(idx) == 0:
        return -1
    order = idx[np.argsort(-x[idx], kind="stable")]
    if t == 0:
        return int(order[0])
    if k > 0:
        order = order[:k]
    z = x[order]
    if softcap:
        z = softcap * np.tanh(z / softcap)
    if np.isinf(z[0]):
        w = (z == np.inf).astype(np.float64)
    else:
        with np.errstate(over="ignore"):
            w = np.exp((z - z[0]) / t)
    n = len(w)
    if p <= 0:
        n = 1
    elif p < 1:
        cum = np.cumsum(w)
        n = int(np.searchsorted(cum, p * cum[-1])) + 1
    if m > 0:
        n = min(n, max(int(np.count_nonzero(w >= m)), int(np.count_nonzero(x[order] == x[order[0]]))))
    cum = np.cumsum(w[:n])
    return int(order[min(int(np.searchsorted(cum, u * cum[-1], side="right")), n - 1)])
