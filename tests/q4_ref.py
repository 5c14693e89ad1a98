"""64-bit definitions of the 4-bit KV cache for the tests (CPU, no package code).

Quantiser, dequantiser and attention are written from the format's and the operator's
definitions, in fp64, one sequence and head at a time.
"""
from __future__ import annotations

import math

import torch

GROUP = 64
SLIDING, GLOBAL, RING = 0, 1, 2


def scale_of(top: float) -> float:
    """The smallest number of at most five significant bits, >= 2^-126, with 7 s >= top
    (capped where 7 s would leave bf16's range; the largest code is then still 7)."""
    if top == 0:
        return 0.0
    if not math.isfinite(top):
        return math.nan
    e = math.frexp(top / 7)[1] - 5          # 16 * 2^e <= top / 7 < 32 * 2^e (within rounding)
    best = math.inf
    for de in (-1, 0, 1):
        for j in range(16, 33):
            s = math.ldexp(j, e + de)
            if 7 * s >= top and s < best:   # 7 s is exact in fp64
                best = s
    return min(max(best, 2.0 ** -126), 1.125 * 2.0 ** 125)   # 7 s finite in bf16


def quantise(x: torch.Tensor):
    """x [..., d] -> (signed codes int64 [..., d], scales fp64 [..., d / 64])."""
    d = x.shape[-1]
    g = x.double().reshape(*x.shape[:-1], d // GROUP, GROUP)
    top = g.abs().amax(-1)
    top = torch.where(torch.isfinite(g).all(-1), top, torch.full_like(top, math.inf))
    s = torch.tensor([scale_of(t) for t in top.flatten().tolist()],
                     dtype=torch.float64).reshape(top.shape)
    ok = (s > 0)
    q = torch.where(ok[..., None], g / torch.where(ok, s, torch.ones_like(s))[..., None],
                    torch.zeros_like(g))
    return torch.round(q).long().reshape(x.shape), s


def pack(codes: torch.Tensor, negative: torch.Tensor) -> torch.Tensor:
    """Signed codes [..., d] and the elements' signs -> bytes [..., d / 2]."""
    d = codes.shape[-1]
    mag = codes.abs().reshape(-1, d // 8, 8)
    neg = negative.long().reshape(-1, d // 8, 8)
    word = torch.zeros(mag.shape[:2], dtype=torch.int64)
    for e in range(8):
        m0 = 4 * (e // 2) + 16 * (e % 2)
        word += (mag[..., e] << m0) + (neg[..., e] << ((m0 + 15) % 32))
    byte = torch.stack([(word >> (8 * i)) & 255 for i in range(4)], -1).to(torch.uint8)
    return byte.reshape(*codes.shape[:-1], d // 2)


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values of packed rows: codes uint8 [..., d / 2], scales bf16 [..., d / 64]."""
    b = codes.long().reshape(*codes.shape[:-1], -1, 4)
    word = b[..., 0] + (b[..., 1] << 8) + (b[..., 2] << 16) + (b[..., 3] << 24)
    out = []
    for e in range(8):
        m0 = 4 * (e // 2) + 16 * (e % 2)
        m, n = (word >> m0) & 7, (word >> ((m0 + 15) % 32)) & 1
        out.append(torch.where(n == 1, -m, m))
    v = torch.stack(out, -1).reshape(*scales.shape, GROUP).double()
    return (v * scales.double()[..., None]).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def locate(j, b, kind, cap, table=None, page=0):
    """(leading index, slot) of position(s) j of sequence b in a [rows][n_kv][slots] cache."""
    if table is not None:
        return table[b].long()[j // page], j % page
    return torch.full_like(j, b), (j % cap if kind == RING else j)


def attention(q, k, v, lens, kind, window, scale, softcap=0.0, table=None, page=0):
    """q [B][n][n_q][d]; k, v: fp64 values [rows][n_kv][slots][d]. Returns (out, weight of the
    rounding terms sum_j p_j |v_j|), both fp64 [B][n][n_q][d]; invalid sequences give zeros."""
    B, n, n_q, d = q.shape
    n_kv, cap = k.shape[1], k.shape[2]
    out = torch.zeros(B, n, n_q, d, dtype=torch.float64)
    mass = torch.zeros_like(out)
    for b in range(B):
        L = int(lens[b])
        if L < n:
            continue
        for i in range(n):
            p = L - n + i
            lo = 0 if kind == GLOBAL else max(0, p - window + 1)
            at, slot = locate(torch.arange(lo, p + 1), b, kind, cap, table, page)
            for h in range(n_kv):
                G = n_q // n_kv
                kk, vv = k[at, h, slot], v[at, h, slot]
                s = q[b, i, h * G:(h + 1) * G].double() @ kk.T * scale
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                w = torch.softmax(s, -1)
                out[b, i, h * G:(h + 1) * G] = w @ vv
                mass[b, i, h * G:(h + 1) * G] = w @ vv.abs()
    return out, mass
