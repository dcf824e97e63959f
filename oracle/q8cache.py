"""The 8-bit cache with block scales, its attention, weights and eviction, fp64.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see oracle/__init__.py).

Forcing-KV's reading notes combine the method with FP8; the reading here is K and V
held as E4M3 codes times one scale per block of tokens and head, the scale the
smallest power of two that keeps the block's values within the format.  One head at
a time; codes are held as the values they stand for.

Pins: ``tests/test_oracle_q8.py``.
"""
from __future__ import annotations

import numpy as np

from .fp8 import MAX_E4M3, e4m3

MIN_EXP, MAX_EXP = -100, 119


def block_scale(x) -> float:
    """2^e, the smallest with max|x| / 2^e <= 448 over the finite values of x, e in [-100, 119]."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    m = x[np.isfinite(x)].max(initial=0.0)
    e = MIN_EXP
    while e < MAX_EXP and m > MAX_E4M3 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def encode(x, scale: float) -> np.ndarray:
    """The E4M3 value nearest to x / scale; infinities saturate, NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    q = e4m3(np.clip(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf) / scale, -MAX_E4M3, MAX_E4M3))
    return np.where(np.isnan(x), np.nan, q)


def append(codes, scales, block: int, start: int, x):
    """codes [cap][d] (values of codes), scales [cap/block] with rows x [n][d] written at
    start: new arrays."""
    codes, scales = codes.copy(), scales.copy()
    end = start + len(x)
    for b in range(start // block, -(-end // block)):
        lo, hi = max(b * block, start), min((b + 1) * block, end)
        new = x[lo - start:hi - start]
        s = block_scale(new)
        if lo > b * block:
            if scales[b] >= s:
                s = scales[b]
            else:
                codes[b * block:lo] = encode(codes[b * block:lo] * scales[b], s)
        scales[b] = s
        codes[lo:hi] = encode(new, s)
    return codes, scales


def values(codes, scales, block: int, n: int) -> np.ndarray:
    return codes[:n] * np.repeat(scales, block)[:n, None]


def attend(Q, K, V, scale: float):
    """(O, lse, weighted mean of |V|) of rows Q over the held K, V; zeros and -inf without a token."""
    Q = np.asarray(Q, dtype=np.float64)
    if len(K) == 0:
        return np.zeros((len(Q), Q.shape[1])), np.full(len(Q), -np.inf), np.zeros((len(Q), Q.shape[1]))
    S = Q @ K.T * scale
    m = S.max(1, keepdims=True)
    E = np.exp(S - m)
    z = E.sum(1, keepdims=True)
    return E @ V / z, (m + np.log(z))[:, 0], E @ np.abs(V) / z


def mass(Q, K, scale: float, lse, decay: float = 0.0, prev=None) -> np.ndarray:
    """decay * prev + sum over rows of exp(scale q.k - lse)."""
    w = np.zeros(len(K))
    for q, z in zip(np.asarray(Q, dtype=np.float64), np.asarray(lse, dtype=np.float64)):
        if z != -np.inf:
            w += np.exp(K @ q * scale - z)
    return w if prev is None else decay * np.asarray(prev, dtype=np.float64) + w


def keep(weights, n: int, budget: int, sink: int, recent: int) -> np.ndarray:
    """Positions that stay, ascending: the first `sink`, the last `recent`, and of the
    rest those of largest weight (ties: lower position; NaN least)."""
    if n <= budget:
        return np.arange(n)
    w = np.where(np.isnan(weights[:n]), -np.inf, weights[:n]).astype(np.float64)
    nan = np.isnan(weights[:n])
    middle = sorted(range(sink, n - recent), key=lambda i: (nan[i], -w[i], i))[:budget - sink - recent]
    return np.array(sorted([*range(sink), *middle, *range(n - recent, n)]), dtype=np.int64)


def gather(codes, scales, block: int, kept):
    """Codes and scales of a cache that holds rows `kept` of this one, in that order."""
    each = scales[kept // block]
    out = codes[kept].copy()
    to = np.array([each[b:b + block].max() for b in range(0, len(kept), block)])
    for i, s in enumerate(each):
        if s != to[i // block]:
            out[i] = encode(out[i] * s, to[i // block])
    return out, to
