"""Rotary positions over three axes, fp64.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see oracle/__init__.py).

DensityKV, Supplementary "Post-RoPE Attention Geometry": the backbone rotates
queries and keys over (frame, row, column) before they reach a cache.  Reading:
pair j of an axis with n pairs turns by position * base^(-j/n); axes follow one
another over the pairs of a head, pairs past their sum are not turned.

Pins: ``tests/test_oracle_q8.py`` (the generator's own rotation, norms, inverses).
"""
from __future__ import annotations

import numpy as np


def angles(pos, axis_pairs, half: int, base: float = 10000.0) -> np.ndarray:
    """[n_tok][half] angles of pos [n_tok][3] (0 for pairs past the axes)."""
    pos = np.asarray(pos, dtype=np.float64)
    out = np.zeros((pos.shape[0], half))
    k = 0
    for axis, n in enumerate(axis_pairs):
        for j in range(n):
            out[:, k] = pos[:, axis] * np.float64(base) ** (-j / n)
            k += 1
    return out


def rope(x, pos, axis_pairs, base: float = 10000.0, halves: bool = False, inverse: bool = False) -> np.ndarray:
    """x [..., n_tok, d] turned by its tokens' angles; pairs are elements (2j, 2j+1), or
    (j, j + d/2) with ``halves``."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    a = angles(pos, axis_pairs, d // 2, base)
    if inverse:
        a = -a
    i, j = (np.arange(d // 2), np.arange(d // 2) + d // 2) if halves else (np.arange(0, d, 2), np.arange(1, d, 2))
    out = x.copy()
    turned = slice(0, sum(axis_pairs))
    c, s = np.cos(a)[:, turned], np.sin(a)[:, turned]
    p, q = x[..., i[turned]], x[..., j[turned]]
    out[..., i[turned]] = p * c - q * s
    out[..., j[turned]] = p * s + q * c
    return out
