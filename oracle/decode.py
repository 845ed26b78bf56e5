"""Attention of one query token per sequence over explicit keys, in fp64.

S_j = scale q.k_j, LSE = ln sum_j exp(S_j), O = sum_j exp(S_j - LSE) v_j; query
head h reads KV head h / G.  No key: O = 0, LSE = -inf.
"""
from __future__ import annotations

import numpy as np


def attend_one(q, k, v, scale):
    """q [Hq][d], k and v [tokens][Hkv][d] -> (o [Hq][d], lse [Hq], spread [Hq][d]),
    spread = sum_j p_j |v_j|, the size that roundings of p are measured by."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    Hq, d = q.shape
    if not len(k):
        return np.zeros((Hq, d)), np.full(Hq, -np.inf), np.zeros((Hq, d))
    G = Hq // k.shape[1]
    k, v = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    s = scale * np.einsum("hd,jhd->hj", q, k)
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    total = e.sum(axis=1, keepdims=True)
    p = e / total
    return (np.einsum("hj,jhd->hd", p, v), (m + np.log(total))[:, 0],
            np.einsum("hj,jhd->hd", p, np.abs(v)))
