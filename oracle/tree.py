"""Attention of a tree of drafted tokens, and keeping its accepted path — test infrastructure only.

The definition, row by row in float64: with base = kv_len - q_len, draft i sees cache slot t iff t < base,
or t < kv_len and bit t - base of mask[i] is set; o = softmax(scale q.k) v over the slots it sees.
Rows that see nothing, and rows at or past q_len, have o = 0, lse = -inf.
"""
from __future__ import annotations

import numpy as np

from .attention import as_f64


def decode_tree(q, k, v, kv_lens, mask, *, scale: float, q_lens=None, k_scale=None, v_scale=None):
    """q [B, n_q, Hq, D]; k, v [B, T, Hkv, D] values; mask [B, n_q] integers (bit sets).
    Returns (o [B, n_q, Hq, D], lse [B, n_q, Hq]) in float64."""
    q = as_f64(q)
    B, n_q, Hq, D = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    o = np.zeros((B, n_q, Hq, D))
    lse = np.full((B, n_q, Hq), -np.inf)
    for b in range(B):
        n = min(max(int(kv_lens[b]), 0), T)
        qn = n_q if q_lens is None else min(max(int(q_lens[b]), 0), n_q)
        base = n - qn
        for h in range(Hkv):
            K, V = as_f64(k[b, :n, h]), as_f64(v[b, :n, h])
            if k_scale is not None:
                K = K * as_f64(k_scale[b, :n, h])[:, None]
                V = V * as_f64(v_scale[b, :n, h])[:, None]
            for i in range(qn):
                m = int(mask[b][i])
                see = np.array([t for t in range(n) if t < base or (m >> (t - base)) & 1], dtype=np.int64)
                if see.size == 0:
                    continue
                s = scale * (q[b, i, h * G:(h + 1) * G] @ K[see].T)
                mx = s.max(axis=1, keepdims=True)
                with np.errstate(invalid="ignore"):
                    e = np.exp(s - np.where(mx == -np.inf, 0.0, mx))
                    tot = e.sum(axis=1, keepdims=True)
                    o[b, i, h * G:(h + 1) * G] = (e / tot) @ V[see]
                    lse[b, i, h * G:(h + 1) * G] = (mx + np.log(tot))[:, 0]
    return o, lse
