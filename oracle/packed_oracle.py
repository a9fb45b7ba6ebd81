"""Plain float64 oracle of the packed-token operators: append, prefill, chunk.

TEST INFRASTRUCTURE ONLY (imported by the tests). Written from the definitions,
one sequence and head at a time, in NumPy float64; it shares no code with the
library.

* rotation: pair p of a row at position pos turns by pos * inv_freq[p]; pairs
  (x[p], x[p + rot/2]), or (x[2p], x[2p + 1]) interleaved.
* causal attention: new token i of nq, nk keys in all, attends to keys
  j <= nk - nq + i with z_j = <q, k_j> / sqrt(d) (HashAttention: Semantic Sparsity
  for Faster Inference, Sec. 4 with every visible token selected); lse as in
  Nectar Eq. (3.1). A row without keys gives out = 0, lse = -inf.
"""
from __future__ import annotations

import math

import numpy as np


def rotate(x, pos, inv_freq, interleaved=False):
    """x [..., d] at position pos, rotated in its first 2 len(inv_freq) dims."""
    x = np.array(x, dtype=np.float64)
    w = np.asarray(inv_freq, dtype=np.float64)
    n = len(w)
    c, s = np.cos(float(pos) * w), np.sin(float(pos) * w)
    if interleaved:
        a, b = x[..., 0:2 * n:2].copy(), x[..., 1:2 * n:2].copy()
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :n].copy(), x[..., n:2 * n].copy()
        x[..., :n], x[..., n:2 * n] = a * c - b * s, a * s + b * c
    return x


def causal_attention(q, K, V):
    """q [nq, d], K and V [nk, d]: (out [nq, d], lse [nq], mag [nq, d], zmax [nq]) with
    mag = sum_j p_j |v_j| (what an error of the weights is relative to) and zmax =
    max_j sum_k |q_k K_jk| / sqrt(d) (what an error of a score is relative to)."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    (nq, d), nk = q.shape, K.shape[0]
    out, mag = np.zeros((nq, d)), np.zeros((nq, d))
    lse, zmax = np.full(nq, -math.inf), np.zeros(nq)
    for i in range(nq):
        n = nk - nq + i + 1
        if n <= 0:
            continue
        z = K[:n] @ q[i] / math.sqrt(d)
        top = z.max()
        w = np.exp(z - top)
        out[i] = w @ V[:n] / w.sum()
        mag[i] = w @ np.abs(V[:n]) / w.sum()
        lse[i] = top + math.log(w.sum())
        zmax[i] = (np.abs(K[:n]) @ np.abs(q[i])).max() / math.sqrt(d)
    return out, lse, mag, zmax


def page_rows(pool, table_row, n):
    """The first n tokens [n, d] of a sequence from one head's pool [n_pages, page_size, d]."""
    ps = pool.shape[1]
    return np.stack([pool[table_row[i // ps], i % ps] for i in range(n)]) if n else pool[:0, 0]
