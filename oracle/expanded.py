"""Expanded-form attention and drafted-tree visibility in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Expanded form ("DeepSeek R1 Architecture & Deployment Guide", section 1.1,
before absorption): every head has its own keys and values, the RoPE part of a
key is shared by the heads.  Readings: the causal mask is aligned at the
bottom right (query i of n_q sees key j of n_k when j <= i + n_k - n_q); a
query that sees no key gives out = 0, lse = -inf.
"""
from __future__ import annotations

import numpy as np


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, see: np.ndarray, scale: float):
    """One head: q [n, d], k [m, d], v [m, e], see [n, m] bool -> out [n, e],
    lse [n], and sum_j p_j |v_j| [n, e] (what a rounding of p is worth).
    Masked keys and values take no part, whatever they hold."""
    n = q.shape[0]
    out, mag = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    lse = np.full(n, -np.inf)
    for i in range(n):
        j = np.nonzero(see[i])[0]
        if j.size == 0:
            continue
        s = scale * (k[j] @ q[i])
        m = s.max()
        e = np.exp(s - m)
        lse[i] = m + np.log(e.sum())
        p = e / e.sum()
        out[i], mag[i] = p @ v[j], p @ np.abs(v[j])
    return out, lse, mag


def prefill(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale, causal, heads):
    """float64 arrays as the entry point takes them; `heads`: those computed.
    Returns out [nq, len(heads), 128], lse [nq, len(heads)], mag like out;
    rows of no sequence are NaN."""
    nq = q_nope.shape[0]
    out = np.full((nq, len(heads), v.shape[2]), np.nan)
    mag = np.full_like(out, np.nan)
    lse = np.full((nq, len(heads)), np.nan)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        see = np.ones((q1 - q0, k1 - k0), dtype=bool)
        if causal:
            see = np.tril(see, (k1 - k0) - (q1 - q0))
        for n, h in enumerate(heads):
            q = np.concatenate([q_nope[q0:q1, h], q_rope[q0:q1, h]], -1)
            k = np.concatenate([k_nope[k0:k1, h], k_rope[k0:k1]], -1)
            out[q0:q1, n], lse[q0:q1, n], mag[q0:q1, n] = attend(q, k, v[k0:k1, h], see, scale)
    return out, lse, mag


def tree_sees(parents, n_nodes: int, i: int, ctx: int):
    """Token positions node i of a drafted tree sees: the context [0, ctx),
    itself, and its ancestors (node a is token ctx + a)."""
    if i >= n_nodes:
        return np.empty(0, dtype=np.int64)
    path, a = [], i
    while a >= 0:
        path.append(ctx + a)
        a = int(parents[a])
    return np.concatenate([np.arange(ctx), np.array(sorted(path))]).astype(np.int64)
