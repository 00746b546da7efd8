"""fp64 CPU oracle of causal softmax attention with grouped heads over packed sequences.

TEST INFRASTRUCTURE ONLY, like moe_oracle: it imports nothing from the product package.

The Swiftlet pages say that the layers which are not Gated DeltaNet (one quarter) keep a
growing key/value cache («Paquets Swiftlet 80B Qwen dans Mac…», xix.ai, paragraph 6): softmax
attention.  The queries of a sequence are its last tokens, so query i of n with len keys sees
the keys 0 .. len - n + i.
"""
from __future__ import annotations

import numpy as np


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """One sequence.  q [n, H_q, d], k and v [len, H_kv, d] (float64).
    Returns (out, mass): out [n, H_q, d], and mass = sum_j p_ij |v_j|, the size that an error
    in the weights p is relative to.  A query that sees no key gives zeros."""
    n, Hq, d = q.shape
    length, Hkv, _ = k.shape
    assert Hq % Hkv == 0
    out, mass = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    last = length - n + np.arange(n)  # the last key that each query sees
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
        for i0 in range(0, n, 1024):
            rows = np.arange(i0, min(i0 + 1024, n))
            rows = rows[last[rows] >= 0]
            if not len(rows):
                continue
            x = scale * (q[rows, h] @ kh.T)
            hidden = np.arange(length)[None, :] > last[rows][:, None]
            x[hidden] = -np.inf
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[rows, h] = p @ vh
            mass[rows, h] = p @ np.abs(vh)
    return out, mass
