"""The operators of a speculative step in fp64 (oracle; test infrastructure only): norm and rotation
of query and key rows, and attention of a tree of drafted tokens over a cached context.

Written from the definitions:
  rows:  y = x / sqrt(mean(x^2) + eps) * w, then the rotate-half rotation by the token's angle;
  tree:  drafted token i attends all cached tokens and the drafted tokens of its mask, one softmax.
"""
from __future__ import annotations

import numpy as np


def norm_rows(x, w, eps: float) -> np.ndarray:
    """Rows x [..][D] divided by their root mean square (of x^2 + eps) and scaled by w [D]."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rotate_rows(y, cos, sin) -> np.ndarray:
    """The pairs (i, i + D/2) of y [..][D] turned by the angles whose cos and sin [..][D/2] are given."""
    h = y.shape[-1] // 2
    a, b = y[..., :h], y[..., h:]
    c, s = np.asarray(cos, np.float64), np.asarray(sin, np.float64)
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def tree_weights(q, K, k_draft, mask: int, n_draft: int):
    """Softmax weights of one drafted query q [D] over the cached keys K [n][D] and the drafted keys
    [N][D] whose bit is set in ``mask`` (bits from n_draft on do not count).

    Returns (p [n + N], seen [n + N]): the weights, 0 where nothing is attended.
    """
    K = np.asarray(K, np.float64).reshape(-1, len(q))
    seen = np.array([True] * len(K) + [bool(mask >> j & 1) and j < n_draft for j in range(len(k_draft))], dtype=bool)
    p = np.zeros(len(seen))
    if not seen.any():
        return p, seen
    keys = np.concatenate([K, np.asarray(k_draft, np.float64)])[seen]
    s = keys @ np.asarray(q, np.float64) / np.sqrt(len(q))
    e = np.exp(s - s.max())
    p[seen] = e / e.sum()
    return p, seen


def tree_attention(q, K, V, k_draft, v_draft, mask: int, n_draft: int) -> np.ndarray:
    """Attention output [D] of one drafted query; 0 for a row that attends nothing."""
    p, seen = tree_weights(q, K, k_draft, mask, n_draft)
    vals = np.concatenate([np.asarray(V, np.float64).reshape(-1, len(q)), np.asarray(v_draft, np.float64)])
    return p[seen] @ vals[seen]
