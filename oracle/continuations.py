"""The operators of serving many continuations of one prompt in fp64 (oracle; test infrastructure only):
slots of a cache that continue others, and verification of drafted tokens.

Written from the definitions: a slot holds its lengths' worth of rows; speculative sampling accepts a
child of token x with probability min(1, R(x) / Q(x)) and leaves the residual max(0, R - Q), normalised.
"""
from __future__ import annotations

import numpy as np

KEEP, FREE = -1, -2


def kivi_rows(name: str, n: int, nqk: int, nqv: int, residual: int):
    """The rows of a KIVI cache array (dimension 2) that a slot of these lengths holds."""
    if name == "v_resid":
        return [t % residual for t in range(nqv, n)]
    return list(range({"k_codes": nqk, "k_scale": nqk // 32, "k_zero": nqk // 32, "k_resid": n - nqk}.get(name, nqv)))


def vq_rows(name: str, n: int, pages: int, sink: int, recent: int):
    """The rows of a LoopVQ cache array (dimension 4) that a slot of these lengths holds."""
    if name.startswith("idx"):
        return list(range(pages))
    return list(range(min(n, sink))) + [sink + (t - sink) % (recent + 8) for t in range(sink + 8 * pages, n)]


def fork(dst: dict, src: dict, lens: dict, from_lens: dict, source, b0: int, dim: int, rows_of) -> None:
    """In place: slot b0 + i of dst (dimension ``dim`` of its arrays, rows in dimension dim + 2) becomes slot source[i]
    of src as it was; lens: arrays [slots] by name. rows_of(name, *lengths): what a slot holds."""
    old = {k: v.copy() for k, v in src.items()}
    old_lens = {k: v.copy() for k, v in from_lens.items()}
    for i, s in enumerate(source):
        at = b0 + i
        if s == FREE:
            for v in lens.values():
                v[at] = 0
        if s < 0:
            continue
        held = [int(v[s]) for v in old_lens.values()]
        for name in dst:
            rows = rows_of(name, *held)
            to, fro = np.moveaxis(dst[name], dim, 0)[at], np.moveaxis(old[name], dim, 0)[s]
            to, fro = np.moveaxis(to, dim + 1, 0), np.moveaxis(fro, dim + 1, 0)  # views: rows first
            to[rows] = fro[rows]
        for k in lens:
            lens[k][at] = old_lens[k][s]


def verify(P, Q, token, parent, u, n_draft: int):
    """One request: P, Q [N][V] (Q None: point masses), u [N] (None: arg max). Returns (path, next token)."""
    P = np.asarray(P, np.float64)
    Q = None if Q is None else np.asarray(Q, np.float64)
    if n_draft <= 0:
        return [], None
    node, path = 0, [0]
    if u is None:
        best = [int(np.argmax(np.where(np.isnan(row), -np.inf, row))) for row in P]
        for i in range(1, n_draft):
            if parent[i] == node and token[i] == best[node]:
                node = i
                path.append(i)
        return path, best[node]
    u = np.asarray(u, np.float64)
    r, z = P[0].copy(), 1.0  # the residual is r / z
    for i in range(1, n_draft):
        if parent[i] != node:
            continue
        x = token[i]
        if u[i] * z * (1.0 if Q is None else Q[node, x]) < r[x]:
            node = i
            path.append(i)
            r, z = P[i].copy(), 1.0
        elif Q is None:
            z -= r[x]
            r[x] = 0.0
        else:
            r = np.maximum(r - z * Q[node], 0.0)
            z = r.sum()
    if not r.sum() > 0:
        r = P[node]
    upto = np.cumsum(r)
    past = upto > u[0] * upto[-1]
    return path, int(np.argmax(past)) if past.any() else None
