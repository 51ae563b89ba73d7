"""Seeded cases of the operators that serve many continuations of one prompt (test infrastructure)."""
from __future__ import annotations

import numpy as np
import torch

from oracle import drafts as odr
from oracle import kivi as okivi
from sub_bit_quantized_gb300 import kvq
from tests import _cases as C
from tests import _drafts as T

D = 128
KIVI_ARRAYS = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "k_resid", "v_resid")
VQ_ARRAYS = ("idx_k", "idx_v", "win_k", "win_v")


def prefix_reference(case: T.TreeCase, prefix: C.KiviCase, slot: int, drafts: bool = True):
    """(out, bound), both [B][N][Hq][D] fp64, of rows that attend slot ``slot`` of ``prefix``, their own cache and
    (with ``drafts``) the drafted tokens of their mask; rows of padding tokens are NaN in out.

    The roundings are those that tests/_drafts.py counts, over both contexts: elements of stored keys and values by
    2^-11 of themselves and of |s z|, scores by 2^-16 of their absolute sum, weights by 2^-11, weights below 2^-26 of
    the largest lost (the kernel for many rows takes weights up to 2^15 and lets the largest start at 2^1; half a step of
    an fp16 subnormal is 2^-25: each of n weights is off by at most 2^-26 of the largest). Joining the two parts adds a few fp32 steps to each (log2 of a sum: 2^-21 of the weight, two
    products, a sum, a reciprocal: under 2^-19 of sum p |v|), which 2^-16 of it covers together with the rest."""
    base = case.base
    B, N, Hq, _ = case.q.shape
    H = base.cfg.n_heads
    out = np.full(case.q.shape, np.nan)
    bound = np.zeros(case.q.shape)
    for h in range(H):
        K0, V0, kc0, vc0 = T.context(prefix, slot, h)
        for b in range(B):
            nd = min(max(case.n_draft[b], 0), N)
            K1, V1, kc1, vc1 = T.context(base, b, h)
            K, V = np.concatenate([K0, K1]), np.concatenate([V0, V1])
            kc, vc = np.concatenate([kc0, kc1]), np.concatenate([vc0, vc1])
            kd, vd = case.kd[b, :, h].astype(np.float64), case.vd[b, :, h].astype(np.float64)
            keys, vals = np.abs(np.concatenate([K, kd])), np.abs(np.concatenate([V, vd]))
            dk = np.concatenate([T.U16 * (np.abs(K) + kc), np.zeros_like(kd)])
            dv = np.concatenate([T.U16 * (np.abs(V) + vc), np.zeros_like(vd)])
            for hq in [x for x in range(Hq) if okivi.kv_head(x, Hq, H) == h]:
                for i in range(nd):
                    q = case.q[b, i, hq].astype(np.float64)
                    m = int(case.mask[b, i]) if drafts else 0
                    p, seen = odr.tree_weights(q, K, kd, m, nd)
                    out[b, i, hq] = odr.tree_attention(q, K, V, kd, vd, m, nd)
                    if not seen.any():
                        continue
                    f = np.expm1(((dk + 2.0 ** -16 * keys)[seen] @ np.abs(q)) / np.sqrt(D)) + T.U16
                    ps, av = p[seen], vals[seen]
                    bound[b, i, hq] = 1.1 * ((ps * (f + ps @ f)) @ av + ps @ dv[seen] +
                                             seen.sum() * 2.0 ** -26 * ps.max() * av.max() + 2.0 ** -16 * (ps @ av))
    return out, bound


def run_prefix(case: T.TreeCase, prefix: C.KiviCase, slot: int = 0, drafts: bool = True, dtype=torch.float32, fill=7.0,
               ws=None) -> np.ndarray:
    cache, pcache = C.fill_kivi_cache(case.base), C.fill_kivi_cache(prefix)
    q, kd, vd, mask, nd = T.tensors(case)
    out = torch.full(q.shape, fill, dtype=dtype, device="cuda")
    more = dict(k_draft=kd, v_draft=vd, mask=mask) if drafts else {}
    kvq.kvq_kivi_prefix_attn(case.base.cfg, cache, prefix.cfg, pcache, slot, q, out, n_draft=nd, ws=ws, **more)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    return out.double().cpu().numpy()


def dists(g, B, N, V, dtype, near=0.8, sharp=3.0):
    """Target and draft distributions of that type, and what a child of every node would be drawn from."""
    logits = sharp * torch.randn((B, N, V), generator=g)
    P = torch.softmax(logits, -1).to(dtype)
    Q = torch.softmax(logits + near * torch.randn((B, N, V), generator=g), -1).to(dtype)
    return P, Q


def tree(g, B, N, chain=False):
    parent = torch.zeros((B, N), dtype=torch.int32)
    for i in range(1, N):
        parent[:, i] = i - 1 if chain else (torch.rand(B, generator=g) ** 0.5 * i).int().clamp(max=i - 1)
    return parent


def draw_tokens(g, Q, parent):
    """Every node's token drawn from its parent's row of Q."""
    B, N, V = Q.shape
    token = torch.zeros((B, N), dtype=torch.int32)
    for i in range(N):
        rows = Q[torch.arange(B), parent[:, i].long().clamp(min=0)].double()
        token[:, i] = torch.multinomial(rows, 1, generator=g)[:, 0].int()
    return token


def run_verify(P, Q, token, parent, u, n_draft=None, fill=-7):
    """The call's outputs on the host: path [B][N], n_accept [B], next [B] (``fill`` where nothing was written)."""
    B, N, _ = P.shape
    dev = lambda x: None if x is None else x if x.is_cuda else x.cuda()  # noqa: E731
    path = torch.full((B, N), fill, dtype=torch.int32, device="cuda")
    count, nxt = (torch.full((B,), fill, dtype=torch.int32, device="cuda") for _ in range(2))
    kvq.kvq_verify_draft(dev(P), dev(Q), dev(token), dev(parent), dev(u), path, count, nxt, n_draft=dev(n_draft))
    torch.cuda.synchronize()
    return path.cpu().numpy(), count.cpu().numpy(), nxt.cpu().numpy()
