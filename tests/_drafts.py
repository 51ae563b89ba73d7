"""Seeded cases of the speculative step (test infrastructure): a KIVI cache with drafted tokens
beside it, the fp64 result of every row, and how far rounding may take the kernel from it."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

import synth
from oracle import drafts as odr
from oracle import kivi as okivi
from sub_bit_quantized_gb300 import kvq
from tests import _cases as C

D = 128
U16 = 2.0 ** -11   # half a step of fp16, relative


@dataclass
class TreeCase:
    base: C.KiviCase
    q: np.ndarray        # [B][N][Hq][D] bf16 values
    kd: np.ndarray       # [B][N][H][D] fp16
    vd: np.ndarray
    mask: np.ndarray     # [B][N] uint64
    n_draft: list


def random_masks(g, B, N) -> np.ndarray:
    """Ancestor masks of random trees: node i sees itself and what its parent (or nothing) sees."""
    m = np.zeros((B, N), np.uint64)
    for b in range(B):
        for i in range(N):
            parent = int(g.integers(-1, i)) if i else -1
            m[b, i] = (m[b, parent] if parent >= 0 else np.uint64(0)) | np.uint64(1 << i)
    return m


def make_tree_case(seed, B, H, N, n_quant, n_resid, rep=1, n_draft=None, k_bits=2, v_bits=2, residual=128,
                   max_tokens=None, n_quant_v=None, q_scale=1.0) -> TreeCase:
    base = C.make_kivi_case(seed, B, H, n_quant, n_resid, max_tokens=max_tokens, residual=residual, Hq=H * rep,
                            k_bits=k_bits, v_bits=v_bits, n_quant_v=n_quant_v)
    g = synth.rng(seed + 1000)
    q = synth.bf16_round(synth.gaussian(g, (B, N, H * rep, D)) * q_scale)
    kd = np.asarray(synth.gaussian(g, (B, N, H, D)), np.float16)
    vd = np.asarray(synth.gaussian(g, (B, N, H, D)), np.float16)
    return TreeCase(base, q, kd, vd, random_masks(g, B, N), [N] * B if n_draft is None else list(n_draft))


def context(case: C.KiviCase, b: int, h: int):
    """Cached keys and values [n][D] in fp64 and |s z| of their quantized elements (0 in fp16 rows)."""
    n, nqk, nqv = case.n_tok[b], case.n_quant_k[b], case.n_quant_v[b]
    ks, kz = case.k_scale[b, h, :nqk // 32], case.k_zero[b, h, :nqk // 32]
    vs, vz = case.v_scale[b, h, :nqv], case.v_zero[b, h, :nqv]
    K = np.concatenate([okivi.dequantize_keys(case.k_codes[b, h, :nqk], ks, kz) if nqk else np.zeros((0, D)),
                        case.k_res[b, h, :n - nqk].astype(np.float64)])
    V = np.concatenate([okivi.dequantize_values(case.v_codes[b, h, :nqv], vs, vz) if nqv else np.zeros((0, D)),
                        case.v_res[b, h, :n - nqv].astype(np.float64)])
    kc, vc = np.zeros_like(K), np.zeros_like(V)
    kc[:nqk] = np.repeat(np.abs(ks.astype(np.float64) * kz.astype(np.float64)), 32, axis=0)
    vc[:nqv] = np.repeat(np.abs(vs.astype(np.float64) * vz.astype(np.float64)), 32, axis=1)
    return K, V, kc, vc


def reference(case: TreeCase):
    """(out, bound), both [B][N][Hq][D] fp64; rows of padding tokens are NaN in out.

    The bound follows the roundings. A dequantized element X = s q - s z enters as fp16: at most
    2^-11 |X| for the result and 2^-11 |s z| for the constant. (With few rows the keys enter as
    exact codes and q_d s as fp16, in the codes' sum and the zero-points': 2^-11 |q_d X|, less.) A
    score is off by
      e_t = (sum_d |q_d| dK_td + 2^-16 sum_d |q_d K_td|) / sqrt(D)
    (q is exact in fp16 after its power-of-two scaling up to 2^-24 of its largest element, fp32
    accumulation of 128 products stays under 2^-17 of the absolute sum: 2^-16 covers both and the
    fp32 steps of the exponent). Weights are off by the factor exp(+-e_t), by 2^-11 for their own
    fp16 rounding, and by 2^-30 of the largest where they are subnormal there; normalising adds the
    sum's mean error, which gives
      |do_d| <= sum_t p_t (f_t + f_mean) |v_td| + sum_t p_t dV_td + n 2^-30 pmax max|v| + 2^-16 sum p |v|,
    f_t = expm1(e_t) + 2^-11, f_mean = sum_t p_t f_t (second-order terms: a factor 1.1).
    """
    base = case.base
    B, N, Hq, _ = case.q.shape
    H = base.cfg.n_heads
    out = np.full(case.q.shape, np.nan)
    bound = np.zeros(case.q.shape)
    for b in range(B):
        nd = min(max(case.n_draft[b], 0), N)
        for h in range(H):
            K, V, kc, vc = context(base, b, h)
            kd, vd = case.kd[b, :, h].astype(np.float64), case.vd[b, :, h].astype(np.float64)
            keys, vals = np.abs(np.concatenate([K, kd])), np.abs(np.concatenate([V, vd]))
            dk = np.concatenate([U16 * (np.abs(K) + kc), np.zeros_like(kd)])
            dv = np.concatenate([U16 * (np.abs(V) + vc), np.zeros_like(vd)])
            for hq in [x for x in range(Hq) if okivi.kv_head(x, Hq, H) == h]:
                for i in range(nd):
                    q = case.q[b, i, hq].astype(np.float64)
                    p, seen = odr.tree_weights(q, K, kd, int(case.mask[b, i]), nd)
                    out[b, i, hq] = odr.tree_attention(q, K, V, kd, vd, int(case.mask[b, i]), nd)
                    if not seen.any():
                        continue
                    aq = np.abs(q)
                    f = np.expm1(((dk + 2.0 ** -16 * keys)[seen] @ aq) / np.sqrt(D)) + U16
                    ps, av = p[seen], vals[seen]
                    bound[b, i, hq] = 1.1 * ((ps * (f + ps @ f)) @ av + ps @ dv[seen] +
                                             seen.sum() * 2.0 ** -30 * ps.max() * av.max() + 2.0 ** -16 * (ps @ av))
    return out, bound


def tensors(case: TreeCase):
    """GPU tensors of the drafted tokens: q, k_draft, v_draft, mask, n_draft."""
    return (C.bf16_tensor(case.q), C.fp16_tensor(case.kd), C.fp16_tensor(case.vd),
            torch.from_numpy(case.mask.view(np.int64)).cuda(), torch.tensor(case.n_draft, dtype=torch.int32).cuda())


def check_rows(got: np.ndarray, ref: np.ndarray, bound: np.ndarray, fill: float):
    """Real rows within the bound of the reference, padding rows still ``fill``."""
    pad = np.isnan(ref)
    assert np.array_equal(got[pad], np.full(pad.sum(), fill))
    d = np.abs(got - ref)[~pad]
    assert np.isfinite(d).all()
    worst = np.max(d - bound[~pad]) if d.size else 0.0
    assert worst <= 0, f"off by {d.max():.3e}, {worst:.3e} over the bound"


def run_tree(case: TreeCase, cache=None, dtype=torch.float32, fill=7.0, ws=None) -> np.ndarray:
    cache = C.fill_kivi_cache(case.base) if cache is None else cache
    q, kd, vd, mask, nd = tensors(case)
    out = torch.full(q.shape, fill, dtype=dtype, device="cuda")
    kvq.kvq_kivi_tree_attn(case.base.cfg, cache, q, kd, vd, mask, out, n_draft=nd, ws=ws)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    return out.double().cpu().numpy()
