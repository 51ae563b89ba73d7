"""How near the attention of drafted tokens comes to fp64: the library's bound for attention (max-abs
2e-3, rel-L2 1e-3 of the fp32 output, as the decode's tests hold it) on queries as they come, and keys
and queries of unequal magnitudes within one group."""
import numpy as np
import pytest
import torch

import synth
from oracle import drafts as odr
from sub_bit_quantized_gb300 import kvq
from tests import _cases as C
from tests import _drafts as T
from tests import _layout

pytestmark = pytest.mark.gpu
D = 128


def exact(case):
    """fp64 rows [B][N][Hq][D], NaN in padding tokens."""
    out = np.full(case.q.shape, np.nan)
    H = case.base.cfg.n_heads
    rep = case.q.shape[2] // H
    for b in range(case.q.shape[0]):
        for h in range(H):
            K, V, _, _ = T.context(case.base, b, h)
            for i in range(case.n_draft[b]):
                for r in range(h * rep, (h + 1) * rep):
                    out[b, i, r] = odr.tree_attention(case.q[b, i, r], K, V, case.kd[b, :, h], case.vd[b, :, h],
                                                      int(case.mask[b, i]), case.n_draft[b])
    return out


def check_attention_bound(case, cache=None):
    ref, got = exact(case), T.run_tree(case, cache)
    real = ~np.isnan(ref)
    assert (got[~real] == 7.0).all()
    C.check_close(got[real], ref[real])
    for b in range(ref.shape[0]):  # each request by itself too
        C.check_close(got[b][real[b]], ref[b][real[b]])


SMALL, LARGE = [(1, 1), (1, 8), (2, 7), (4, 4)], [(4, 5), (3, 16), (7, 33), (2, 64)]
BITS = [(2, 2), (4, 4), (2, 4), (4, 2)]


def ragged_case(rep, N, kb, vb):
    nq, nr, nqv = [0, 32, 96, 640, 960], [1, 95, 33, 128, 128], [0, 20, 90, 640, 960]
    return T.make_tree_case(4000 + rep * 100 + N, B=5, H=2, N=N, n_quant=nq, n_resid=nr, rep=rep, k_bits=kb, v_bits=vb,
                            n_draft=[N, max(1, N - 3), N, max(1, N // 2), N], n_quant_v=nqv)


@pytest.mark.parametrize("kb,vb", BITS)
@pytest.mark.parametrize("rep,N", SMALL)
def test_up_to_16_rows_within_the_attention_bound(rep, N, kb, vb):
    check_attention_bound(ragged_case(rep, N, kb, vb))


@pytest.mark.parametrize("kb,vb", BITS)
@pytest.mark.parametrize("rep,N", LARGE)
def test_more_rows_within_the_attention_bound(rep, N, kb, vb):
    check_attention_bound(ragged_case(rep, N, kb, vb))


def prefilled_case(seed, n, rep, N, kb, vb, offset=0.0):
    """A cache that kvq_kivi_prefill quantized: keys with six channels of 20 times the others', all
    keys and values moved by a constant. Returns the case with the cache's own codes, and the cache."""
    g = synth.rng(seed)
    B, H, R = 1, 2, 128
    nq = (n - R + 31) // 32 * 32
    case = T.make_tree_case(seed, B=B, H=H, N=N, n_quant=[nq], n_resid=[n - nq], rep=rep, k_bits=kb, v_bits=vb)
    outl = synth.outlier_channels(g, D, 6)
    k, v = synth.kivi_kv(g, B * H * n, D, outl)
    k, v = (np.asarray(x.reshape(B, H, n, D) + offset, np.float16) for x in (k, v))
    cache = kvq.KiviCache(case.base.cfg)
    kvq.kvq_kivi_prefill(case.base.cfg, cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    torch.cuda.synchronize()
    base = case.base
    assert [int(x) for x in (cache.n_tok, cache.n_quant_k, cache.n_quant_v)] == [n, nq, nq]
    base.k_codes = _layout.unpack_codes(cache.k_codes.cpu().numpy(), kb)
    base.v_codes = _layout.unpack_codes(cache.v_codes.cpu().numpy(), vb)
    for name in ("k_scale", "k_zero", "v_scale", "v_zero"):
        setattr(base, name, getattr(cache, name).cpu().numpy())
    base.k_res = cache.k_resid.cpu().numpy()
    ring = cache.v_resid.cpu().numpy()
    base.v_res = ring[:, :, (nq + np.arange(R)) % R]
    case.kd[:] = synth.kivi_kv(g, B * N * H, D, outl)[0].reshape(B, N, H, D) + offset
    return case, cache


@pytest.mark.parametrize("kb,vb", BITS)
@pytest.mark.parametrize("rep,N", [(1, 8), (2, 8)])
def test_up_to_16_rows_over_a_prefilled_cache(rep, N, kb, vb):
    check_attention_bound(*prefilled_case(4100, 3000, rep, N, kb, vb))


@pytest.mark.parametrize("kb,vb", BITS)
@pytest.mark.parametrize("rep,N", [(4, 8), (4, 48)])
def test_more_rows_over_a_prefilled_cache(rep, N, kb, vb):
    check_attention_bound(*prefilled_case(4200, 3000, rep, N, kb, vb))


@pytest.mark.parametrize("what", ["dead", "outlier"])
@pytest.mark.parametrize("rep,kb", [(1, 2), (1, 4), (2, 2), (2, 4), (6, 2), (6, 4)])
@pytest.mark.parametrize("down", [9, 12, 14, 16])
def test_small_key_scales_beside_a_large_one(rep, kb, down, what):
    # keys times 2^-down and queries times 2^down, the same scores, with one channel whose scale is 1 in every group: a
    # dead channel as the quantizer stores it (scale 1, codes and zero-point 0), or keys 2^down times as large as the
    # others under queries 2^down times as small
    case = T.make_tree_case(4300, B=2, H=2, N=6, n_quant=[256, 32], n_resid=[40, 3], rep=rep, k_bits=kb, q_scale=0.5)
    base, f = case.base, np.float16(2.0 ** -down)
    for x in (base.k_scale, base.k_res, case.kd):
        x *= f
    case.q *= 2.0 ** down
    for x in (base.k_scale, base.k_res, case.kd):
        x[..., 77] = 1 if what == "outlier" else 0
    if what == "outlier":
        base.k_res[..., 77] = base.k_res[..., 76] / f  # neighbours' values in the outlier's range
        case.kd[..., 77] = case.kd[..., 76] / f
        case.q[..., 77] *= 2.0 ** -down
    else:
        base.k_scale[..., 77], base.k_zero[..., 77], base.k_codes[..., 77] = 1, 0, 0
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("rep", [1, 2, 4, 9])
@pytest.mark.parametrize("power", [60, 104, 118])
def test_queries_whose_scores_still_fit_fp32(rep, power):
    # elements up to 2^120: one token takes all the weight, so rows whose largest score stands out by more than the
    # scores' own rounding (2^-12 of the absolute sums: fp32 sums of fp16 products, far below) equal its value
    case = T.make_tree_case(4400, B=1, H=1, N=4, n_quant=[64], n_resid=[30], rep=rep)
    case.q *= 2.0 ** power
    got = T.run_tree(case)
    assert np.isfinite(got).all()
    K, V, _, _ = T.context(case.base, 0, 0)
    keys, vals = (np.concatenate([x, y[0, :, 0].astype(np.float64)]) for x, y in ((K, case.kd), (V, case.vd)))
    clear = []
    for i in range(4):
        seen = np.array([True] * len(K) + [bool(int(case.mask[0, i]) >> j & 1) for j in range(4)])
        for r in range(rep):
            q = case.q[0, i, r]
            s, a = keys[seen] @ q, np.abs(keys[seen]) @ np.abs(q)
            top = np.argsort(s)[-2:]
            clear.append(s[top[1]] - s[top[0]] > 2.0 ** -12 * a.max())
            if clear[-1]:
                C.check_close(got[0, i, r], vals[seen][top[1]])
    assert np.mean(clear) > 0.5


@pytest.mark.parametrize("rep", [1, 2, 5])
def test_a_state_with_too_few_quantized_values_stays_in_the_buffers(rep):
    # n_quant_v below n_tok - residual is no valid state: it counts as n_tok - residual
    case = T.make_tree_case(4700, B=2, H=2, N=6, n_quant=[32 * 40, 256], n_resid=[90, 128], rep=rep,
                            n_quant_v=[32 * 40 + 90 - 128, 256])
    cache = C.fill_kivi_cache(case.base)
    want = T.run_tree(case, cache)
    cache.n_quant_v.copy_(torch.tensor([0, -5], dtype=torch.int32))
    assert np.array_equal(T.run_tree(case, cache), want)
