"""Precision of attention under a shared prefix: the same for any number of rows that share it and for both
output types, over shares of several tiles a block."""
import numpy as np
import pytest
import torch

from oracle import kivi as okivi
from sub_bit_quantized_gb300 import kvq
from tests import _cases as C
from tests import _drafts as T
from tests.test_gpu_continuations import prefix_case
from tests.test_gpu_kivi_long_splits import copies

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4)])
@pytest.mark.parametrize("own", [3.0, 2.0 ** -8])
@pytest.mark.parametrize("B", [8, 40, 300])
def test_small_weights_beside_a_large_one_add_up(B, own, kb, vb):
    # One token's score lies 2^27.5 above those of all others, whose values are 3 where its own is 0 (code 0; its group spans
    # ``own``): the output is what the others' weights add up to. A weight is off by at most 2^-30 of the row's largest (half a
    # step of fp16's subnormals, 2^-25, where the largest is 2^5), 2^-2.5 of itself; the others' own roundings (2^-11, 2^-16)
    # are below 2^-6 of the output. The products add 16 tokens a step to fp32 sums that hold the large token's s (0 - c0) and
    # c0 s apart, each step off by up to 2^-23 of those: n / 16 steps, two sums.
    # 160 heads, so that a block of the GPU takes a head's prefix almost whole (152 blocks, 304 or 608 with few rows).
    H, n = 160, 2976
    cfg = kvq.KiviConfig(n_heads=H, n_q_heads=H, k_bits=kb, v_bits=vb, residual=32, max_batch=B, max_tokens=32)
    pcfg = kvq.KiviConfig(n_heads=H, n_q_heads=H, k_bits=kb, v_bits=vb, residual=32, max_batch=1, max_tokens=n)
    cache, prefix = kvq.KiviCache(cfg), kvq.KiviCache(pcfg)
    top = 2 ** kb - 1
    step = 13.5 / top                                   # 4.5 or 0.9
    prefix.k_scale.fill_(1.0)
    prefix.k_scale[..., 0] = step
    prefix.k_codes[:, :, 0, 0] = top                    # token 0: channel 0 is top * step, all else 0
    prefix.v_scale.fill_(3.0 / top)
    prefix.v_scale[:, :, 0] = own / top
    prefix.v_codes[:, :, 1:] = 255                      # every code the top one
    for name in ("n_tok", "n_quant_k", "n_quant_v"):
        getattr(prefix, name).fill_(n)
    q = torch.zeros((B, 1, H, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 16.0
    out = torch.zeros((B, 1, H, D), device="cuda")
    kvq.kvq_kivi_prefix_attn(cfg, cache, pcfg, prefix, 0, q, out)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    w = np.exp(-16.0 * top * float(np.float16(step)) / np.sqrt(D))
    assert 2.0 ** -27.6 < w < 2.0 ** -27.4
    ref = (n - 1) * w * top * float(np.float16(3.0 / top)) / (1 + (n - 1) * w)
    c0 = 1 if vb == 2 else 8
    bound = ref * (2.0 ** -30 / w + 2.0 ** -6) + 2 * n / 16 * 2.0 ** -23 * c0 * own / top
    assert (out.double() - ref).abs().max().item() <= bound


def parts(case, b, h):
    """Keys and values of a context [n][D], and sizes that errors are counted from: |s (c - c0)| + |s (z - c0)| of keys, what
    rounds of values, |s (c - c0)| + |s z| + |s c0| of values (all of fp16 rows: exact, their magnitude)."""
    K, V, _, _ = T.context(case, b, h)
    c, nqk, nqv = case.cfg, case.n_quant_k[b], case.n_quant_v[b]
    a, dv, av = np.abs(K), np.zeros_like(V), np.abs(V)
    c0 = 1.0 if c.k_bits == 2 else 8.0
    s, z = (np.repeat(x[b, h, :nqk // 32].astype(np.float64), 32, 0) for x in (case.k_scale, case.k_zero))
    a[:nqk] = np.abs(s * (case.k_codes[b, h, :nqk] - c0)) + np.abs(s * (z - c0))
    c0 = 1.0 if c.v_bits == 2 else 8.0
    s, z = (np.repeat(x[b, h, :nqv].astype(np.float64), 32, 1) for x in (case.v_scale, case.v_zero))
    own = np.abs(s * (case.v_codes[b, h, :nqv] - c0))
    dv[:nqv] = (2.0 ** -11 * own if c.v_bits == 4 else 0.0) + 2.0 ** -24
    av[:nqv] = own + np.abs(s * z) + np.abs(s * c0)
    return K, V, a, dv, av


def reference(case, prefix, drafts=True):
    """(out, bound), both [B][N][Hq][D] fp64; padding rows are NaN in out.

    Keys enter in two fp16 parts (2^-21 of s (c - c0) and of s (z - c0)), products of 128 channels are 8 or 16 steps of 16 in
    fp32, each off by 2^-23 at most: scores by 2^-17 of sum |q| (|s (c - c0)| + |s (z - c0)|) / sqrt(D) with the exponent's
    fp32 steps. Weights are off by 2^-11 and 2^-30 of the row's largest, 4-bit values by 2^-11 of |s (c - c0)|, values are halved
    (2^-24); sums of up to 60 steps a block by 60 2^-23 < 2^-17 of their absolute terms, and the joins by as much."""
    B, N, Hq, _ = case.q.shape
    H = case.base.cfg.n_heads
    out, bound = np.full(case.q.shape, np.nan), np.zeros(case.q.shape)
    for h in range(H):
        heads = [x for x in range(Hq) if okivi.kv_head(x, Hq, H) == h]
        shared = parts(prefix, 0, h)
        q = case.q[:, :, heads].astype(np.float64).reshape(-1, D)
        scores = lambda x, y: x @ y.T / np.sqrt(D)  # noqa: E731
        S0, E0 = scores(q, shared[0]), scores(np.abs(q), shared[2])
        for b in range(B):
            nd = min(max(case.n_draft[b], 0), N)
            if nd == 0:
                continue
            own = parts(case.base, b, h)
            kd, vd = (x[b, :nd, h].astype(np.float64) for x in (case.kd, case.vd))
            new = (kd, vd, np.abs(kd), np.zeros_like(vd), np.abs(vd))
            at = slice(b * N * len(heads), (b * N + nd) * len(heads))
            K, V, A, dV, AV = (np.concatenate(x) for x in zip(own, new))
            S = np.concatenate([S0[at], scores(q[at], K)], 1)
            E = np.concatenate([E0[at], scores(np.abs(q[at]), A)], 1)
            for i in range(nd):
                for j in range(nd):
                    if not drafts or not int(case.mask[b, i]) >> j & 1:
                        S[i * len(heads):(i + 1) * len(heads), S.shape[1] - nd + j] = -np.inf
            p = np.exp(S - S.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            n0 = len(shared[1])
            mix = lambda w, x, y: w[:, :n0] @ x + w[:, n0:] @ y  # noqa: E731
            f = np.expm1(2.0 ** -17 * E) + 2.0 ** -11
            f = p * (f + (p * f).sum(1, keepdims=True))
            most = max(x.max() if x.size else 0.0 for x in (np.abs(shared[1]), np.abs(V)))
            o = mix(p, shared[1], V)
            d = 1.1 * (mix(f, np.abs(shared[1]), np.abs(V)) + mix(p, shared[3], dV) + 2.0 ** -16 * mix(p, shared[4], AV) +
                       (np.isfinite(S).sum(1) * 2.0 ** -30 * p.max(1) * most)[:, None])
            out[b, :nd, heads] = o.reshape(nd, len(heads), D).transpose(1, 0, 2)
            bound[b, :nd, heads] = d.reshape(nd, len(heads), D).transpose(1, 0, 2)
    return out, bound


def both_types(case, prefix, nh, drafts=True):
    """Outputs of the call in fp32, and in bf16 (checked to be those, rounded), with every head nh times."""
    cfg, cache = copies(case.base, 1, nh)
    pcfg, pcache = copies(prefix, 1, nh)
    q, kd, vd, mask, nd = T.tensors(case)
    q, kd, vd = (x.repeat(1, 1, nh, 1) for x in (q, kd, vd))
    more = dict(k_draft=kd, v_draft=vd, mask=mask) if drafts else {}
    outs = []
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
        kvq.kvq_kivi_prefix_attn(cfg, cache, pcfg, pcache, 0, q, out, n_draft=nd, **more)
        outs.append(out)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    assert torch.equal(outs[0].bfloat16(), outs[1])
    return outs[0].double().cpu().numpy()


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("B,rep,N", [(3, 4, 2), (9, 4, 1), (70, 4, 1), (40, 1, 1), (1, 1, 64)])
def test_bf16_outputs_are_the_fp32_ones_rounded(B, rep, N, kb, vb):
    # 24 rows a KV head over the prefix, 36, 280, 40 and 64 (masks of 64 tokens)
    case, prefix = prefix_case(B + N, B, 2, rep, N, (64, 9), (512, 41), kb, vb)
    ref, bound = reference(case, prefix)
    T.check_rows(both_types(case, prefix, 1), ref, bound, 7.0)


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("B", [35, 64, 75])
def test_many_tiles_a_block(B, late, kb, vb):
    # 140, 256 and 300 rows over 8191 tokens of eight heads: a block takes four to ten tiles, its second row tile on, full, and
    # on and off by turns. late: keys that grow along the prefix, so that maxima move to its end
    case, prefix = prefix_case(B, B, 2, 4, 1, (64, 9), (8160, 31), kb, vb, n_draft=[int(b % 9 != 4) for b in range(B)])
    if late:
        grow = np.linspace(0.1, 2.0, 255).astype(np.float16)[None, None, :, None]
        prefix.k_scale = (prefix.k_scale * grow).astype(np.float16)
    ref, bound = reference(case, prefix)
    got = both_types(case, prefix, 4)
    for i in range(4):  # each copy of the heads lies elsewhere in the blocks' shares
        T.check_rows(got[:, :, 8 * i:8 * (i + 1)], ref, bound, 7.0)
