"""Precision of attention under a shared prefix: the same for any number of rows that share it and for both
output types, over shares of several tiles a block."""
import numpy as np
import pytest
import torch

from sub_bit_quantized_gb300 import kvq

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
