"""A split of many chunks, on a GPU that is full: over tens of chunks the warps of a block drift as far
apart as its ring of stages lets them. Every (request, head) is a copy of one of four, so any two copies
have the same bits, and the four are checked against the fp64 oracle."""
import pytest
import torch

from sub_bit_quantized_gb300 import kvq
from tests import _cases as C
from tests import _continuations as K
from tests import _drafts as T
from tests.test_gpu_continuations import prefix_case

pytestmark = pytest.mark.gpu
PARTS = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "k_resid", "v_resid")


def copies(case, nb, nh):
    """The cache of `case` nb times along the requests, nh times along the heads."""
    small, c = C.fill_kivi_cache(case), case.cfg
    cfg = kvq.KiviConfig(n_heads=c.n_heads * nh, n_q_heads=c.q_heads * nh, k_bits=c.k_bits, v_bits=c.v_bits,
                         residual=c.residual, max_batch=c.max_batch * nb, max_tokens=c.max_tokens)
    big = kvq.KiviCache(cfg)
    for name in PARTS:
        x = getattr(small, name)
        getattr(big, name).copy_(x.repeat(nb, nh, *[1] * (x.dim() - 2)))
    for name in ("n_tok", "n_quant_k", "n_quant_v"):
        getattr(big, name).copy_(getattr(small, name).repeat(nb))
    return cfg, big


@pytest.mark.parametrize("k_bits,v_bits", [(4, 4), (2, 2), (4, 2), (2, 4)])
@pytest.mark.parametrize("rep", [1, 4])
def test_decode_of_many_chunks_a_split(k_bits, v_bits, rep):
    case = C.make_kivi_case(61, B=2, H=2, n_quant=[5120, 4000], n_resid=[40, 128], Hq=2 * rep, k_bits=k_bits, v_bits=v_bits,
                            n_quant_v=[5100, 4000])
    cfg, cache = copies(case, 8, 16)
    q = C.bf16_tensor(case.q).repeat(8, 16, 1)
    ws = kvq.make_workspace(cfg, 16, 1)
    out = torch.zeros((16, 32 * rep, 128), device="cuda")
    for _ in range(5):
        out.fill_(7.0)
        kvq.kvq_decode_attn(cfg, cache, 0, 1, q, out, 1, ws)
        torch.cuda.synchronize()
        assert kvq.device_error() == 0
        assert torch.equal(out, out[:2, :2 * rep].repeat(8, 16, 1))
    for b in range(2):
        for h in range(2 * rep):
            C.check_close(out[b, h].cpu().numpy(), C.oracle_kivi(case, b, h))


@pytest.mark.parametrize("k_bits,v_bits", [(4, 4), (2, 2), (4, 2), (2, 4)])
@pytest.mark.parametrize("nb,nh", [(8, 16), (20, 8)])
def test_prefix_and_own_tokens_of_many_chunks(nb, nh, k_bits, v_bits):
    # 16 and 40 rows a KV head over the prefix; own tokens by the decode's kernel
    case, prefix = prefix_case(67, 2, 2, 1, 1, [(2048, 100), (1536, 7)], (4096, 31), k_bits, v_bits)
    ref, bound = K.prefix_reference(case, prefix, 0)
    cfg, cache = copies(case.base, nb, nh)
    pcfg, pcache = copies(prefix, 1, nh)
    q, kd, vd, mask, nd = T.tensors(case)
    q, kd, vd = (x.repeat(nb, 1, nh, 1) for x in (q, kd, vd))
    more = dict(k_draft=kd, v_draft=vd, mask=mask.repeat(nb, 1), n_draft=None if nd is None else nd.repeat(nb))
    out = torch.empty(q.shape, device="cuda")
    for _ in range(5):
        out.fill_(7.0)
        kvq.kvq_kivi_prefix_attn(cfg, cache, pcfg, pcache, 0, q, out, **more)
        torch.cuda.synchronize()
        assert kvq.device_error() == 0
        # shares of the prefix end at other places for other heads; its rows and the own tokens' are each in one order
        T.check_rows(out[:2, :, :2].double().cpu().numpy(), ref, bound, 7.0)
        for b in range(0, 2 * nb, 2):
            for h in range(0, 2 * nh, 2):
                T.check_rows(out[b:b + 2, :, h:h + 2].double().cpu().numpy(), ref, bound, 7.0)
