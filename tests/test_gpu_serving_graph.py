"""A serving step captured whole: slots that take over others, attention under the shared prefix, verification
and commit in one graph, replayed over new inputs, against the same calls made one by one."""
import pytest
import torch

from sub_bit_quantized_gb300 import kvq
from tests import _continuations as K

pytestmark = pytest.mark.gpu
D = 128
LENS = ("n_tok", "n_quant_k", "n_quant_v")


@pytest.mark.parametrize("bits", [(2, 2), (4, 4)])
@pytest.mark.parametrize("B,H,rep,N", [(4, 2, 2, 5), (20, 2, 4, 3), (40, 8, 1, 1)])
def test_a_captured_step(B, H, rep, N, bits):
    # 20 to 240 rows a KV head over the prefix, and one row with so many requests that the decode's kernel takes their own tokens
    g = torch.Generator(device="cuda").manual_seed(B)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    R, V = 32, 3001
    kw = dict(n_heads=H, n_q_heads=H * rep, k_bits=bits[0], v_bits=bits[1], residual=R)
    cfg, pcfg = kvq.KiviConfig(max_batch=B, max_tokens=256, **kw), kvq.KiviConfig(max_batch=1, max_tokens=512, **kw)
    caches, prefix = [kvq.KiviCache(cfg) for _ in range(2)], kvq.KiviCache(pcfg)
    kvq.kvq_kivi_prefill(pcfg, prefix, rnd(1, H, 500, D).half(), rnd(1, H, 500, D).half())
    k, v = rnd(B, H, 90, D).half(), rnd(B, H, 90, D).half()
    for cache in caches:
        kvq.kvq_kivi_prefill(cfg, cache, k, v)
    parent = K.tree(torch.Generator().manual_seed(3), B, N)
    see = torch.zeros((B, N), dtype=torch.int64)
    for b in range(B):
        for i in range(N):
            see[b, i] = (int(see[b, parent[b, i]]) if i else 0) | 1 << i
    mask, parent = see.cuda(), parent.cuda()
    source = torch.full((B,), kvq.SLOT_KEEP, dtype=torch.int32, device="cuda")
    q, kd, vd = rnd(B, N, H * rep, D).bfloat16(), rnd(B, N, H, D).half(), rnd(B, N, H, D).half()
    P, Q = (torch.softmax(2 * rnd(B, N, V), -1) for _ in range(2))
    token = torch.randint(0, V, (B, N), generator=g, device="cuda").int()
    u = torch.rand((B, N), generator=g, device="cuda")
    n_draft = torch.full((B,), N, dtype=torch.int32, device="cuda")

    def buffers():
        return (torch.zeros((B, N, H * rep, D), device="cuda"), torch.zeros((B, N), dtype=torch.int32, device="cuda"),
                torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"),
                kvq.make_prefix_workspace(cfg, pcfg, B, N))

    def step(cache, out, path, count, nxt, ws):
        kvq.kvq_cache_fork(cfg, cache, source)
        kvq.kvq_kivi_prefix_attn(cfg, cache, pcfg, prefix, 0, q, out, kd, vd, mask, n_draft, ws)
        kvq.kvq_verify_draft(P, Q, token, parent, u, path, count, nxt, n_draft)
        kvq.kvq_kivi_commit(cfg, cache, kd, vd, path, count)

    one, two = buffers(), buffers()
    for cache, given in ((caches[0], one), (caches[1], two)):  # once each, so that both caches go on together
        step(cache, *given)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[1], *two)
    accepted = 0
    for turn in range(6):
        source.copy_(torch.randint(-1, B, (B,), generator=g, device="cuda"))
        n_draft.copy_(torch.randint(0, N + 1, (B,), generator=g, device="cuda"))
        for x, y in ((q, rnd(*q.shape)), (kd, rnd(*kd.shape)), (vd, rnd(*vd.shape)), (u, torch.rand(u.shape, generator=g, device="cuda"))):
            x.copy_(y)
        P.copy_(torch.softmax(2 * rnd(B, N, V), -1))
        Q.copy_((P + 0.3 * torch.softmax(2 * rnd(B, N, V), -1)) / 1.3)
        at = parent.long().clamp(min=0)
        rows = Q.gather(1, at[:, :, None].expand(-1, -1, V)).flatten(0, 1)
        token.copy_(torch.multinomial(rows, 1, generator=g).view(B, N))
        step(caches[0], *one)
        graph.replay()
        torch.cuda.synchronize()
        assert kvq.device_error() == 0
        for x, y in zip(one[:4], two[:4]):
            assert torch.equal(x, y)
        for name in K.KIVI_ARRAYS + LENS:
            x, y = getattr(caches[0], name), getattr(caches[1], name)
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
        accepted += int(two[2].clamp(min=1).sub(1).sum())
    assert accepted > 0 or N == 1
    assert caches[1].n_tok.max().item() > 90
