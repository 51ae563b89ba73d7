"""Calls with nothing to do (no request, no token) are no-ops, also where empty arrays have no address."""
import ctypes

import pytest
import torch

from sub_bit_quantized_gb300 import _build, kvq

D = 128
FAKE = 0x10000  # aligned, never dereferenced
BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


@pytest.mark.parametrize("p", [None, FAKE])
def test_empty_calls_need_no_addresses(L, p):
    c = kvq.KiviConfig(n_heads=8, max_batch=16, max_tokens=32).to_c()
    k = kvq.KiviCacheC(*([FAKE] * len(kvq.KIVI_CACHE_FIELDS)))
    for n_seq, N in ((0, 4), (3, 0), (0, 0)):
        assert L.kvq_kivi_commit(BY(c), BY(k), p, p, p, p, n_seq, N, None) == 0
    for B, n in ((0, 5), (2, 0)):
        assert L.kvq_kivi_read(BY(c), BY(k), p, 0, B, n, p, p, 0, 0, 0, None) == 0
    r = kvq.Rows(p, 0, 0, 0, 8, 0)
    for B, N in ((0, 3), (3, 0)):
        assert L.kvq_qk_norm_rope(D, B, N, BY(r), BY(r), BY(r), FAKE, FAKE, 1e-6, FAKE, FAKE, 64, p, BY(r), BY(r), BY(r), None) == 0
    # what is wrong with an empty call is still said
    assert L.kvq_kivi_commit(BY(c), BY(k), p, p, p, p, 17, 0, None) == 2
    assert L.kvq_kivi_read(BY(c), BY(k), p, 16, 1, 0, p, p, 0, 0, 0, None) == 2
    assert L.kvq_kivi_read(BY(c), BY(k), p, 0, 0, 5, p, p, 9, 0, 0, None) == 1
    assert L.kvq_qk_norm_rope(D, 0, 3, BY(r), None, None, None, None, 1e-6, None, None, 0, p, BY(r), None, None, None) == 1


@pytest.mark.gpu
def test_empty_tensors_through_the_binding():
    cfg = kvq.KiviConfig(n_heads=2, max_batch=3, max_tokens=32)
    cache = kvq.KiviCache(cfg)
    new = lambda *s, dt=torch.float16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    for B, N in ((0, 4), (3, 0)):
        x = new(B, N, 2, D)
        kvq.kvq_kivi_commit(cfg, cache, x, x, new(B, N, dt=torch.int32), torch.zeros(B, dtype=torch.int32, device="cuda"))
        w, t = new(D).fill_(1), torch.ones((8, D // 2), device="cuda")
        kvq.kvq_qk_norm_rope(x, x, x, w, w, 1e-6, t, t, new(B, N, dt=torch.int32), new(B, N, 2, D), new(B, N, 2, D), new(B, N, 2, D))
        out = new(B, 2, N, D)
        kvq.kvq_kivi_read(cfg, cache, out, out.clone(), tok_begin=torch.zeros(B, dtype=torch.int32, device="cuda"))
        kvq.kvq_kivi_read(cfg, cache, None, out)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0 and not cache.n_tok.any()
