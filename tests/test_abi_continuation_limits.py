"""CPU checks of the sizes from which on calls over many continuations are refused, as the header states them
(no call here reaches a kernel)."""
import ctypes

import pytest

from sub_bit_quantized_gb300 import _build, kvq

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first
BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


def fork(L, fmt, cfg):
    kind, n = (kvq.KiviCacheC, len(kvq.KIVI_CACHE_FIELDS)) if fmt == kvq.FMT_KIVI else (kvq.VqCacheC, len(kvq.VqCacheC._fields_))
    return L.kvq_cache_fork(fmt, BY(cfg.to_c()), BY(kind(*([FAKE] * n))), None, None, FAKE, 0, 2, None)


def test_fork_refuses_slots_beyond_its_indexes(L):
    kivi = lambda **kw: kvq.KiviConfig(**{**dict(n_heads=1, max_batch=4, max_tokens=64), **kw})  # noqa: E731
    assert fork(L, kvq.FMT_KIVI, kivi(max_tokens=1 << 25)) == kvq.ERR_UNSUPPORTED
    # 2^36 bytes of codes a slot: 2^11 heads of 2^20 tokens of 32 bytes
    assert fork(L, kvq.FMT_KIVI, kivi(max_tokens=1 << 20, n_heads=1 << 11)) == kvq.ERR_UNSUPPORTED
    vq = lambda **kw: kvq.VqConfig(**{**dict(n_layers=1, n_heads=1, max_pages=10, max_batch=4, max_ctx=512), **kw})  # noqa: E731
    assert fork(L, kvq.FMT_LOOPVQ, vq(max_pages=1 << 25)) == kvq.ERR_UNSUPPORTED
    assert fork(L, kvq.FMT_LOOPVQ, vq(n_layers=1 << 15, n_heads=1 << 14)) == kvq.ERR_UNSUPPORTED


def test_verify_refuses_rows_beyond_its_indexes(L):
    d = kvq.Dist(FAKE, 0, 0, kvq.DT_FP32)
    call = lambda V: L.kvq_verify_draft(1, 1, V, BY(d), None, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None)  # noqa: E731
    assert call((1 << 30) + 1) == kvq.ERR_UNSUPPORTED and call(0) == kvq.ERR_INVALID_ARG
