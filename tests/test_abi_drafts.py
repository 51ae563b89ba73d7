"""CPU checks of the speculative step's entry points: argument errors are found on the host before
anything is launched. No call here reaches a kernel."""
import ctypes

import pytest
import torch

from sub_bit_quantized_gb300 import _build, kvq

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first
BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


def kivi(**kw):
    return kvq.KiviConfig(**{**dict(n_heads=8, n_q_heads=32, max_batch=16, max_tokens=3968), **kw}).to_c()


def cache():
    return kvq.KiviCacheC(*([FAKE] * len(kvq.KIVI_CACHE_FIELDS)))


def test_commit_argument_checks(L):
    f, c, k = L.kvq_kivi_commit, kivi(), cache()
    assert f(BY(c), BY(k), None, FAKE, FAKE, FAKE, 1, 4, None) == 1
    assert f(BY(c), BY(k), FAKE, FAKE + 8, FAKE, FAKE, 1, 4, None) == 1
    assert f(BY(c), BY(k), FAKE, FAKE, None, FAKE, 1, 4, None) == 1
    assert f(BY(c), BY(k), FAKE, FAKE, FAKE, FAKE, -1, 4, None) == 1
    assert f(BY(c), BY(k), FAKE, FAKE, FAKE, FAKE, 1, -4, None) == 1
    assert f(BY(c), BY(k), FAKE, FAKE, FAKE, FAKE, 17, 4, None) == 2     # n_seq > max_batch
    assert f(BY(kivi(residual=0)), BY(k), FAKE, FAKE, FAKE, FAKE, 1, 4, None) == 1
    assert f(BY(kivi(k_bits=3)), BY(k), FAKE, FAKE, FAKE, FAKE, 1, 4, None) == 3
    assert f(BY(c), BY(k), FAKE, FAKE, FAKE, FAKE, 0, 4, None) == 0      # nothing to do
    assert f(BY(c), BY(k), FAKE, FAKE, FAKE, FAKE, 1, 0, None) == 0
    k.n_tok = None
    assert f(BY(c), BY(k), FAKE, FAKE, FAKE, FAKE, 1, 4, None) == 1


def test_read_argument_checks(L):
    f, c, k = L.kvq_kivi_read, kivi(), cache()
    assert f(BY(c), BY(k), None, 0, 1, 5, None, None, 0, 0, 0, None) == 1      # nothing to write
    assert f(BY(c), BY(k), None, 0, 1, 5, FAKE + 4, None, 0, 0, 0, None) == 1  # misaligned
    assert f(BY(c), BY(k), FAKE + 4, 0, 1, 5, FAKE, None, 0, 0, 0, None) == 1
    assert f(BY(c), BY(k), None, 0, 1, 5, FAKE, None, 3, 0, 0, None) == 1      # type
    assert f(BY(c), BY(k), None, 0, 1, 5, FAKE, None, 0, 12, 0, None) == 1     # stride
    assert f(BY(c), BY(k), None, 0, 1, -5, FAKE, None, 0, 0, 0, None) == 1
    assert f(BY(c), BY(k), None, -1, 1, 5, FAKE, None, 0, 0, 0, None) == 1
    assert f(BY(c), BY(k), None, 15, 2, 5, FAKE, None, 0, 0, 0, None) == 2     # b0 + B > max_batch
    assert f(BY(c), BY(k), None, (1 << 31) - 1, 2, 5, FAKE, None, 0, 0, 0, None) == 2
    assert f(BY(c), BY(k), None, 0, 0, 5, FAKE, None, 0, 0, 0, None) == 0
    big = kivi(n_heads=65535, n_q_heads=65535, max_batch=65535)
    assert f(BY(big), BY(k), None, 0, 65535, 32, FAKE, None, 0, 0, 0, None) == 3


def rows(heads=8, dtype=0, p=FAKE, st=(0, 0, 0)):
    return kvq.Rows(p, *st, heads, dtype)


def test_norm_rope_argument_checks(L):
    f = L.kvq_qk_norm_rope

    def call(D=128, B=1, N=1, q=None, k=None, v=None, wq=FAKE, wk=FAKE, eps=1e-6, cos=None, sin=None, ctx=0, pos=None,
             qo=None, ko=None, vo=None):
        r = [None if x is None else BY(x) for x in (q, k, v, qo, ko, vo)]
        return f(D, B, N, *r[:3], wq, wk, eps, cos, sin, ctx, pos, *r[3:], None)

    ok = dict(q=rows(), qo=rows())
    assert call() == 1                                                  # no rows
    assert call(D=64, **ok) == 3
    assert call(B=-1, **ok) == 1
    for eps in (0.0, -1e-6, float("nan"), float("inf"), 1e-31, 2.0):
        assert call(eps=eps, **ok) == 1
    assert call(q=rows()) == 1 and call(qo=rows(), k=rows(), ko=rows()) == 1  # half a pair
    assert call(q=rows(), qo=rows(heads=4)) == 1
    assert call(q=rows(heads=0), qo=rows(heads=0)) == 1
    assert call(q=rows(dtype=5), qo=rows()) == 1
    assert call(q=rows(), qo=rows(), k=rows(dtype=2), ko=rows()) == 1   # inputs of two types
    assert call(q=rows(p=FAKE + 2), qo=rows()) == 1
    assert call(q=rows(st=(4, 0, 0)), qo=rows()) == 1
    assert call(q=rows(st=(0, -8, 0)), qo=rows()) == 1
    assert call(wq=None, **ok) == 1
    assert call(wk=None, k=rows(), ko=rows()) == 1
    assert call(cos=FAKE, ctx=8, pos=FAKE, **ok) == 1                   # no sin
    assert call(cos=FAKE, sin=FAKE, ctx=0, pos=FAKE, **ok) == 1
    assert call(cos=FAKE, sin=FAKE, ctx=8, **ok) == 1                   # no positions
    assert call(B=1 << 20, N=1 << 12, **ok) == 3                        # 2^32 tokens
    assert call(B=0, **ok) == 0


def test_tree_argument_checks(L):
    f, c, k = L.kvq_kivi_tree_attn, kivi(), cache()

    def call(cfg=c, q=FAKE, kd=FAKE, vd=FAKE, mask=FAKE, nd=None, B=1, N=4, out=FAKE, dt=0, ws=FAKE, n=1 << 40):
        return f(BY(cfg), BY(k), q, kd, vd, mask, nd, B, N, out, dt, ws, n, None)

    for name in ("q", "kd", "vd", "mask", "out"):
        assert call(**{name: None}) == 1 and call(**{name: FAKE + 8}) == 1
    assert call(nd=FAKE + 4) == 1
    assert call(dt=2) == 1
    assert call(B=0) == 1 and call(N=0) == 1
    assert call(B=17) == 2
    assert call(N=65) == 3
    assert call(cfg=kivi(k_bits=8)) == 3
    assert call(ws=None) == 5 and call(ws=FAKE + 8) == 5 and call(n=16) == 5
    big = kivi(n_heads=4096, n_q_heads=65536, max_batch=4096)
    assert call(cfg=big, B=4096, N=64) == 3
    assert L.kvq_kivi_tree_workspace_size(BY(c), 1, 65) == 0
    assert L.kvq_kivi_tree_workspace_size(BY(c), 1, 64) > 0


def test_binding_refuses_tensors_it_cannot_pass(L):
    cfg = kvq.KiviConfig(n_heads=2, max_batch=1, max_tokens=32)
    x = torch.zeros((1, 3, 2, 128), dtype=torch.float16)
    path = torch.zeros((1, 3), dtype=torch.int32)
    fake = type("FakeCache", (), {"c_struct": lambda self: cache()})()
    with pytest.raises(TypeError):
        kvq.kvq_kivi_commit(cfg, fake, x.float(), x, path, path[:, 0])
    with pytest.raises(ValueError):
        kvq.kvq_kivi_commit(cfg, fake, x[:, :2], x, path, path[:, 0])  # shape
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_kivi_commit(cfg, fake, x, x, path, path[:, 0])         # host memory
    with pytest.raises(ValueError):
        kvq.kvq_kivi_read(cfg, fake, None, None)
    with pytest.raises(ValueError):
        kvq.kvq_qk_norm_rope(None, None, None, None, None, 1e-6, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        kvq.kvq_qk_norm_rope(x, None, None, x[0, 0, 0], None, 1e-6, None, None, None, None, None, None)
