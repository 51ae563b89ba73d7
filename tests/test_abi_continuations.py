"""CPU checks of the entry points that serve many continuations of one prompt: argument errors are found
on the host before anything is launched (no call here reaches a kernel), and the oracles against plain
restatements."""
import ctypes
import types

import numpy as np
import pytest
import torch

from oracle import continuations as oc
from sub_bit_quantized_gb300 import _build, kvq

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first
BY = ctypes.byref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kvq.lib()


def kivi(**kw):
    return kvq.KiviConfig(**{**dict(n_heads=8, n_q_heads=32, max_batch=16, max_tokens=3968), **kw}).to_c()


def vq(**kw):
    return kvq.VqConfig(**{**dict(n_layers=2, n_heads=4, max_pages=10, max_batch=8, max_ctx=512), **kw}).to_c()


def kivi_cache(at=FAKE):
    return kvq.KiviCacheC(*([at] * len(kvq.KIVI_CACHE_FIELDS)))


def vq_cache(at=FAKE):
    return kvq.VqCacheC(*([at] * len(kvq.VqCacheC._fields_)))


def test_prefix_argument_checks(L):
    f, c, k = L.kvq_kivi_prefix_attn, kivi(), kivi_cache()
    p, pk = kivi(max_batch=3, k_bits=4, residual=64), kivi_cache()

    def call(cfg=c, pre=p, cache=k, pcache=pk, slot=0, q=FAKE, kd=FAKE, vd=FAKE, mask=FAKE, nd=None, B=1, N=4, out=FAKE, dt=0,
             ws=FAKE, n=1 << 40):
        ref = lambda x: None if x is None else BY(x)  # noqa: E731
        return f(ref(cfg), ref(cache), ref(pre), ref(pcache), slot, q, kd, vd, mask, nd, B, N, out, dt, ws, n, None)

    for name in ("q", "out"):
        assert call(**{name: None}) == 1 and call(**{name: FAKE + 8}) == 1
    for name in ("cfg", "pre", "cache", "pcache"):
        assert call(**{name: None}) == 1
    assert call(kd=None) == 1 and call(vd=None) == 1 and call(mask=FAKE + 4) == 1
    assert call(mask=None) == 1 and call(mask=None, kd=None) == 1       # drafts without a mask
    assert call(mask=None, kd=None, vd=None, ws=None) == 5               # none at all is a call
    assert call(nd=FAKE + 4) == 1
    assert call(dt=2) == 1
    assert call(B=0) == 1 and call(N=0) == 1
    assert call(B=17) == 2
    assert call(N=65) == 3
    assert call(slot=-1) == 1 and call(slot=3) == 2
    assert call(pre=kivi(n_heads=4)) == 1 and call(pre=kivi(n_q_heads=8)) == 1
    assert call(cfg=kivi(k_bits=8)) == 3 and call(pre=kivi(v_bits=3)) == 3
    assert call(ws=None) == 5 and call(ws=FAKE + 8) == 5 and call(n=16) == 5
    big = kivi(n_heads=4096, n_q_heads=65536, max_batch=4096)
    assert call(cfg=big, pre=big, B=4096, N=64) == 3
    wide = kivi(max_batch=65535, max_tokens=32)
    assert call(cfg=wide, pre=kivi(max_tokens=1 << 30), B=65535, N=64) == 3  # rows times prefix tiles
    size = L.kvq_kivi_prefix_workspace_size
    assert size(BY(c), BY(p), 1, 65) == 0 and size(BY(c), BY(kivi(n_heads=2)), 1, 1) == 0 and size(BY(c), None, 1, 1) == 0
    assert size(BY(c), BY(p), 16, 4) >= 2 * 16 * 4 * 32 * (128 + 1) * 4
    bad = kivi_cache()
    bad.v_zero = FAKE + 2
    assert call(pcache=bad) == 1


def test_fork_argument_checks(L):
    f, c, k = L.kvq_cache_fork, kivi(), kivi_cache()

    def call(fmt=1, cfg=c, cache=k, fc=None, fk=None, source=FAKE, b0=0, n=4):
        ref = lambda x: None if x is None else BY(x)  # noqa: E731
        return f(fmt, ref(cfg), ref(cache), ref(fc), ref(fk), source, b0, n, None)

    assert call(fmt=2) == 1
    assert call(cfg=None) == 1 and call(cache=None) == 1
    assert call(source=None) == 1 and call(source=FAKE + 8) == 1
    assert call(fc=c) == 1 and call(fk=k) == 1                         # half of another cache
    assert call(b0=-1) == 1 and call(n=-1) == 1
    assert call(b0=13) == 2 and call(n=17) == 2 and call(b0=(1 << 31) - 1, n=4) == 2
    assert call(cfg=kivi(max_batch=600), n=257) == 3
    assert call(n=0, source=None) == 0
    other = kivi_cache(2 * FAKE)
    for kw in (dict(n_heads=4), dict(k_bits=4), dict(v_bits=4), dict(residual=64)):
        assert call(fc=kivi(**kw), fk=other) == 1
    assert call(fc=kivi(n_q_heads=8, max_tokens=32, max_batch=1), fk=other, n=0) == 0
    assert call(fc=kivi(max_tokens=64), fk=k, n=0) == 1                # one cache with two shapes
    assert call(cfg=kivi(k_bits=3)) == 3
    v, vk = vq(), vq_cache()
    assert call(0, v, vk, n=0) == 0
    assert call(0, v, vk, n=9) == 2
    for kw in (dict(T=2), dict(Tc=1, G=8), dict(n_layers=1), dict(n_heads=2), dict(sink=4), dict(recent=256)):
        assert call(0, v, vk, vq(**kw), vq_cache(2 * FAKE)) == 1
    assert call(0, v, vk, vq(max_pages=99, max_batch=2, max_ctx=9999), vq_cache(2 * FAKE), n=0) == 0
    vk.win_k = None
    assert call(0, v, vk, n=0) == 1


def test_verify_argument_checks(L):
    f = L.kvq_verify_draft

    def dist(p=FAKE, sb=0, st=0, dt=1):
        return kvq.Dist(p, sb, st, dt)

    def call(B=2, N=4, V=100, p=dist(), q=None, token=FAKE, parent=FAKE, nd=None, u=FAKE, path=FAKE, acc=FAKE, nxt=FAKE):
        ref = lambda x: None if x is None else BY(x)  # noqa: E731
        return f(B, N, V, ref(p), ref(q), token, parent, nd, u, path, acc, nxt, None)

    for name in ("token", "parent", "path", "acc", "nxt"):
        assert call(**{name: None}) == 1 and call(**{name: FAKE + 8}) == 1
    assert call(nd=FAKE + 4) == 1 and call(u=FAKE + 4) == 1
    assert call(p=None) == 1 and call(p=dist(None)) == 1 and call(p=dist(FAKE + 4)) == 1
    assert call(p=dist(sb=-1)) == 1 and call(p=dist(st=-4)) == 1 and call(p=dist(dt=3)) == 1
    assert call(q=dist(None)) == 1 and call(q=dist(dt=0)) == 1 and call(q=dist(st=-4)) == 1
    assert call(q=dist(), u=None) == 1                                  # a draft distribution without sampling
    assert call(B=-1) == 1 and call(N=-1) == 1 and call(V=0) == 1
    assert call(N=65) == 3 and call(B=65536) == 3 and call(V=(1 << 30) + 1) == 3
    assert call(B=0, token=None, p=dist(None)) == 0 and call(N=0, token=None) == 0


def test_binding_refuses_tensors_it_cannot_pass(L):
    cfg = kvq.KiviConfig(n_heads=2, max_batch=1, max_tokens=32)
    fake = types.SimpleNamespace(c_struct=kivi_cache)
    q, out = torch.zeros((1, 3, 2, 128), dtype=torch.bfloat16), torch.zeros((1, 3, 2, 128))
    with pytest.raises(TypeError):
        kvq.kvq_kivi_prefix_attn(cfg, fake, cfg, fake, 0, q.half(), out)
    with pytest.raises(ValueError):
        kvq.kvq_kivi_prefix_attn(cfg, fake, cfg, fake, 0, q[0], out)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_kivi_prefix_attn(cfg, fake, cfg, fake, 0, q, out)
    source = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_cache_fork(cfg, fake, source)
    with pytest.raises(TypeError):
        kvq.kvq_cache_fork(cfg, fake, source.long())
    with pytest.raises(ValueError):
        kvq.kvq_cache_fork(cfg, fake, source, from_cfg=cfg)
    with pytest.raises(TypeError):
        kvq.kvq_cache_fork(cfg, fake, source, from_cfg=kvq.VqConfig(), from_cache=fake)
    P, t = torch.zeros((1, 2, 9)), torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        kvq.kvq_verify_draft(P.double(), None, t, t, P[:, :, 0], t, t[:, 0], t[:, 0])
    with pytest.raises(ValueError):
        kvq.kvq_verify_draft(P[0], None, t, t, P[:, :, 0], t, t[:, 0], t[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        kvq.kvq_verify_draft(P, None, t, t, P[:, :, 0], t, t[:, 0], t[:, 0])


def test_oracle_walk_equals_the_closed_form():
    # after k rejections the residual is max(0, P - a Q) with a the sum of the earlier normalisers, Z_0 = 1
    g = np.random.default_rng(3)
    P, Q = g.dirichlet(np.ones(40) * 0.3, 1), g.dirichlet(np.ones(40) * 0.3, 1)
    r, z, a = P[0].copy(), 1.0, 0.0
    for _ in range(5):
        a += z
        r = np.maximum(r - z * Q[0], 0)
        z = r.sum()
        np.testing.assert_allclose(r, np.maximum(P[0] - a * Q[0], 0), atol=1e-15)
    path, nxt = oc.verify(P, Q, [0], [0], [0.5], 1)
    assert path == [0] and nxt == int(np.argmax(np.cumsum(P[0]) > 0.5 * P[0].sum()))


def test_oracle_verify_keeps_the_targets_distribution():
    # 20000 walks: three children drawn from q; a share's standard deviation is below 0.0036, five of them
    g = np.random.default_rng(4)
    p, q = np.array([0.1, 0.45, 0.15, 0.3]), np.array([0.4, 0.1, 0.3, 0.2])
    P, Q = np.tile(p, (4, 1)), np.tile(q, (4, 1))
    first = []
    for _ in range(20000):
        token = [0, *g.choice(4, 3, p=q)]
        path, nxt = oc.verify(P, Q, token, [0, 0, 0, 0], g.random(4), 4)
        first.append(token[path[1]] if len(path) > 1 else nxt)
    assert np.abs(np.bincount(first, minlength=4) / 20000 - p).max() < 5 * 0.0036


def test_oracle_fork_takes_every_slot_as_it_was():
    x = {"k_codes": np.arange(24, dtype=np.uint8).reshape(4, 1, 6, 1)}
    lens = {"n": np.array([5, 6, 2, 3]), "nqk": np.array([5, 6, 2, 3]), "nqv": np.array([5, 6, 2, 3])}
    was = x["k_codes"].copy()
    oc.fork(x, x, lens, lens, [1, 0, oc.FREE, 2], 0, 0, lambda name, *n: oc.kivi_rows(name, *n, 32))
    got = x["k_codes"][:, 0, :, 0]
    assert got[0].tolist() == was[1, 0, :, 0].tolist() and got[1].tolist() == [*was[0, 0, :5, 0], was[1, 0, 5, 0]]
    assert got[3].tolist() == [*was[2, 0, :2, 0], *was[3, 0, 2:, 0]] and lens["n"].tolist() == [6, 5, 0, 2]
    assert oc.kivi_rows("v_resid", 70, 64, 62, 32) == [30, 31, 0, 1, 2, 3, 4, 5]
    assert oc.vq_rows("win_k", 90, 1, 8, 64) == list(range(8)) + [16 + i for i in range(64)] + list(range(8, 18))[:10]
