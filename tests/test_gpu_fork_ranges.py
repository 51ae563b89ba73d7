"""Slots that continue others where a call covers some of a cache's slots, short ones in great number, and on
another stream than the current one: every byte against the oracle."""
import numpy as np
import pytest
import torch

from oracle import continuations as oc
from sub_bit_quantized_gb300 import kvq
from tests import _continuations as K
from tests.test_gpu_continuations import check_fork, host, kivi_cache, vq_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(6))
def test_part_of_a_caches_slots_in_place(seed):
    # sources before, inside and behind the range: those inside are overwritten in the same call
    g = np.random.default_rng(seed)
    for cfg, cache in (kivi_cache(seed, 24, 2, 96), vq_cache(seed, 24, 2, 4)):
        for n, b0 in ((5, 3), (16, 8), (23, 1), (1, 23)):
            check_fork(cfg, cache, [int(x) for x in g.integers(-2, 24, n)], b0)
            check_fork(cfg, cache, [b0 + int(x) for x in g.permutation(n)], b0)
    assert kvq.device_error() == 0


@pytest.mark.parametrize("n", [9, 200, 256])
def test_many_short_slots(n):
    # far more moves than pieces of 2 KB: 256 slots of one head and a few tokens, from one prompt, and among one another
    cfg, cache = kivi_cache(n, n, 1, 32, R=32)
    other_cfg, other = kivi_cache(n + 1, 2, 1, 32, R=32)
    check_fork(cfg, cache, [1] * n, 0, other_cfg, other)
    check_fork(cfg, cache, [i // 2 * 2 for i in range(n)])
    check_fork(cfg, cache, [int(x) for x in np.random.default_rng(n).permutation(n)])
    cfg, cache = vq_cache(n, n, 1, 2, L=1, T=1)
    check_fork(cfg, cache, [n // 2] * n)
    check_fork(cfg, cache, [(i + 1) % n for i in range(n)])
    assert kvq.device_error() == 0


def test_on_another_stream_behind_its_work():
    cfg, cache = kivi_cache(3, 12, 2, 96)
    arrays, lens = host(cache)
    s = torch.cuda.Stream()
    source = torch.full((12,), -1, dtype=torch.int32, device="cuda")
    new = [int(x) for x in np.random.default_rng(5).permutation(12)]
    dev = torch.tensor(new, dtype=torch.int32, device="cuda")
    call = kvq.CacheForkCall(cfg, cache, source, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        source.copy_(dev)
    call()                                   # behind the copy, on its stream
    torch.cuda.synchronize()
    oc.fork(arrays, arrays, lens, lens, new, 0, 0, lambda name, *n: oc.kivi_rows(name, *n, cfg.residual))
    got, got_lens = host(cache)
    assert all(np.array_equal(got[x], arrays[x]) for x in K.KIVI_ARRAYS)
    assert all(np.array_equal(got_lens[x], lens[x]) for x in lens)
