"""Attention under a shared prefix with queries so large that a row is its best token's value: every row whose
two best scores lie apart is checked, and how many those are."""
import numpy as np
import pytest

from tests import _continuations as K
from tests import _drafts as T
from tests.test_gpu_continuations import prefix_case

pytestmark = pytest.mark.gpu
D = 128


def best_values(case, prefix):
    """(b, query head, value) of rows whose two best scores lie further apart than their errors."""
    H, rep = case.base.cfg.n_heads, case.q.shape[2] // case.base.cfg.n_heads
    rows = []
    for b in range(case.q.shape[0]):
        for h in range(H):
            K0, V0, _, _ = T.context(prefix, 0, h)
            K1, V1, _, _ = T.context(case.base, b, h)
            k = np.concatenate([K0, K1, case.kd[b, :, h].astype(np.float64)])
            v = np.concatenate([V0, V1, case.vd[b, :, h].astype(np.float64)])
            for hq in range(h * rep, (h + 1) * rep):
                x = k @ case.q[b, 0, hq].astype(np.float64) / np.sqrt(D)
                s = np.sort(x)
                # scores are off by 2^-16 of their absolute terms, a few times the score itself; a weight of exp(-60) is nothing
                if s[-1] - s[-2] > 60 + 2.0 ** -9 * np.abs(s).max():
                    rows.append((b, hq, v[np.argmax(x)]))
    return rows


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4)])
@pytest.mark.parametrize("B,scale", [(3, 2.0 ** 12), (40, 2.0 ** 12), (40, 2.0 ** 20), (40, 2.0 ** 60)])
def test_a_row_is_its_best_tokens_value(B, scale, kb, vb):
    case, prefix = prefix_case(77, B, 2, 2, 1, (32, 5), (160, 40), kb, vb)
    case.mask[:] = 1
    case.q = np.asarray(case.q * scale, np.float32).astype(np.float64)
    rows = best_values(case, prefix)
    assert len(rows) >= 0.9 * B * 4
    got = K.run_prefix(case, prefix)
    for b, hq, v in rows:
        assert np.abs(got[b, 0, hq] - v).max() <= 2.0 ** -9 * (np.abs(v).max() + 8), (b, hq)
