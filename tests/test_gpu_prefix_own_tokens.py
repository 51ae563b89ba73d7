"""Attention under a shared prefix, one row a KV head: one long request among short ones, at both sides of the
capacity up to which a block takes a request's own tokens whole."""
import pytest

from tests import _drafts as T
from tests.test_gpu_continuations import prefix_case
from tests.test_gpu_prefix_precision import both_types, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("long", [2048, 2080, 8192])
@pytest.mark.parametrize("drafts", [True, False])
def test_one_long_request_among_short_ones(long, drafts, kb, vb):
    own = [(32 * (b % 3), b % 30) for b in range(9)] + [(long, 77)]
    case, prefix = prefix_case(long, 10, 2, 1, 1, own, (96, 20), kb, vb)
    ref, bound = reference(case, prefix, drafts)
    got = both_types(case, prefix, 16, drafts)  # 320 requests and heads
    for i in range(16):
        T.check_rows(got[:, :, 2 * i:2 * (i + 1)], ref, bound, 7.0)
