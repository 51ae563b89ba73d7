"""Verification of drafted tokens at the ends of its ranges: rows so long that a chunk's sum covers several
pieces of the draw, other streams, captured and replayed calls."""
import numpy as np
import pytest
import torch

from oracle import continuations as oc
from sub_bit_quantized_gb300 import kvq
from tests import _continuations as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,B", [(600011, 320), (2100000, 160)])
@pytest.mark.parametrize("draft", [True, False])
def test_rows_of_many_chunks(V, B, draft, dtype):
    # one block a request and more than 2^19 entries: sums are kept of 1024 or 4096 entries. One row for all nodes (strides of
    # 0); the numbers of the draw reach every part of the row, tests go either way
    g = torch.Generator().manual_seed(V)
    row = torch.rand(V, generator=g) ** 8
    other = torch.rand(V, generator=g) ** 8
    P, Q = ((x / x.sum() * 2).to(dtype) for x in (row, other))  # a row need not sum to 1 for the draw
    u = torch.rand((B, 2), generator=g)
    u[:, 0] = (torch.arange(B) + 0.5) / B
    u[::3, 1] = 0.0
    u[1::3, 1] = 0.999
    parent = torch.zeros((B, 2), dtype=torch.int32)
    token = torch.randint(0, V, (B, 2), generator=g).int()
    wide = lambda x: x.cuda().expand(B, 2, V)  # noqa: E731
    path, count, nxt = K.run_verify(wide(P), wide(Q) if draft else None, token, parent, u)
    assert kvq.device_error() == 0
    Pn, Qn = (np.broadcast_to(x.double().numpy(), (2, V)) for x in (P, Q))
    seen = set()
    for b in range(B):
        want, after = oc.verify(Pn, Qn if draft else None, token[b].tolist(), [0, 0], u[b].numpy(), 2)
        assert count[b] == len(want) and path[b, :len(want)].tolist() == want and nxt[b] == after, b
        seen.add(int(nxt[b]) % 4096 // 512)
    assert len(seen) == 8  # all pieces of a chunk
    assert 0 < (count == 2).sum() < B


def inputs(seed, B, N, V, draft=True):
    g = torch.Generator().manual_seed(seed)
    P, Q = K.dists(g, B, N, V, torch.float32)
    parent = K.tree(g, B, N)
    token = K.draw_tokens(g, Q, parent)
    u = torch.rand((B, N), generator=g)
    n_draft = torch.randint(0, N + 1, (B,), generator=g).int()
    return P, Q if draft else None, token, parent, u, n_draft


@pytest.mark.parametrize("kind", ["draft", "points", "greedy"])
@pytest.mark.parametrize("B", [3, 200])
def test_captured_and_on_two_streams(B, kind):
    N, V = 7, 9001
    P, Q, token, parent, u, n_draft = (None if x is None else x.cuda() for x in inputs(1, B, N, V, kind == "draft"))
    given = None if kind == "greedy" else u
    outs = [[torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B,))] for _ in range(3)]
    call = kvq.VerifyDraftCall(P, Q, token, parent, given, *outs[0], n_draft=n_draft)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [kvq.VerifyDraftCall(P, Q, token, parent, given, *o, n_draft=n_draft, stream=s) for o, s in zip(outs[1:], streams)]
    for seed in range(2, 5):
        new = inputs(seed, B, N, V, kind == "draft")
        if kind == "greedy":  # children that are the arg max, half of them
            best = new[0].argmax(-1).gather(1, new[3].long()).int()
            new = new[:2] + (torch.where(new[4] < 0.5, best, new[2]),) + new[3:]
        for x, y in zip((P, Q, token, parent, u, n_draft), new):
            if x is not None:
                x.copy_(y)
        want = K.run_verify(P, Q, token, parent, given, n_draft)
        for o in outs:
            for x in o:
                x.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        for _ in range(3):
            for c in calls:
                c()
        torch.cuda.synchronize()
        for o in outs:
            assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(o, want))
        if B == 200:  # the inputs go both ways
            assert (want[1] > 1).any() and (want[1] < N).any()
    assert kvq.device_error() == 0
