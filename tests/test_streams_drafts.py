"""Workspaces that the binding allocates itself: on the stream the call runs on, whatever stream is
current. The order is checked on the CPU, with streams and allocations that only say where they are; the
GPU test runs the mended calls."""
import contextlib
import types

import numpy as np
import pytest
import torch

from sub_bit_quantized_gb300 import kvq

D = 128


class Streams:
    """Stands in for torch's streams: `now` is the current one's handle, `used` the allocations' and launches'."""

    def __init__(self, monkeypatch):
        self.now, self.used = 1, []
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=self.now))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: None, raising=False)  # as the CPU tensors'
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: self.now, raising=False)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: types.SimpleNamespace(cuda_stream=h))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(kvq, "_operand", lambda name, t, *a, **k: t)
        monkeypatch.setattr(kvq, "_bits", lambda t, *a: t)
        monkeypatch.setattr(kvq, "make_tree_workspace", self.alloc)
        monkeypatch.setattr(kvq, "make_workspace", self.alloc)
        monkeypatch.setattr(kvq, "lib", lambda: self)

    @contextlib.contextmanager
    def on(self, s):
        before, self.now = self.now, s.cuda_stream
        yield
        self.now = before

    def alloc(self, *a, **k):
        self.used.append(("alloc", self.now))
        return torch.zeros(64, dtype=torch.uint8)

    def launch(self, *args):
        s = args[-1]
        self.used.append(("run", (s.value or 0) if hasattr(s, "value") else s))
        return 0

    launch.argtypes = []

    def __getattr__(self, name):
        f = lambda *a: self.launch(*a)  # noqa: E731
        f.argtypes = kvq._SIGS[name][1]
        return f

    def __getitem__(self, name):
        return self.launch


def tree_args():
    cfg = kvq.KiviConfig(n_heads=2, max_batch=1, max_tokens=32)
    cache = types.SimpleNamespace(c_struct=lambda: kvq.KiviCacheC(*([0x10000] * len(kvq.KIVI_CACHE_FIELDS))))
    q, kd = torch.zeros((1, 3, 2, D), dtype=torch.bfloat16), torch.zeros((1, 3, 2, D), dtype=torch.float16)
    return cfg, cache, q, kd, kd, torch.zeros((1, 3), dtype=torch.int64), torch.zeros((1, 3, 2, D))


@pytest.mark.parametrize("stream", [7, 0, types.SimpleNamespace(cuda_stream=9)])
def test_tree_workspace_comes_from_the_stream_of_the_call(monkeypatch, stream):
    s = Streams(monkeypatch)
    kvq.kvq_kivi_tree_attn(*tree_args(), stream=stream)
    h = stream if isinstance(stream, int) else stream.cuda_stream
    assert s.used == [("alloc", h), ("run", h)] and s.now == 1


def test_tree_call_kept_for_several_streams(monkeypatch):
    s = Streams(monkeypatch)
    call = kvq.TreeAttnCall(*tree_args())
    call()
    call()
    assert s.used == [("alloc", 1), ("run", 1), ("run", 1)]
    s.used, s.now = [], 5  # as under `with torch.cuda.stream(other)`
    call()
    call()
    assert s.used == [("alloc", 5), ("run", 5), ("run", 5)]


@pytest.mark.gpu
def test_tree_workspace_is_what_it_says():
    cfg, cache, q, kd, vd, mask, out = [x.cuda() if isinstance(x, torch.Tensor) else x for x in tree_args()]
    size = kvq.kvq_kivi_tree_workspace_size(cfg, 1, 3)
    byte = torch.empty(1, dtype=torch.uint8, device="cuda")
    for ws in (byte.expand(size), torch.empty((size, 2), dtype=torch.uint8, device="cuda")[:, 0],
               torch.empty(size, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="ws"):
            kvq.TreeAttnCall(cfg, cache, q, kd, vd, mask, out, ws=ws)
    kvq.TreeAttnCall(cfg, cache, q, kd, vd, mask, out, ws=torch.empty(size, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
def test_tree_without_a_workspace_captured():
    from tests import _cases as C
    from tests import _drafts as T
    case = T.make_tree_case(4550, B=2, H=4, N=7, n_quant=[32 * 90, 640], n_resid=[50, 128], rep=5, q_scale=0.5)
    cache = C.fill_kivi_cache(case.base)
    want = T.run_tree(case, cache)
    q, kd, vd, mask, nd = T.tensors(case)
    outs = [torch.zeros(q.shape, device="cuda") for _ in range(3)]
    call = kvq.TreeAttnCall(case.base.cfg, cache, q, kd, vd, mask, outs[2], n_draft=nd)
    call()  # the kernels are loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs[:2]:
            kvq.kvq_kivi_tree_attn(case.base.cfg, cache, q, kd, vd, mask, out, n_draft=nd)
        call()
    for _ in range(3):
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert np.array_equal(out.double().cpu().numpy(), want)
    call()  # and eagerly again
    torch.cuda.synchronize()
    assert kvq.device_error() == 0 and np.array_equal(outs[2].double().cpu().numpy(), want)


@pytest.mark.parametrize("stream", [7, types.SimpleNamespace(cuda_stream=9), None])
def test_decode_workspace_comes_from_the_stream_of_the_call(monkeypatch, stream):
    s = Streams(monkeypatch)
    cfg, cache = tree_args()[:2]
    q = torch.zeros((1, 2, D), dtype=torch.bfloat16)
    kvq.kvq_decode_attn(cfg, cache, 0, 1, q, q.float(), stream=stream)
    h = stream if isinstance(stream, int) else stream.cuda_stream if stream else 1
    assert s.used == [("alloc", h), ("run", h)]


@pytest.mark.gpu
def test_tree_calls_on_a_side_stream_without_a_workspace():
    from tests import _cases as C
    from tests import _drafts as T
    case = T.make_tree_case(4500, B=2, H=4, N=7, n_quant=[32 * 90, 640], n_resid=[50, 128], rep=5, q_scale=0.5)
    cache = C.fill_kivi_cache(case.base)
    want = T.run_tree(case, cache)
    q, kd, vd, mask, nd = T.tensors(case)
    out = torch.empty(q.shape, device="cuda")
    size = kvq.kvq_kivi_tree_workspace_size(case.base.cfg, 2, 7)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(20):
        kvq.kvq_kivi_tree_attn(case.base.cfg, cache, q, kd, vd, mask, out, n_draft=nd, stream=side if k % 2 else side.cuda_stream)
        for _ in range(4):  # what the current stream allocates and writes meanwhile
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert kvq.device_error() == 0 and np.array_equal(out.double().cpu().numpy(), want)
    call = kvq.TreeAttnCall(case.base.cfg, cache, q, kd, vd, mask, out, n_draft=nd)
    for st in (torch.cuda.current_stream(), side, torch.cuda.current_stream()):
        torch.cuda.synchronize()
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            call()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.mark.gpu
def test_decode_on_a_side_stream_without_a_workspace():
    from tests import _cases as C
    case = C.make_kivi_case(4600, B=1, H=2, n_quant=[32 * 200], n_resid=[60], Hq=8)
    cache = C.fill_kivi_cache(case)
    q = C.bf16_tensor(case.q)
    out, want = torch.empty(q.shape, device="cuda"), torch.empty(q.shape, device="cuda")
    kvq.kvq_decode_attn(case.cfg, cache, 0, 1, q, want)
    size = kvq.kvq_decode_workspace_size(case.cfg, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(20):
        out.zero_()
        torch.cuda.synchronize()
        kvq.kvq_decode_attn(case.cfg, cache, 0, 1, q, out, stream=side if k % 2 else side.cuda_stream)
        for _ in range(4):
            torch.full((max(size, 1),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert (out - want).abs().max() <= 2.0 ** -20 * want.abs().max()  # fp32 sums, in any order
    assert kvq.device_error() == 0
