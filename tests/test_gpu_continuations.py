"""GPU parity of the operators that serve many continuations of one prompt: attention under a shared
prefix, slots that continue others, verification of drafted tokens. Attention against fp64 within the
roundings that tests/_continuations.py counts; the others exactly."""
import numpy as np
import pytest
import torch

from oracle import continuations as oc
from sub_bit_quantized_gb300 import kvq
from tests import _cases as C
from tests import _continuations as K
from tests import _drafts as T

pytestmark = pytest.mark.gpu
D = 128


# ------------------------------------------------------------------------------------ prefix

def prefix_case(seed, B, H, rep, N, own, pre, kb=2, vb=2, residual=128, nqv=None, n_draft=None, pkb=None, pvb=None,
                presid=128, slots=1, **kw):
    """own, pre: (quantized, fp16) tokens, one pair or one for each request / slot."""
    per = lambda x, n: [x] * n if isinstance(x, tuple) else list(x)  # noqa: E731
    own, pre = per(own, B), per(pre, slots)
    case = T.make_tree_case(seed, B, H, N, [o[0] for o in own], [o[1] for o in own], rep=rep, n_draft=n_draft, k_bits=kb,
                            v_bits=vb, residual=residual, **kw)
    prefix = C.make_kivi_case(seed + 7, slots, H, [p[0] for p in pre], [p[1] for p in pre], residual=presid, Hq=H * rep,
                              k_bits=pkb or kb, v_bits=pvb or vb, n_quant_v=nqv)
    return case, prefix


SHAPES = [  # B, H, rep, N: rows a KV head over the prefix 1, 8, 12, 15, 30, 64, 70, 140, 268
    (1, 1, 1, 1), (2, 2, 4, 1), (3, 1, 4, 1), (5, 1, 1, 3), (5, 2, 2, 3), (16, 1, 4, 1), (10, 1, 7, 1), (5, 1, 4, 7),
    (67, 1, 4, 1)]


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("B,H,rep,N", SHAPES)
def test_prefix_rows_and_bits(B, H, rep, N, kb, vb):
    case, prefix = prefix_case(B * 100 + N, B, H, rep, N, (64, 9), (192, 77), kb, vb)
    ref, bound = K.prefix_reference(case, prefix, 0)
    T.check_rows(K.run_prefix(case, prefix), ref, bound, 7.0)


@pytest.mark.parametrize("kb,vb", [(4, 4), (4, 2), (2, 2)])
@pytest.mark.parametrize("B,H,rep,N", [(11, 2, 3, 1), (33, 1, 4, 1), (13, 1, 4, 5)])
def test_prefix_bf16_outputs_of_many_rows(B, H, rep, N, kb, vb):
    # 4-bit keys enter rounded to one fp16: 2^-11 of themselves, which the bound counts; then half a step of bf16
    case, prefix = prefix_case(B * 10 + N, B, H, rep, N, (32, 9), (288, 50), kb, vb)
    ref, bound = K.prefix_reference(case, prefix, 0)
    got = K.run_prefix(case, prefix, dtype=torch.bfloat16)
    T.check_rows(got, ref, bound + 2.0 ** -8 * (np.abs(np.nan_to_num(ref)) + bound), 7.0)


@pytest.mark.parametrize("B,rep", [(3, 2), (40, 2)])
def test_prefix_without_residuals_and_padding_without_drafts(B, rep):
    # attention-only caches (residual 0) hold quantized tokens alone; rows behind n_draft are padding without drafts too
    case, prefix = prefix_case(31, B, 2, rep, 3, (64, 0), (224, 0), 4, 2, residual=0, presid=0, n_draft=[b % 4 for b in range(B)])
    ref, bound = K.prefix_reference(case, prefix, 0, drafts=False)
    T.check_rows(K.run_prefix(case, prefix, drafts=False), ref, bound, 7.0)


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("B,H,rep", [(10, 32, 1), (39, 8, 1), (77, 4, 2), (155, 2, 4), (310, 1, 4), (103, 1, 3)])
def test_prefix_one_row_a_request_and_many_of_them(B, H, rep, kb, vb):
    # from two blocks an SM on a request's own tokens are attended as the decode does, its drafted token apart; some
    # requests hold nothing, some are padding, some do not see their drafted token
    own = [(0, 0) if b % 7 == 0 else (32 * (b % 3), 1 + b % 30) for b in range(B)]
    case, prefix = prefix_case(B + H, B, H, rep, 1, own, (96, 20), kb, vb, residual=32 * (1 + B % 3),
                               n_draft=[0 if b % 11 == 3 else 1 for b in range(B)])
    case.mask[::5] = 0
    ref, bound = K.prefix_reference(case, prefix, 0)
    T.check_rows(K.run_prefix(case, prefix), ref, bound, 7.0)
    got = K.run_prefix(case, prefix, dtype=torch.bfloat16)
    T.check_rows(got, ref, bound + 2.0 ** -8 * (np.abs(np.nan_to_num(ref)) + bound), 7.0)
    ref, bound = K.prefix_reference(case, prefix, 0, drafts=False)
    T.check_rows(K.run_prefix(case, prefix, drafts=False), ref, bound, 7.0)
    case.vd[::5] = np.nan  # unseen
    ref, bound = K.prefix_reference(case, prefix, 0, drafts=False)
    got = K.run_prefix(case, prefix)
    rows = [b for b in range(0, B, 5) if case.n_draft[b]]
    T.check_rows(got[rows], ref[rows], bound[rows], 7.0)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -30, 2.0 ** 12, 2.0 ** 60])
@pytest.mark.parametrize("B", [3, 40])
def test_prefix_queries_of_any_magnitude(B, scale):
    # tiny ones average the values, huge ones pick the largest score's
    case, prefix = prefix_case(32, B, 1, 2, 1, (32, 5), (160, 40), 2, 2)
    case.q = case.q * scale
    case.q = np.asarray(case.q, np.float32).astype(np.float64)
    got = K.run_prefix(case, prefix)
    ref, bound = K.prefix_reference(case, prefix, 0)
    assert np.isfinite(got).all()
    if scale < 1:
        T.check_rows(got, ref, bound, 7.0)
    else:  # a row whose two best scores lie further apart than their errors is the best token's value
        for b in range(B):
            K0, V0, _, _ = T.context(prefix, 0, 0)
            K1, V1, _, _ = T.context(case.base, b, 0)
            k = np.concatenate([K0, K1, case.kd[b, :, 0]]).astype(np.float64)
            v = np.concatenate([V0, V1, case.vd[b, :, 0]]).astype(np.float64)
            for r in range(2):
                s = np.sort(k @ case.q[b, 0, r])
                if (s[-1] - s[-2]) / np.sqrt(D) > 60 + 2.0 ** -9 * np.abs(s).max() / np.sqrt(D):
                    best = v[np.argmax(k @ case.q[b, 0, r])]
                    assert np.abs(got[b, 0, r] - best).max() <= 2.0 ** -9 * (np.abs(best).max() + 8), (b, r)


def test_prefix_workspace_of_the_calls_own_on_other_streams():
    make, out, ref, bound, _ = prepared(33, 40, 2, (96, 10))
    call = make(None)
    for s in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s) if s is not None else torch.cuda.stream(torch.cuda.current_stream()):
            call()
        torch.cuda.synchronize()
        T.check_rows(out.double().cpu().numpy(), ref, bound, 7.0)


@pytest.mark.parametrize("n,nqk,nqv", [(1, 0, 0), (31, 0, 0), (127, 32, 10), (128, 64, 64), (129, 96, 33), (160, 160, 160),
                                       (300, 192, 175), (515, 512, 401)])
@pytest.mark.parametrize("B,rep", [(3, 1), (9, 4), (40, 4)])
def test_prefix_lengths(B, rep, n, nqk, nqv):
    own = [(0, 0) if b % 3 == 0 else (32 * (b % 4), 1 + b) for b in range(B)]  # some requests hold nothing yet
    case, prefix = prefix_case(n, B, 1, rep, 1, own, (nqk, n - nqk), 4, 2, nqv=[nqv])
    ref, bound = K.prefix_reference(case, prefix, 0)
    T.check_rows(K.run_prefix(case, prefix), ref, bound, 7.0)


@pytest.mark.parametrize("B,rep,N", [(2, 1, 1), (6, 4, 3), (30, 4, 3)])
def test_prefix_without_drafts(B, rep, N):
    own = [(0, 0) if b == 1 else (64, b) for b in range(B)]
    case, prefix = prefix_case(11, B, 2, rep, N, own, (96, 5))
    ref, bound = K.prefix_reference(case, prefix, 0, drafts=False)
    T.check_rows(K.run_prefix(case, prefix, drafts=False), ref, bound, 7.0)


@pytest.mark.parametrize("B,rep,N", [(2, 2, 2), (20, 4, 2)])
def test_prefix_empty_on_either_side(B, rep, N):
    case, prefix = prefix_case(12, B, 1, rep, N, (0, 0), (0, 0))
    case.mask[0] = 0
    ref, bound = K.prefix_reference(case, prefix, 0)  # drafts alone; request 0 attends nothing
    got = K.run_prefix(case, prefix)
    T.check_rows(got, ref, bound, 7.0)
    assert not got[0].any()
    assert not K.run_prefix(case, prefix, drafts=False).any()
    case, prefix = prefix_case(13, B, 1, rep, N, (32, 4), (0, 0))
    ref, bound = K.prefix_reference(case, prefix, 0)
    T.check_rows(K.run_prefix(case, prefix), ref, bound, 7.0)


@pytest.mark.parametrize("B,rep", [(6, 1), (24, 3)])
def test_prefix_padding_slots_and_shapes(B, rep):
    # padding tokens, slot 2 of a prefix cache with other bits, residual and capacity
    nd = [(3, 0, 5, -1, 9, 1)[b % 6] for b in range(B)]
    case, prefix = prefix_case(14, B, 2, rep, 5, (32, 20), [(64, 3), (0, 7), (224, 50), (32, 0)], 2, 4, residual=64,
                               n_draft=nd, pkb=4, pvb=2, presid=96, slots=4)
    ref, bound = K.prefix_reference(case, prefix, 2)
    T.check_rows(K.run_prefix(case, prefix, slot=2), ref, bound, 7.0)
    got = K.run_prefix(case, prefix, slot=2, dtype=torch.bfloat16)
    T.check_rows(got, ref, bound + 2.0 ** -8 * (np.abs(np.nan_to_num(ref)) + bound), 7.0)


@pytest.mark.parametrize("B", [2, 33])
def test_prefix_of_the_same_cache(B):
    # the prefix is a slot of the batch's own cache, behind the requests
    case, _ = prefix_case(15, B + 1, 1, 4, 1, [(32, b % 5) for b in range(B)] + [(256, 30)], (0, 0))
    cache = C.fill_kivi_cache(case.base)
    q, kd, vd, mask, _ = T.tensors(case)
    out = torch.empty_like(q[:B], dtype=torch.float32)
    kvq.kvq_kivi_prefix_attn(case.base.cfg, cache, case.base.cfg, cache, B, q[:B], out, kd[:B], vd[:B], mask[:B])
    ref, bound = K.prefix_reference(case, case.base, B)
    T.check_rows(out.double().cpu().numpy(), ref[:B], bound[:B], 7.0)


@pytest.mark.parametrize("B,rep", [(4, 1), (40, 4)])
@pytest.mark.parametrize("side", ["prefix", "own"])
def test_prefix_one_side_outweighs_the_other(B, rep, side):
    case, prefix = prefix_case(16, B, 1, rep, 1, (64, 12), (128, 40))
    base = prefix if side == "prefix" else case.base
    base.k_res[:] *= np.float16(8)    # scores of some tens to hundreds
    ref, bound = K.prefix_reference(case, prefix, 0)
    T.check_rows(K.run_prefix(case, prefix), ref, bound, 7.0)


@pytest.mark.parametrize("B,rep", [(2, 1), (40, 4)])
def test_prefix_values_that_are_not_finite(B, rep):
    # a drafted value that a row does not see changes nothing; one of the prefix reaches every row
    case, prefix = prefix_case(17, B, 1, rep, 3, (32, 3), (64, 20))
    clean = K.run_prefix(case, prefix)
    case.vd[:, 2] = np.inf
    case.mask[:, 2] = 0b011
    case.mask[:, 0], case.mask[:, 1] = 0b001, 0b010
    ref, bound = K.prefix_reference(case, prefix, 0)
    got = K.run_prefix(case, prefix)
    assert np.isfinite(got).all() and np.isfinite(clean).all()
    keep = np.where(np.isinf(case.vd), 0, case.vd)
    case.vd = keep
    ref, bound = K.prefix_reference(case, prefix, 0)
    T.check_rows(got, ref, bound, 7.0)
    prefix.v_res[0, 0, 6, 5] = np.nan  # of token 70
    got = K.run_prefix(case, prefix)
    assert np.isnan(got[..., 5]).all() and np.isfinite(got[..., :5]).all()


def prepared(seed, B, rep, pre):
    case, prefix = prefix_case(seed, B, 2, rep, 2, (64, 9), pre)
    cache, pcache = C.fill_kivi_cache(case.base), C.fill_kivi_cache(prefix)
    q, kd, vd, mask, nd = T.tensors(case)
    out = torch.zeros(q.shape, device="cuda")
    make = lambda ws, stream=None, out=out: kvq.PrefixAttnCall(  # noqa: E731
        case.base.cfg, cache, prefix.cfg, pcache, 0, q, out, kd, vd, mask, nd, ws=ws, stream=stream)
    ref, bound = K.prefix_reference(case, prefix, 0)
    return make, out, ref, bound, lambda: kvq.make_prefix_workspace(case.base.cfg, prefix.cfg, B, 2)


@pytest.mark.parametrize("B,rep", [(2, 2), (50, 4)])
def test_prefix_in_a_graph_and_on_two_streams(B, rep):
    make, out, ref, bound, ws = prepared(18, B, rep, (320, 40))
    call = make(ws())
    call()
    torch.cuda.synchronize()
    once = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, once)
    T.check_rows(out.double().cpu().numpy(), ref, bound, 7.0)
    outs = [torch.zeros_like(out) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [make(ws(), stream=s, out=o) for s, o in zip(streams, outs)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c in calls:
            c()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], once) and torch.equal(outs[1], once)
    assert kvq.device_error() == 0


@pytest.mark.parametrize("B,rep,n", [(2, 4, 20000), (96, 4, 6000)])
def test_prefix_long(B, rep, n):
    # thousands of tokens split over the blocks, against torch in fp64
    case, prefix = prefix_case(19, B, 2, rep, 1, (32, 3), (n // 32 * 32, 19), 4, 4)
    got = torch.from_numpy(K.run_prefix(case, prefix))
    for h in range(2):
        K0, V0, _, _ = T.context(prefix, 0, h)
        K0, V0 = torch.from_numpy(K0).cuda(), torch.from_numpy(V0).cuda()
        for b in range(0, B, 7):
            K1, V1, _, _ = T.context(case.base, b, h)
            k = torch.cat([K0, torch.from_numpy(K1).cuda(), torch.from_numpy(case.kd[b, :, h]).cuda().double()])
            v = torch.cat([V0, torch.from_numpy(V1).cuda(), torch.from_numpy(case.vd[b, :, h]).cuda().double()])
            q = torch.from_numpy(case.q[b, 0, h * rep:(h + 1) * rep]).cuda().double()
            ref = torch.softmax(q @ k.T / D ** 0.5, -1) @ v
            C.check_close(got[b, 0, h * rep:(h + 1) * rep].numpy(), ref.cpu().numpy())


# ------------------------------------------------------------------------------------ fork

def kivi_cache(seed, B, H, T, R=64, kb=2, vb=4, full=False):
    """A cache of random bytes with valid lengths; (config, cache)."""
    cfg = kvq.KiviConfig(n_heads=H, k_bits=kb, v_bits=vb, residual=R, max_batch=B, max_tokens=T)
    cache = kvq.KiviCache(cfg)
    g = np.random.default_rng(seed)
    for name in K.KIVI_ARRAYS:
        t = getattr(cache, name)
        t.view(torch.uint8).copy_(torch.from_numpy(g.integers(0, 256, t.view(torch.uint8).shape, np.uint8)))
    for b in range(B):
        nqk = int(T if full else 32 * g.integers(0, T // 32 + 1))
        n = nqk + int(g.integers(0, R + 1))
        nqv = int(g.integers(max(0, n - R), nqk + 1))
        cache.n_tok[b], cache.n_quant_k[b], cache.n_quant_v[b] = n, nqk, nqv
    return cfg, cache


def vq_cache(seed, B, H, P, L=2, T=2, recent=64, Tc=1, G=8):
    cfg = kvq.VqConfig(T=T, Tc=Tc, G=G, n_layers=L, n_heads=H, recent=recent, max_pages=P, max_batch=B, max_ctx=8 * P + 500)
    cache = kvq.VqCache(cfg)
    g = np.random.default_rng(seed)
    for name in K.VQ_ARRAYS:
        t = getattr(cache, name)
        t.view(torch.uint8).copy_(torch.from_numpy(g.integers(0, 256, t.view(torch.uint8).shape, np.uint8)))
    for b in range(B):
        pages = int(g.integers(0, P + 1))
        n = 8 + 8 * pages + int(g.integers(recent, recent + 8)) if pages else int(g.integers(0, 8 + recent + 8))
        cache.seq_len[b], cache.n_pages[b] = n, pages
    return cfg, cache


def host(cache):
    vq = isinstance(cache, kvq.VqCache)
    arrays = {n: getattr(cache, n).view(torch.uint8).cpu().numpy() for n in (K.VQ_ARRAYS if vq else K.KIVI_ARRAYS)}
    lens = {n: getattr(cache, n).cpu().numpy() for n in (("seq_len", "n_pages") if vq else ("n_tok", "n_quant_k", "n_quant_v"))}
    return arrays, lens


def check_fork(cfg, cache, source, b0=0, from_cfg=None, from_cache=None, expected=None):
    """The call against the oracle, every byte of the cache (``expected``: the source as the oracle is to take it)."""
    arrays, lens = host(cache)
    src, src_lens = (arrays, lens) if from_cache is None else host(from_cache)
    kvq.kvq_cache_fork(cfg, cache, torch.tensor(source, dtype=torch.int32, device="cuda"), from_cfg, from_cache, b0)
    torch.cuda.synchronize()
    if isinstance(cache, kvq.VqCache):
        rows, dim = (lambda name, *n: oc.vq_rows(name, *n, cfg.sink, cfg.recent)), 2
    else:
        rows, dim = (lambda name, *n: oc.kivi_rows(name, *n, cfg.residual)), 0
    oc.fork(arrays, src, lens, src_lens, source if expected is None else expected, b0, dim, rows)
    got, got_lens = host(cache)
    for name in lens:
        assert np.array_equal(got_lens[name], lens[name]), name
    for name in arrays:
        assert np.array_equal(got[name], arrays[name]), name


def maps(B):
    g = np.random.default_rng(B)
    some = np.where(g.random(B) < 0.5, np.arange(B), g.integers(0, B, B))
    return {"keep": [oc.KEEP] * B, "self": list(range(B)), "free": [oc.FREE] * B, "one": [B // 2] * B,
            "shift": [(i + 1) % B for i in range(B)], "chain": [oc.KEEP] + list(range(B - 1)),
            "swap": [i ^ 1 if i ^ 1 < B else oc.KEEP for i in range(B)],
            "permutation": [int(x) for x in g.permutation(B)], "any": [int(x) for x in g.integers(0, B, B)],
            "some": [int(x) for x in some], "mixed": [int(x) for x in g.integers(-2, B, B)],
            "compact": list(range(B // 3, B)) + [oc.FREE] * (B // 3)}


@pytest.mark.parametrize("name", list(maps(4)))
@pytest.mark.parametrize("B", [1, 2, 7, 16, 17, 40])
def test_fork_in_place(B, name):
    cfg, cache = kivi_cache(B, B, 3, 96)
    check_fork(cfg, cache, maps(B)[name])
    assert kvq.device_error() == 0
    cfg, cache = vq_cache(B, B, 2, 5)
    check_fork(cfg, cache, maps(B)[name])
    assert kvq.device_error() == 0


@pytest.mark.parametrize("name", ["permutation", "any", "shift", "one", "mixed"])
@pytest.mark.parametrize("B", [100, 256])
def test_fork_of_many_slots(B, name):
    cfg, cache = kivi_cache(B, B, 1, 64, R=32, kb=4, vb=2)
    check_fork(cfg, cache, maps(B)[name])
    cfg, cache = vq_cache(B, B, 1, 3, L=1, T=1)
    check_fork(cfg, cache, maps(B)[name])
    assert kvq.device_error() == 0


@pytest.mark.parametrize("R", [0, 32, 128])
def test_fork_from_another_cache(R):
    for (kb, vb), (T, F) in (((2, 2), (320, 160)), ((4, 2), (96, 96))):
        cfg, cache = kivi_cache(1, 9, 2, T, R, kb, vb)
        if R == 0:
            cache.n_tok.copy_(cache.n_quant_k)
            cache.n_quant_v.copy_(cache.n_quant_k)
        other_cfg, other = kivi_cache(2, 3, 2, F, R, kb, vb)
        if R == 0:
            other.n_tok.copy_(other.n_quant_k)
            other.n_quant_v.copy_(other.n_quant_k)
        other_cfg.n_q_heads = 8
        check_fork(cfg, cache, [2, 0, 0, oc.KEEP, oc.FREE, 1], 2, other_cfg, other)
    cfg, cache = vq_cache(3, 5, 2, 9, recent=256, Tc=2, G=16)
    other_cfg, other = vq_cache(4, 2, 2, 6, recent=256, Tc=2, G=16)
    check_fork(cfg, cache, [1, oc.FREE, 0, 0], 1, other_cfg, other)
    assert kvq.device_error() == 0


def test_fork_leaves_what_it_cannot_move():
    cfg, cache = kivi_cache(5, 6, 2, 64)
    for bad in (-3, 6, 1 << 30, -(1 << 31)):
        check_fork(cfg, cache, [1, bad, 0, oc.KEEP, 2, oc.FREE], expected=[1, oc.KEEP, 0, oc.KEEP, 2, oc.FREE])
        assert kvq.device_error() == kvq.ERR_INVALID_ARG
    for n, nqk, nqv in ((-1, 0, 0), (40, 32, 33), (30, 32, 32), (200, 64, 64), (50, 20, 20), (160, 96, 96)):
        cfg, cache = kivi_cache(6, 3, 2, 64)
        cache.n_tok[0], cache.n_quant_k[0], cache.n_quant_v[0] = n, nqk, nqv
        check_fork(cfg, cache, [oc.KEEP, 0, 1], expected=[oc.KEEP, oc.KEEP, 1])
        assert kvq.device_error() == kvq.ERR_INVALID_ARG
    small_cfg, small = kivi_cache(7, 2, 2, 32)
    cfg, cache = kivi_cache(8, 2, 2, 96, full=True)
    check_fork(small_cfg, small, [oc.FREE, 0], 0, cfg, cache, expected=[oc.FREE, oc.KEEP])
    assert kvq.device_error() == kvq.ERR_CAPACITY
    cfg, cache = vq_cache(9, 3, 1, 4)
    for n, pages in ((20, 4), (400, 4), (8, -1), (48, 5)):
        cache.seq_len[2], cache.n_pages[2] = n, pages
        check_fork(cfg, cache, [2, 0, oc.KEEP], expected=[oc.KEEP, 0, oc.KEEP])
        assert kvq.device_error() == kvq.ERR_INVALID_ARG


def test_fork_in_a_graph():
    cfg, cache = kivi_cache(10, 8, 2, 160)
    source = torch.full((8,), kvq.SLOT_KEEP, dtype=torch.int32, device="cuda")
    call = kvq.CacheForkCall(cfg, cache, source)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(4):
        arrays, lens = host(cache)
        new = [int(x) for x in np.random.default_rng(turn).integers(-2, 8, 8)]
        source.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        oc.fork(arrays, arrays, lens, lens, new, 0, 0, lambda name, *n: oc.kivi_rows(name, *n, cfg.residual))
        got, got_lens = host(cache)
        assert all(np.array_equal(got[n], arrays[n]) for n in arrays) and all(np.array_equal(got_lens[n], lens[n]) for n in lens)
    assert kvq.device_error() == 0


# ------------------------------------------------------------------------------------ verify

def check_verify(P, Q, token, parent, u, n_draft=None):
    path, count, nxt = K.run_verify(P, Q, token, parent, u, n_draft)
    assert kvq.device_error() == 0
    B, N, _ = P.shape
    Pn, Qn = P.double().cpu().numpy(), None if Q is None else Q.double().cpu().numpy()
    walked = 0
    for b in range(B):
        nd = N if n_draft is None else min(max(int(n_draft[b]), 0), N)
        want, token_next = oc.verify(Pn[b], None if Q is None else Qn[b], token[b].tolist(), parent[b].tolist(),
                                     None if u is None else u[b].numpy(), nd)
        assert count[b] == len(want) and path[b, :len(want)].tolist() == want, b
        assert (path[b, len(want):] == -7).all()
        assert nxt[b] == (-7 if nd == 0 else token_next), b
        walked += len(want)
    return walked


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,N,V", [(1, 1, 1), (3, 4, 2), (2, 5, 511), (5, 9, 2049), (2, 17, 8192), (3, 6, 20011), (1, 64, 3001),
                                   (160, 3, 700)])
@pytest.mark.parametrize("kind", ["chain", "tree", "points", "greedy"])
def test_verify(B, N, V, dtype, kind):
    g = torch.Generator().manual_seed(B * 1000 + N)
    P, Q = K.dists(g, B, N, V, dtype)
    parent = K.tree(g, B, N, chain=kind == "chain")
    token = K.draw_tokens(g, P if kind in ("points", "greedy") else Q, parent)
    n_draft = torch.randint(0, N + 2, (B,), generator=g).int() if B > 1 else None
    u = torch.rand((B, N), generator=g)
    if kind == "greedy":
        best = P.float().argmax(-1).gather(1, parent.long().clamp(min=0)).int()
        token = torch.where(torch.rand((B, N), generator=g) < 0.7, best, token)
        u = None
    check_verify(P, Q if kind in ("chain", "tree") else None, token, parent, u, n_draft)


@pytest.mark.parametrize("V", [3001, 65536])
def test_verify_many_children_of_one_node(V):
    # rejection after rejection at the root, the draft far from the target
    g = torch.Generator().manual_seed(V)
    P, Q = K.dists(g, 6, 20, V, torch.float32, near=3.0, sharp=1.0)
    parent = torch.zeros((6, 20), dtype=torch.int32)
    token = K.draw_tokens(g, Q, parent)
    u = torch.rand((6, 20), generator=g) * 0.2 + 0.79
    check_verify(P, Q, token, parent, u)
    check_verify(P, None, token, parent, u)          # the same token twice among them


def test_verify_border_cases():
    g = torch.Generator().manual_seed(4)
    P, Q = K.dists(g, 4, 4, 1000, torch.float32)
    parent = K.tree(g, 4, 4, chain=True)
    token = K.draw_tokens(g, Q, parent)
    top = 1 - 2.0 ** -24
    for x in (0.0, top):
        for y in (0.0, top):  # the next token's number, the tests'
            u = torch.full((4, 4), y)
            u[:, 0] = x
            check_verify(P, Q, token, parent, u)
            check_verify(P, None, token, parent, u)
    check_verify(P, P, token, parent, torch.full((4, 4), top))   # p = q: everything is accepted
    P[:, :, ::2] = 0                                              # tokens that the target never says
    Q[:, :, 1::2] = 0
    token = token // 2 * 2
    check_verify(P, Q, token, parent, torch.rand((4, 4), generator=g))
    check_verify(P, Q, token, parent, torch.zeros((4, 4)))
    # all mass on the rejected token: the residual is empty and the target itself is drawn from
    P = torch.zeros((1, 2, 600))
    P[:, :, 77] = 1
    token, parent = torch.tensor([[0, 77]], dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    Q = P * 2
    path, count, nxt = K.run_verify(P, Q, token, parent, torch.tensor([[0.3, 0.9]]))
    assert count[0] == 1 and nxt[0] == 77
    # no mass at all: some token in range
    path, count, nxt = K.run_verify(torch.zeros((2, 2, 600)), None, token.repeat(2, 1), parent.repeat(2, 1), torch.full((2, 2), 0.5))
    assert (count == 1).all() and ((nxt >= 0) & (nxt < 600)).all()
    assert kvq.device_error() == 0


@pytest.mark.parametrize("V", [1, 700, 9001])
def test_verify_greedy_ties_infinities_and_nan(V):
    g = torch.Generator().manual_seed(V)
    P = torch.randint(-3, 4, (8, 3, V), generator=g).float()     # many ties: the lowest index
    P[1, :, :] = -np.inf
    P[2, :, :] = np.nan
    P[3, :, V // 2:] = np.nan
    P[4, :, V // 3] = np.inf
    P[5, :, :] = -0.0
    P[5, :, V - 1] = 0.0                                          # equal to -0
    best = torch.tensor([[int(np.argmax(np.where(np.isnan(r), -np.inf, r))) for r in p] for p in P.numpy()], dtype=torch.int32)
    parent = torch.tensor([[0, 0, 1]] * 8, dtype=torch.int32)
    token = torch.stack([best[:, 0], best[:, 0], best[:, 1]], 1)
    for dt in (torch.float32, torch.bfloat16):
        assert check_verify(P.to(dt), None, token, parent, None) == 24


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 9, 517, 5003, 50021])
def test_verify_greedy_paths_of_every_length(V, dt):
    # chains accepted up to node k, and the same behind a rejected first child of every node
    g = torch.Generator().manual_seed(V)
    N = 9
    P = torch.randint(-50, 50, (2 * N, N, V), generator=g).to(dt)
    best = torch.from_numpy(P.float().numpy().argmax(-1).astype(np.int32))
    parent = torch.zeros((2 * N, N), dtype=torch.int32)
    token = torch.zeros((2 * N, N), dtype=torch.int32)
    for k in range(N):
        parent[k, 1:] = torch.arange(N - 1)
        token[k, 1:] = best[k, :-1]
        if k + 1 < N:
            token[k, k + 1] = (best[k, k] + 1) % V
        # nodes 1, 3, 5, 7 rejected where there is another token, 2, 4, 6, 8 go on up to the k-th
        b = N + k
        for i in range(1, N):
            parent[b, i] = 2 * ((i - 1) // 2)
            token[b, i] = best[b, parent[b, i]] if i % 2 == 0 and i <= k else (best[b, parent[b, i]] + 1) % V
    accepted = check_verify(P, None, token, parent, None)
    if V > 1:
        assert accepted == sum(range(1, N + 1)) + sum(1 + k // 2 for k in range(N))


def test_verify_strides_and_alignment():
    g = torch.Generator().manual_seed(9)
    P, Q = K.dists(g, 3, 5, 1003, torch.float32)
    parent = K.tree(g, 3, 5)
    token, u = K.draw_tokens(g, Q, parent), torch.rand((3, 5), generator=g)
    wide = torch.zeros((3, 7, 1024), device="cuda")
    wide[:, 1:6, :1003] = P.cuda()
    odd = torch.zeros((5, 3, 1005), device="cuda")
    odd[:, :, :1003] = Q.cuda().transpose(0, 1)
    want = K.run_verify(P, Q, token, parent, u)
    got = K.run_verify(wide[:, 1:6, :1003], odd.transpose(0, 1)[:, :, :1003], token, parent, u)
    assert all(np.array_equal(x, y) for x, y in zip(want, got))
    # one row for every node and request (strides of 0)
    one = P[:1, :1].cuda().expand(3, 5, 1003)
    check_verify(one, None, token, parent, u)


def test_verify_leaves_requests_with_bad_trees():
    g = torch.Generator().manual_seed(10)
    P, Q = K.dists(g, 7, 4, 300, torch.float32)
    parent = K.tree(g, 7, 4)
    token, u = K.draw_tokens(g, Q, parent), torch.rand((7, 4), generator=g)
    good = K.run_verify(P, Q, token, parent, u)
    token, parent = token.clone(), parent.clone()
    parent[1, 2], parent[2, 3], parent[3, 1] = 2, -1, 1 << 30
    token[4, 1], token[5, 0] = 300, -1
    path, count, nxt = K.run_verify(P, Q, token, parent, u)
    assert kvq.device_error() == kvq.ERR_INVALID_ARG
    for b in range(7):
        if 1 <= b <= 5:
            assert count[b] == 0 and nxt[b] == -7 and (path[b] == -7).all()
        else:
            assert count[b] == good[1][b] and nxt[b] == good[2][b] and np.array_equal(path[b], good[0][b])
    parent[0, 0] = 99  # not read
    n_draft = torch.tensor([4, 2, 3, 1, 1, 0, 4], dtype=torch.int32)  # bad nodes behind the last one do not count
    token[5, 0] = 5
    path, count, nxt = K.run_verify(P, Q, token, parent, u, n_draft)
    assert kvq.device_error() == 0 and (count[[0, 1, 2, 3, 4, 6]] >= 1).all() and count[5] == 0


def test_verified_tokens_follow_the_target():
    # the point of it: whatever the draft, the first new token is distributed as the target says. 60000 draws over 4
    # tokens: a share's standard deviation is below sqrt(0.25 / 60000) = 0.00205; five of them
    g = torch.Generator().manual_seed(11)
    n = 60000
    p, q = torch.tensor([0.1, 0.45, 0.15, 0.3]), torch.tensor([0.4, 0.1, 0.3, 0.2])
    P, Q = p.expand(n, 4, 4).cuda(), q.expand(n, 4, 4).cuda()
    parent = torch.zeros((n, 4), dtype=torch.int32)               # three children of the root, drawn from q
    token = torch.multinomial(q.expand(n, 4), 4, replacement=True, generator=g).int()
    path, count, nxt = K.run_verify(P, Q, token, parent, torch.rand((n, 4), generator=g))
    first = np.where(count > 1, token.numpy()[np.arange(n), path[:, 1].clip(0)], nxt)
    share = np.bincount(first, minlength=4) / n
    assert np.abs(share - p.numpy()).max() < 5 * 0.00205
    token = torch.stack([torch.randperm(4, generator=g) for _ in range(2000)]).int().repeat(30, 1)  # points: any tokens
    path, count, nxt = K.run_verify(P, None, token, parent, torch.rand((n, 4), generator=g))
    first = np.where(count > 1, token.numpy()[np.arange(n), path[:, 1].clip(0)], nxt)
    assert np.abs(np.bincount(first, minlength=4) / n - p.numpy()).max() < 5 * 0.00205


# ------------------------------------------------------------------------------------ together

def test_a_serving_step():
    """A prompt cached once; a slot takes over another; drafts attend under the prefix, are verified and committed; the
    next step attends what was committed."""
    g = torch.Generator(device="cuda").manual_seed(21)
    B, H, rep, N, V, R = 4, 2, 2, 5, 500, 64
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    cfg = kvq.KiviConfig(n_heads=H, n_q_heads=H * rep, residual=R, max_batch=B, max_tokens=128)
    pcfg = kvq.KiviConfig(n_heads=H, n_q_heads=H * rep, residual=R, max_batch=1, max_tokens=320)
    cache, prefix = kvq.KiviCache(cfg), kvq.KiviCache(pcfg)
    kvq.kvq_kivi_prefill(pcfg, prefix, rnd(1, H, 300, D).half(), rnd(1, H, 300, D).half())
    kvq.kvq_kivi_prefill(cfg, cache, rnd(B, H, 90, D).half(), rnd(B, H, 90, D).half())
    kvq.kvq_cache_fork(cfg, cache, torch.tensor([-1, 0, -1, -2], dtype=torch.int32, device="cuda"))
    assert cache.n_tok.tolist() == [90, 90, 90, 0]
    parent = K.tree(torch.Generator().manual_seed(3), B, N)
    mask = torch.zeros((B, N), dtype=torch.int64)
    for b in range(B):
        for i in range(N):
            mask[b, i] = (int(mask[b, parent[b, i]]) if i else 0) | 1 << i
    mask, parent = mask.cuda(), parent.cuda()
    for step in range(3):
        q, kd, vd = rnd(B, N, H * rep, D).bfloat16(), rnd(B, N, H, D).half(), rnd(B, N, H, D).half()
        out = torch.empty((B, N, H * rep, D), device="cuda")
        kvq.kvq_kivi_prefix_attn(cfg, cache, pcfg, prefix, 0, q, out, kd, vd, mask)
        lens = cache.n_tok.tolist()
        # what the caches hold, read back, attended in fp64
        read = lambda c, cc, n, b: [x.double() for x in read_back(c, cc, n, b)]  # noqa: E731
        k0, v0 = read(pcfg, prefix, 300, 0)
        for b in range(B):
            k1, v1 = read(cfg, cache, lens[b], b)
            for i in range(N):
                see = [j for j in range(N) if int(mask[b, i]) >> j & 1]
                k = torch.cat([k0, k1, kd[b, see].double().transpose(0, 1)], 1)
                v = torch.cat([v0, v1, vd[b, see].double().transpose(0, 1)], 1)
                x = q[b, i].double().view(H, rep, D)
                ref = torch.softmax(x @ k.transpose(1, 2) / D ** 0.5, -1) @ v
                C.check_close(out[b, i].cpu().numpy(), ref.reshape(H * rep, D).cpu().numpy())
        P, Q = (torch.softmax(2 * rnd(B, N, V), -1) for _ in range(2))
        token = torch.randint(0, V, (B, N), generator=g, device="cuda").int()
        path = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        count, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        kvq.kvq_verify_draft(P, Q, token, parent, torch.rand((B, N), generator=g, device="cuda"), path, count, nxt)
        kvq.kvq_kivi_commit(cfg, cache, kd, vd, path, count)
        torch.cuda.synchronize()
        assert kvq.device_error() == 0
        assert cache.n_tok.tolist() == [n + c for n, c in zip(lens, count.tolist())]


def read_back(cfg, cache, n, b):
    k, v = (torch.zeros((1, cfg.n_heads, max(n, 1), D), device="cuda") for _ in range(2))
    if n:
        kvq.kvq_kivi_read(cfg, cache, k, v, b0=b)
    return k[0, :, :n], v[0, :, :n]
