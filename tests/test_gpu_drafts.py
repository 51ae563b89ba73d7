"""GPU parity of the speculative step over a KIVI cache: norm and rotation of rows, attention of
drafted tokens, commit of the accepted ones, reading the cache back; each against fp64 or, where the
result is a sequence of exact steps, bit for bit. The bounds count roundings (tests/_drafts.py and
beside each test)."""
import numpy as np
import pytest
import torch

import synth
from oracle import drafts as odr
from oracle import kivi as okivi
from sub_bit_quantized_gb300 import kvq
from tests import _cases as C
from tests import _drafts as T
from tests import _layout

pytestmark = pytest.mark.gpu
D = 128
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ARRAYS = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "k_resid", "v_resid", "n_tok", "n_quant_k",
          "n_quant_v", "sync")


# ------------------------------------------------------------------------------------ rows

def rope_table(max_ctx):
    ang = np.arange(max_ctx)[:, None] * 1.0e4 ** (-np.arange(D // 2) * 2.0 / D)
    return torch.from_numpy(np.cos(ang).astype(np.float32)).cuda(), torch.from_numpy(np.sin(ang).astype(np.float32)).cuda()


def check_rows(x, w, eps, cos, sin, pos, got):
    """got against fp64. y carries the error of the sum of 128 squares (a chain of 16 fp32 steps and
    three adds, halved by the root), rsqrtf (2 ulp), two products: under 2^-19 |y|; the rotation adds
    three roundings of |a c| + |b s| <= |a| + |b|. Then half a step of the output's type (2^-25
    absolute for fp16 subnormals)."""
    x64 = x.double().cpu().numpy()
    y = odr.norm_rows(x64, w.double().cpu().numpy(), eps) if w is not None else x64
    mag = np.abs(y)
    if cos is not None and w is not None:
        p = pos.cpu().long()
        c, s = (t.double().cpu().numpy()[p.numpy()][:, :, None] for t in (cos, sin))
        y = odr.rotate_rows(y, c, s)
        mag = np.concatenate([mag[..., :64] + mag[..., 64:]] * 2, axis=-1)
    err = np.abs(got.double().cpu().numpy() - y)
    bound = 2.0 ** -19 * mag + HALF_STEP[got.dtype] * (np.abs(y) + 2.0 ** -19 * mag) + 2.0 ** -25
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,N,Hq,H", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 7, 6, 3), (2, 65, 5, 1)])
def test_rows_fused_projection(dt, B, N, Hq, H):
    g = torch.Generator(device="cuda").manual_seed(B * 1000 + N)
    qkv = torch.randn((B, N, Hq + 2 * H, D), generator=g, device="cuda").to(dt)
    q, k, v = qkv.split([Hq, H, H], dim=2)
    wq, wk = (torch.randn(D, generator=g, device="cuda").to(dt) for _ in range(2))
    cos, sin = rope_table(300)
    pos = torch.randint(0, 300, (B, N), generator=g, device="cuda").int()
    qo = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    ko = torch.empty((B, H, N, D), dtype=torch.float16, device="cuda").transpose(1, 2)  # head-major, as a prefill reads
    vo = torch.empty((B, N, H, D), dtype=torch.float32, device="cuda")
    kvq.kvq_qk_norm_rope(q, k, v, wq, wk, 1e-6, cos, sin, pos, qo, ko, vo)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    check_rows(q, wq, 1e-6, cos, sin, pos, qo)
    check_rows(k, wk, 1e-6, cos, sin, pos, ko)
    assert torch.equal(vo, v.float())


@pytest.mark.parametrize("which", ["q", "k", "v", "qk"])
def test_rows_without_rotation_and_absent_kinds(which):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = {n: torch.randn((2, 5, 3, D), generator=g, device="cuda").bfloat16() for n in "qkv" if n in which}
    o = {n: torch.empty((2, 5, 3, D), dtype=torch.bfloat16, device="cuda") for n in x}
    w = torch.randn(D, generator=g, device="cuda").bfloat16()
    kvq.kvq_qk_norm_rope(x.get("q"), x.get("k"), x.get("v"), w, w, 1e-5, None, None, None, o.get("q"), o.get("k"), o.get("v"))
    for n in x:
        check_rows(x[n], None if n == "v" else w, 1e-5, None, None, None, o[n])


def test_rows_in_place_padding_and_far_positions():
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((2, 9, 4, D), generator=g, device="cuda").half()
    x0 = x.clone()
    w = torch.ones(D, device="cuda").half()
    cos, sin = rope_table(70000)
    pos = torch.randint(60000, 70000, (2, 9), generator=g, device="cuda").int()
    pos[0, 3] = -1                      # padding
    pos[1, 8] = 70000                   # past the table: left, reported
    kvq.kvq_qk_norm_rope(x, None, None, w, None, 1e-6, cos, sin, pos, x, None, None)
    torch.cuda.synchronize()
    assert kvq.device_error() == kvq.ERR_CAPACITY
    skip = torch.zeros((2, 9), dtype=torch.bool, device="cuda")
    skip[0, 3] = skip[1, 8] = True
    assert torch.equal(x[skip], x0[skip])
    check_rows(x0[~skip][None], w, 1e-6, cos, sin, pos[~skip][None], x[~skip][None])


@pytest.mark.parametrize("scale", [1e-25, 1e-4, 1e19, 3e37])
def test_rows_of_extreme_magnitude(scale):
    # squares that pass the fp32 range in both directions; zero rows; one infinite element
    g = torch.Generator(device="cuda").manual_seed(7)
    x = (torch.randn((1, 6, 2, D), generator=g, device="cuda") * scale).clamp(-3e38, 3e38).bfloat16()
    x[0, 0, 0] = 0
    w = torch.randn(D, generator=g, device="cuda").bfloat16()
    o = torch.empty_like(x, dtype=torch.float32)
    kvq.kvq_qk_norm_rope(x, None, None, w, None, 1e-6, None, None, None, o, None, None)
    check_rows(x, w, 1e-6, None, None, None, o)
    x[0, 1, 1, 9] = float("inf")
    kvq.kvq_qk_norm_rope(x, None, None, w, None, 1e-6, None, None, None, o, None, None)
    assert torch.isnan(o[0, 1, 1, 9]) and not o[0, 1, 1, :9].any()  # inf / inf, finite / inf
    check_rows(x[:, 2:], w, 1e-6, None, None, None, o[:, 2:])


@pytest.mark.parametrize("dt,N,Hq,H", [(torch.bfloat16, 30011, 5, 1), (torch.float32, 5003, 32, 8), (torch.float16, 9001, 20, 4)])
def test_rows_of_a_large_call_equal_those_of_small_ones(dt, N, Hq, H):
    g = torch.Generator(device="cuda").manual_seed(N)
    qkv = torch.randn((1, N, Hq + 2 * H, D), generator=g, device="cuda").to(dt)
    wq, wk = (torch.randn(D, generator=g, device="cuda").to(dt) for _ in range(2))
    cos, sin = rope_table(512)
    pos = torch.randint(-1, 512, (1, N), generator=g, device="cuda").int()

    def outs():
        return (torch.full((1, N, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((1, H, N, D), 7.0, dtype=torch.float16, device="cuda").transpose(1, 2),
                torch.full((1, N, H, D), 7.0, device="cuda"))
    whole, parts = outs(), outs()
    kvq.kvq_qk_norm_rope(*qkv.split([Hq, H, H], dim=2), wq, wk, 1e-6, cos, sin, pos, *whole)
    for t in range(0, N, 211):
        u = slice(t, min(t + 211, N))
        kvq.kvq_qk_norm_rope(*qkv[:, u].split([Hq, H, H], dim=2), wq, wk, 1e-6, cos, sin, pos[:, u].clone(),
                             *(x[:, u] for x in parts))
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    for x, y in zip(whole, parts):
        assert torch.equal(x, y)
    assert (whole[0][0, pos[0] < 0] == 7).all()
    mine = qkv.clone()  # in place
    q, k, v = mine.split([Hq, H, H], dim=2)
    kvq.kvq_qk_norm_rope(q, k, v, wq, wk, 1e-6, cos, sin, pos, q, k, v)
    live = pos[0] >= 0
    if dt == torch.float32:  # rounded afterwards instead
        assert torch.equal(mine[0, :, :Hq][live].bfloat16(), whole[0][0][live])
        assert torch.equal(mine[0, :, Hq:Hq + H][live].half(), whole[1][0][live])
    assert torch.equal(mine[0, :, Hq + H:], qkv[0, :, Hq + H:]) and torch.equal(mine[0][~live], qkv[0][~live])


# ------------------------------------------------------------------------------------ read

def read_bound(ref, dtype):
    # s (q - z): two fp32 roundings, then half a step of the output (2^-25 absolute: fp16 subnormals)
    return np.abs(ref) * (2.0 ** -23 + HALF_STEP[dtype] * (1 + 2.0 ** -23)) + 2.0 ** -25


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kb,vb,R", [(2, 2, 128), (4, 2, 32), (2, 4, 64), (4, 4, 0)])
def test_read_rows(dtype, kb, vb, R):
    nq, nr = [96, 0, 320, 32], [min(R, x) for x in (5, 20, 32, 0)]
    nqv = None if R == 0 else [94, 0, 320, 32]
    case = C.make_kivi_case(900 + kb, B=4, H=3, n_quant=nq, n_resid=nr, residual=R, k_bits=kb, v_bits=vb, n_quant_v=nqv)
    cache = C.fill_kivi_cache(case)
    n, begin = 77, [40, -3, 290, 1000]
    out = [torch.full((4, 3, n, D), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    kvq.kvq_kivi_read(case.cfg, cache, out[0], out[1], tok_begin=torch.tensor(begin, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for b in range(4):
        for h in range(3):
            for x, ref in zip(out, T.context(case, b, h)[:2]):
                got = x[b, h].double().cpu().numpy()
                for j in range(n):
                    t = begin[b] + j
                    if 0 <= t < case.n_tok[b]:
                        assert (np.abs(got[j] - ref[t]) <= read_bound(ref[t], dtype)).all()
                    else:
                        assert (got[j] == 9.0).all()  # left as it was


def test_read_one_side_strided_and_from_b0():
    case = C.make_kivi_case(910, B=3, H=2, n_quant=[64, 128, 96], n_resid=[3, 100, 128])
    cache = C.fill_kivi_cache(case)
    big = torch.full((2, 5, 2, 40, D), 3.0, dtype=torch.float32, device="cuda")
    out = big[:, 1]  # strides of a larger array
    kvq.kvq_kivi_read(case.cfg, cache, None, out, b0=1)
    torch.cuda.synchronize()
    for i in range(2):
        for h in range(2):
            ref = T.context(case, 1 + i, h)[1][:40]
            assert (np.abs(out[i, h].double().cpu().numpy() - ref) <= read_bound(ref, torch.float32)).all()
    assert (big[:, 0] == 3).all() and (big[:, 2:] == 3).all()


# ------------------------------------------------------------------------------------ commit

def stream_cache(seed, lens, H, kb, vb, R, extra):
    """A cache after a prefill and `extra` appends, and the drafts' generator."""
    g = synth.rng(seed)
    B = len(lens)
    cfg = kvq.KiviConfig(n_heads=H, k_bits=kb, v_bits=vb, residual=R, max_batch=B, max_tokens=4 * R + max(lens) // 32 * 32)
    cache = kvq.KiviCache(cfg)
    for b, n in enumerate(lens):
        if n:
            k, v = (C.fp16_tensor(synth.gaussian(g, (1, H, n, D))) for _ in range(2))
            kvq.kvq_kivi_prefill(cfg, cache, k, v, b0=b)
    for _ in range(extra):
        kvq.kvq_kivi_append(cfg, cache, C.fp16_tensor(synth.gaussian(g, (B, H, D))), C.fp16_tensor(synth.gaussian(g, (B, H, D))))
    return g, cfg, cache


def copy_cache(cfg, cache):
    other = kvq.KiviCache(cfg)
    for name in ARRAYS:
        getattr(other, name).copy_(getattr(cache, name))
    return other


def check_commit(seed, R, N, extra, kb, vb, H=2):
    lens = [0, 1, R - 1, R, R + 1, 3 * R + 7]
    B = len(lens)
    g, cfg, cache = stream_cache(seed, lens, H, kb, vb, R, extra)
    seq = copy_cache(cfg, cache)
    kd, vd = (C.fp16_tensor(synth.gaussian(g, (B, N, H, D))) for _ in range(2))
    path = torch.from_numpy(g.integers(0, N, size=(B, N)).astype(np.int32)).cuda()  # some index twice
    take = [N, 0, max(1, N // 2), N, 1, N]
    kvq.kvq_kivi_commit(cfg, cache, kd, vd, path, torch.tensor(take, dtype=torch.int32).cuda())
    # the same tokens one at a time, each request by itself
    one = kvq.KiviConfig(n_heads=H, k_bits=kb, v_bits=vb, residual=R, max_batch=1, max_tokens=cfg.max_tokens)
    for b in range(B):
        part = kvq.KiviCache(one)
        for name in ARRAYS:
            getattr(part, name).copy_(getattr(seq, name)[b:b + 1])
        for i in range(take[b]):
            j = int(path[b, i])
            kvq.kvq_kivi_append(one, part, kd[b, j][None].contiguous(), vd[b, j][None].contiguous())
        for name in ARRAYS:
            assert torch.equal(getattr(cache, name)[b:b + 1], getattr(part, name)), (b, name)
    assert kvq.device_error() == 0


@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("R,N,extra", [(32, 32, 0), (32, 5, 31), (128, 64, 100), (64, 1, 0), (96, 17, 90)])
def test_commit_equals_appends(kb, vb, R, N, extra):
    check_commit(1200 + R + N, R, N, extra, kb, vb)


def test_commit_against_the_stream_oracle():
    R, H, N = 32, 1, 8
    g = synth.rng(77)
    K, V = (np.asarray(synth.gaussian(g, (1, H, 50, D)), np.float16) for _ in range(2))
    cfg = kvq.KiviConfig(n_heads=H, residual=R, max_batch=1, max_tokens=256)
    cache = kvq.KiviCache(cfg)
    kvq.kvq_kivi_prefill(cfg, cache, torch.from_numpy(K).cuda(), torch.from_numpy(V).cuda())
    s = okivi.KiviStream(residual=R)
    s.prefill(K[0, 0], V[0, 0])
    for step in range(9):
        kd, vd = (np.asarray(synth.gaussian(g, (1, N, H, D)), np.float16) for _ in range(2))
        m = 1 + (step * 5) % N
        path = g.permutation(N)[None].astype(np.int32)
        kvq.kvq_kivi_commit(cfg, cache, C.fp16_tensor(kd), C.fp16_tensor(vd), torch.from_numpy(path).cuda(),
                            torch.tensor([m], dtype=torch.int32).cuda())
        for i in range(m):
            s.append(kd[0, path[0, i], 0], vd[0, path[0, i], 0])
    assert [int(x) for x in (cache.n_tok, cache.n_quant_k, cache.n_quant_v)] == [s.n_tok, s.n_quant_k, len(s.v_codes)]
    assert np.array_equal(_layout.unpack_codes(cache.k_codes.cpu().numpy())[0, 0, :s.n_quant_k], s.k_codes)
    assert np.array_equal(_layout.unpack_codes(cache.v_codes.cpu().numpy())[0, 0, :len(s.v_codes)], s.v_codes)
    assert np.array_equal(cache.v_scale.cpu().numpy()[0, 0, :len(s.v_codes)], s.v_scale)
    assert np.array_equal(cache.k_resid.cpu().numpy()[0, 0, :len(s.k_resid)], s.k_resid)


@pytest.mark.parametrize("why", ["index", "negative", "count", "minus", "residual", "room", "state"])
def test_commit_leaves_what_it_cannot_commit(why):
    R, H, N, B = 32, 2, 40, 2
    g, cfg, cache = stream_cache(1300, [R + 5, R + 9], H, 2, 2, R, 3)
    kd, vd = (C.fp16_tensor(synth.gaussian(g, (B, N, H, D))) for _ in range(2))
    path = torch.arange(N, dtype=torch.int32).repeat(B, 1)
    take = torch.tensor([4, 4], dtype=torch.int32)
    want = kvq.ERR_INVALID_ARG
    if why == "index":
        path[1, 3] = N
    elif why == "negative":
        path[1, 0] = -1
    elif why == "count":
        take[1] = N + 1
    elif why == "minus":
        take[1] = -2
    elif why == "residual":
        take[1], want = R + 1, kvq.ERR_CAPACITY
    elif why == "room":  # the key residual would flush past max_tokens
        cache.n_quant_k[1] = cache.n_quant_v[1] = cfg.max_tokens
        cache.n_tok[1] = cfg.max_tokens + R
        want = kvq.ERR_CAPACITY
    else:
        cache.n_quant_v[1], want = cache.n_quant_k[1] + 1, kvq.ERR_CAPACITY
    before = copy_cache(cfg, cache)
    kvq.kvq_kivi_commit(cfg, cache, kd, vd, path.cuda(), take.cuda())
    torch.cuda.synchronize()
    assert kvq.device_error() == want
    for name in ARRAYS:
        assert torch.equal(getattr(cache, name)[1], getattr(before, name)[1]), name
    assert int(cache.n_tok[0]) == int(before.n_tok[0]) + 4  # the other request is committed
    assert not cache.sync.any()


# ------------------------------------------------------------------------------------ tree

@pytest.mark.parametrize("kb,vb", [(2, 2), (4, 4), (2, 4), (4, 2)])
@pytest.mark.parametrize("rep,N", [(1, 1), (1, 8), (4, 5), (3, 16), (2, 64), (7, 33)])
def test_tree_ragged_batch(kb, vb, rep, N):
    nq, nr = [0, 32, 96, 640], [1, 95, 33, 128]
    nqv = [0, 20, 90, 640]
    case = T.make_tree_case(2000 + rep * 100 + N, B=4, H=2, N=N, n_quant=nq, n_resid=nr, rep=rep,
                            n_draft=[N, max(1, N - 3), N, max(1, N // 2)], k_bits=kb, v_bits=vb, n_quant_v=nqv, q_scale=0.5)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("n", [0, 1, 31, 126, 127, 128, 129, 255, 256])
def test_tree_lengths_around_tiles(n):
    # cached and drafted tokens meeting at, before and after a tile's edge; nothing cached at all
    N = 6
    nq = max(0, n - 40) // 32 * 32
    case = T.make_tree_case(2100 + n, B=2, H=1, N=N, n_quant=[nq, 64], n_resid=[n - nq, 128], n_draft=[N, 2], rep=2)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


def test_tree_long_context_is_split():
    case = T.make_tree_case(2200, B=2, H=2, N=4, n_quant=[32 * 300, 64], n_resid=[77, 12], k_bits=4, q_scale=0.3)
    ref, bound = T.reference(case)
    got = T.run_tree(case)
    T.check_rows(got, ref, bound, 7.0)
    assert np.array_equal(got, T.run_tree(case))  # joined in a fixed order


@pytest.mark.parametrize("n_draft", [[0, 0, 0], [0, 5, 0], [-4, 99, 1]])
def test_tree_draft_counts(n_draft):
    case = T.make_tree_case(2300, B=3, H=2, N=5, n_quant=[64, 32, 0], n_resid=[9, 0, 50], n_draft=n_draft)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


def test_tree_masks():
    # a full mask, an empty one, only a later token, bits of padding tokens, bit 63
    N = 64
    case = T.make_tree_case(2400, B=3, H=1, N=N, n_quant=[0, 96, 0], n_resid=[0, 40, 10], n_draft=[N, N, 20])
    m = case.mask
    for b in range(3):
        m[b, 0], m[b, 1], m[b, 2] = np.uint64(2 ** 64 - 1), np.uint64(0), np.uint64(1 << 63)
        m[b, 3], m[b, 4] = np.uint64(1 << 19), np.uint64((1 << 63) | (1 << 20))
    ref, bound = T.reference(case)
    got = T.run_tree(case)
    T.check_rows(got, ref, bound, 7.0)
    assert not got[0, 1].any()  # attends nothing: 0


@pytest.mark.parametrize("rep", [1, 6, 16])
def test_tree_many_requests(rep):
    # more requests than a warp has lanes, some with nothing cached, nothing drafted or neither
    B, N = 70, 2
    nq, nr = [32 * (b % 5) for b in range(B)], [(b * 7) % 100 if b % 3 else 0 for b in range(B)]
    nd = [0 if b % 11 == 4 or 30 <= b < 40 else 1 + b % 2 for b in range(B)]
    case = T.make_tree_case(2460, B=B, H=1, N=N, n_quant=nq, n_resid=nr, n_draft=nd, rep=rep, residual=128)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("max_tokens", [32, 96, 160])
@pytest.mark.parametrize("rep,kb,vb", [(1, 2, 4), (2, 4, 2), (6, 2, 2), (20, 4, 4)])
def test_tree_caches_filled_to_the_end(max_tokens, rep, kb, vb):
    # quantized tokens up to the last place of the arrays, values up to it and short of it
    case = T.make_tree_case(2465, B=3, H=2, N=5, n_quant=[max_tokens] * 3, n_resid=[0, 32, 9], rep=rep, k_bits=kb, v_bits=vb,
                            residual=32, max_tokens=max_tokens, n_quant_v=[max_tokens, max_tokens, max_tokens - 23], q_scale=0.5)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("rep,kb", [(1, 2), (1, 4), (2, 2), (6, 4)])
@pytest.mark.parametrize("down", [5, 9, 12, 14])
def test_tree_small_keys_and_large_queries(rep, kb, down):
    # keys times 2^-down, queries times 2^down: the same scores
    case = T.make_tree_case(2469, B=2, H=2, N=6, n_quant=[256, 32], n_resid=[40, 3], rep=rep, k_bits=kb, q_scale=0.5)
    f = np.float16(2.0 ** -down)
    case.base.k_scale[:] *= f
    case.base.k_res[:] *= f
    case.kd *= f
    case.q *= 2.0 ** down
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


def test_tree_many_query_heads():
    case = T.make_tree_case(2467, B=1, H=1, N=64, n_quant=[64], n_resid=[21], rep=33, n_draft=[61], q_scale=0.5)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("rep", [1, 2, 4, 9])
def test_tree_maxima_that_move_late(rep):
    # drafted keys of large scores (exact in fp16): the maxima of a long context's parts move in the last tile only
    case = T.make_tree_case(2470, B=2, H=2, N=8, n_quant=[32 * 70, 128], n_resid=[100, 40], rep=rep, k_bits=4, q_scale=0.3)
    case.kd *= np.float16(8)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("rep", [1, 2, 4, 9])
def test_tree_scores_that_are_not_numbers(rep):
    # a drafted key and a query row of NaN in a context that several blocks share
    N = 8
    case = T.make_tree_case(2480, B=1, H=2, N=N, n_quant=[32 * 90], n_resid=[61], rep=rep, q_scale=0.3)
    fine = T.TreeCase(case.base, case.q.copy(), case.kd.copy(), case.vd, case.mask, case.n_draft)
    case.kd[0, 3, 1], case.q[0, 5, 0] = np.nan, np.nan
    bad = np.zeros(case.q.shape[:3], bool)
    bad[0, :, rep:] = np.array([int(x) >> 3 & 1 for x in case.mask[0]], bool)[:, None]
    bad[0, 5, 0] = True
    ref, bound = T.reference(fine)
    got = T.run_tree(case)
    assert np.isnan(got[bad]).all()
    T.check_rows(got[~bad], ref[~bad], bound[~bad], 7.0)


@pytest.mark.parametrize("rep", [1, 5])
def test_tree_calls_at_once_and_workspaces_as_they_come(rep):
    cases = [T.make_tree_case(2490 + i, B=3, H=4, N=7, n_quant=[32 * 80, 96 * i, 640], n_resid=[50, 9, 128], rep=rep, q_scale=0.5)
             for i in range(2)]
    caches = [C.fill_kivi_cache(c.base) for c in cases]
    args = [T.tensors(c) for c in cases]
    want, wss, outs = [], [], []
    for c, cache, (q, kd, vd, mask, nd) in zip(cases, caches, args):
        ref, bound = T.reference(c)
        got = T.run_tree(c, cache)
        T.check_rows(got, ref, bound, 7.0)
        want.append(got)
        ws = kvq.make_tree_workspace(c.base.cfg, 3, 7)
        ws.fill_(255)  # needs no initialisation
        wss.append(ws)
        outs.append(torch.empty(q.shape, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for c, cache, (q, kd, vd, mask, nd), ws, out, st in zip(cases, caches, args, wss, outs, streams):
            with torch.cuda.stream(st):
                kvq.kvq_kivi_tree_attn(c.base.cfg, cache, q, kd, vd, mask, out, n_draft=nd, ws=ws)
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    for out, w in zip(outs, want):
        assert np.array_equal(out.double().cpu().numpy(), w)


def test_tree_no_residual():
    case = T.make_tree_case(2450, B=2, H=2, N=3, n_quant=[64, 160], n_resid=[0, 0], residual=0, rep=2)
    ref, bound = T.reference(case)
    T.check_rows(T.run_tree(case), ref, bound, 7.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_tree_values_not_attended_cannot_change_a_row(bad):
    N = 12
    case = T.make_tree_case(2500, B=2, H=2, N=N, n_quant=[96, 0], n_resid=[26, 0], n_draft=[N - 2, N], rep=2)
    cache = C.fill_kivi_cache(case.base)
    # what lies behind the lengths: codes' constants, residual rows, padding drafts
    for b, (nqk, nqv, n) in enumerate(zip(case.base.n_quant_k, case.base.n_quant_v, case.base.n_tok)):
        cache.k_scale[b, :, nqk // 32:] = bad
        cache.v_zero[b, :, nqv:] = bad
        cache.k_resid[b, :, n - nqk:] = bad
        for t in range(n, nqv + 128):
            cache.v_resid[b, :, t % 128] = bad
    case.kd[0, N - 2:], case.vd[0, N - 1] = bad, bad
    sees5 = np.array([[bool(int(x) >> 5 & 1) for x in case.mask[b]] for b in range(2)])
    fine = T.TreeCase(case.base, case.q, np.nan_to_num(case.kd, posinf=0, neginf=0),
                      np.nan_to_num(case.vd, posinf=0, neginf=0), case.mask, case.n_draft)
    case.kd[1, 5], case.vd[0, 5] = bad, bad  # a drafted token that some rows see
    ref, bound = T.reference(fine)
    got = T.run_tree(case, cache)
    for b in range(2):
        T.check_rows(got[b][~sees5[b]], ref[b][~sees5[b]], bound[b][~sees5[b]], 7.0)
    assert not np.isfinite(got[0][sees5[0] & (np.arange(N) < N - 2)]).any()  # a value: every channel of the rows that see it
    if np.isnan(bad):
        assert np.isnan(got[1][sees5[1]]).all()


def test_tree_bf16_output_is_the_rounded_fp32_one():
    case = T.make_tree_case(2600, B=2, H=2, N=9, n_quant=[320, 64], n_resid=[50, 3], rep=4)
    a, b = T.run_tree(case), T.run_tree(case, dtype=torch.bfloat16)
    assert np.array_equal(torch.from_numpy(a).float().bfloat16().double().numpy(), b)


@pytest.mark.parametrize("scale", [0.0, 1e-30, 3e4, 1e30])
def test_tree_query_magnitudes(scale):
    # queries past the fp16 range either way: their power of two leaves the fp16 operand in range
    case = T.make_tree_case(2700, B=1, H=1, N=4, n_quant=[64], n_resid=[30], rep=2)
    case.q[:] = synth.bf16_round(case.q * scale)
    got = T.run_tree(case)
    if scale <= 1.0:
        ref, bound = T.reference(case)
        T.check_rows(got, ref, bound, 7.0)
    else:
        assert np.isfinite(got).all()  # one token takes all the weight: the rounding of its score decides which


def test_offsets_past_32_bits():
    # the last head's codes lie more than 2^32 bytes into the arrays
    N, H, T0 = 3, 4, 1 << 25
    cfg = kvq.KiviConfig(n_heads=H, k_bits=4, v_bits=2, residual=32, max_batch=1, max_tokens=T0)
    small = T.make_tree_case(2800, B=1, H=H, N=N, n_quant=[64], n_resid=[7], k_bits=4, residual=32)
    case = C.fill_kivi_cache(small.base)
    cache = kvq.KiviCache(kvq.KiviConfig(n_heads=H, residual=32, max_batch=1))
    for name in ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero"):
        x = getattr(case, name)
        y = torch.empty((1, H, T0 // (32 if name in ("k_scale", "k_zero") else 1), x.shape[3]), dtype=x.dtype, device="cuda")
        y[:, :, :x.shape[2]] = x
        setattr(cache, name, y)
    for name in ("k_resid", "v_resid", "n_tok", "n_quant_k", "n_quant_v", "sync"):
        setattr(cache, name, getattr(case, name))
    q, kd, vd, mask, nd = T.tensors(small)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    kvq.kvq_kivi_tree_attn(cfg, cache, q, kd, vd, mask, out, n_draft=nd)
    ref, bound = T.reference(small)
    T.check_rows(out.double().cpu().numpy(), ref, bound, 7.0)
    k = torch.empty((1, H, 71, D), dtype=torch.float32, device="cuda")
    v = torch.empty_like(k)
    kvq.kvq_kivi_read(cfg, cache, k, v)
    for h in range(H):
        for x, r in zip((k, v), T.context(small.base, 0, h)[:2]):
            assert (np.abs(x[0, h].double().cpu().numpy() - r) <= read_bound(r, torch.float32)).all()


# ------------------------------------------------------------------------------------ together

def test_a_speculative_step_equals_decoding():
    """Rows, tree, commit and read back as a serving step uses them, on a side stream, captured and
    replayed twice: a chain of drafts attends what the same tokens attend when they are appended and
    decoded one at a time, and the committed rows read back as they were."""
    B, N, Hq, H, R = 3, 4, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    cfg = kvq.KiviConfig(n_heads=H, n_q_heads=Hq, residual=R, max_batch=B, max_tokens=512)
    cache = kvq.KiviCache(cfg)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    kvq.kvq_kivi_prefill(cfg, cache, rnd(B, H, 150, D).half(), rnd(B, H, 150, D).half())
    cos, sin = rope_table(1024)
    wq, wk = (1 + 0.1 * rnd(D)).bfloat16(), (1 + 0.1 * rnd(D)).bfloat16()
    qkv = rnd(B, N, Hq + 2 * H, D).bfloat16()
    q, k, v = qkv.split([Hq, H, H], dim=2)
    pos = (150 + torch.arange(N, device="cuda")).int().repeat(B, 1)
    qo = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    ko = torch.empty((B, N, H, D), dtype=torch.float16, device="cuda")
    vo, out = torch.empty_like(ko), torch.empty((B, N, Hq, D), dtype=torch.float32, device="cuda")
    mask = torch.tensor([[(2 << i) - 1 for i in range(N)]] * B, dtype=torch.int64, device="cuda")  # chains
    take = torch.tensor([N, 2, 0], dtype=torch.int32, device="cuda")
    path = torch.arange(N, dtype=torch.int32, device="cuda").repeat(B, 1)
    back = torch.zeros((2, B, H, 16, D), dtype=torch.float16, device="cuda")
    begin = torch.full((B,), 142, dtype=torch.int32, device="cuda")
    ws = kvq.make_tree_workspace(cfg, B, N)
    start = copy_cache(cfg, cache)

    def step(target):
        kvq.kvq_qk_norm_rope(q, k, v, wq, wk, 1e-6, cos, sin, pos, qo, ko, vo)
        kvq.kvq_kivi_tree_attn(cfg, target, qo, ko, vo, mask, out, ws=ws)
        kvq.kvq_kivi_commit(cfg, target, ko, vo, path, take)
        kvq.kvq_kivi_read(cfg, target, back[0], back[1], tok_begin=begin)

    other = copy_cache(cfg, cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(other)  # warm up
        side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache)
    torch.cuda.synchronize()
    for name in ARRAYS:  # captured, not run
        assert torch.equal(getattr(cache, name), getattr(start, name))
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert kvq.device_error() == 0
    first = out.clone()
    # token by token: append, then decode (150 + 4 tokens: no value leaves the window, no key is flushed)
    seq = copy_cache(cfg, start)
    dec = torch.empty((B, Hq, D), dtype=torch.float32, device="cuda")
    for i in range(N):
        kvq.kvq_kivi_append(cfg, seq, ko[:, i].contiguous(), vo[:, i].contiguous())
        kvq.kvq_decode_attn(cfg, seq, 0, 1, qo[:, i].contiguous(), dec)
        # 2e-3 is the decode's own distance from fp64, and the tree's stays as near on such inputs
        assert (dec - first[:, i]).abs().max().item() <= 4e-3
    assert torch.equal(seq.n_quant_v, start.n_quant_v) and torch.equal(seq.n_quant_k, start.n_quant_k)
    assert cache.n_tok.tolist() == [154, 152, 150]
    # the window read back: committed drafts in fp16, exactly
    assert torch.equal(back[0, 0, :, 8:12], ko[0].transpose(0, 1)) and torch.equal(back[1, 1, :, 8:10], vo[1, :2].transpose(0, 1))
    # a second replay commits the same drafts behind the first ones
    graph.replay()
    torch.cuda.synchronize()
    assert cache.n_tok.tolist() == [158, 154, 150] and kvq.device_error() == 0


def test_a_call_refuses_to_run_on_another_device(monkeypatch):
    x = torch.zeros((1, 2, 4, D), device="cuda").half()
    call = kvq.QkNormRopeCall(x, None, None, torch.ones(D, device="cuda").half(), None, 1e-6, None, None, None, x, None, None)
    call()
    other = torch.cuda.current_device() + 1  # as if it were the current one
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: other)
    with pytest.raises(ValueError, match="device"):
        call()
