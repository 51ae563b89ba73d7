"""Cases that measure the operators of a speculative serving step over a KIVI cache.

A step projects the tokens of every request's draft tree, normalises and rotates their queries
and keys (``rows``), attends them to the cached context and to their ancestors in the tree
(``tree``), commits the accepted path into the quantized cache and reads its window back
(``commit``); reading a cache back is also what moves a context out of it (``read``).

``run`` computes a pass in elementary torch operations, or with ``own`` set through the library.
"""
import math

import torch

own = False

D = 128
GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of one request: plain decoding, latency alone counts
        dict(name="rows_one_token", op="rows", B=1, N=1, Hq=32, H=8, x="bf16", rope=True, fused=True, head_major=False),
        # the drafted tokens of a batch, multi-head, read out of the fused projection
        dict(name="rows_drafts", op="rows", B=16, N=17, Hq=32, H=32, x="bf16", rope=True, fused=True, head_major=False),
        # a long prompt, written head-major as the cache's prefill takes it
        dict(name="rows_prompt", op="rows", B=1, N=16381, Hq=32, H=8, x="bf16", rope=True, fused=True, head_major=True),
        # a short chat with a small tree: latency
        dict(name="tree_short", op="tree", B=1, H=8, rep=4, N=5, ctx=701, kb=2, vb=2, R=128),
        # the multi-head batch of the attention benchmark, a chain of drafts
        dict(name="tree_mha_2bit", op="tree", B=16, H=32, rep=1, N=8, ctx=4096, kb=2, vb=2, R=128),
        # the grouped-query batch of the attention benchmark, a wide tree
        dict(name="tree_gqa_4bit", op="tree", B=16, H=8, rep=4, N=48, ctx=4096, kb=4, vb=4, R=128),
        # two long contexts: few requests, the context split over the whole GPU
        dict(name="tree_long", op="tree", B=2, H=8, rep=4, N=16, ctx=32768, kb=4, vb=2, R=128),
        # the accepted path of one request
        dict(name="commit_one", op="commit", B=1, H=8, N=5, kb=2, vb=2, R=128, window=160),
        # the accepted paths of a batch, some of which fill the key residual
        dict(name="commit_batch", op="commit", B=64, H=32, N=8, kb=4, vb=4, R=128, window=160),
        # the newest tokens of a few requests
        dict(name="read_window", op="read", B=4, H=8, ctx=1531, n=96, kb=2, vb=2, R=128, out="bf16"),
        # a whole multi-head cache into fp16, for another engine
        dict(name="read_mha_2bit", op="read", B=16, H=32, ctx=4096, n=4096, kb=2, vb=2, R=128, out="fp16"),
        # a grouped-query cache of odd length into fp32
        dict(name="read_gqa_4bit", op="read", B=3, H=8, ctx=20011, n=20011, kb=4, vb=4, R=64, out="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rows", "tree", "commit", "read"])
    bits = dict(kb=rng.choice([2, 4]), vb=rng.choice([2, 4]), R=rng.choice([32, 64, 128]))
    if op == "rows":
        H = rng.choice([1, 2, 4, 8, 16, 32])
        Hq = H * rng.choice([1, 2, 3, 4]) if H < 16 else H
        most = 16381 * 48 // (Hq + 2 * H)  # tokens in all
        N = _log(rng, 1, min(8000, most))
        return dict(op=op, B=_log(rng, 1, max(1, min(64, most // N))), N=N, Hq=Hq, H=H, x=rng.choice(["bf16", "fp16"]),
                    rope=rng.random() < 0.8, fused=rng.random() < 0.7, head_major=rng.random() < 0.4)
    if op == "tree":
        H = rng.choice([1, 2, 4, 8, 16, 32])
        rep = rng.choice([1, 2, 3, 4, 7, 8]) if H < 16 else 1
        N, room = _log(rng, 1, 64), 16 * 8 * 4096 * 192  # query rows times tokens of the largest case
        ctx = _log(rng, 1, min(32768, room // (H * N * rep)))
        most = min(16 * 32 * 4096 // (H * ctx), room // (H * ctx * N * rep), 32)
        return dict(op=op, B=_log(rng, 1, max(1, most)), H=H, rep=rep, N=N, ctx=ctx, **bits)
    if op == "commit":
        return dict(op=op, B=_log(rng, 1, 64), H=rng.choice([1, 2, 8, 32]), N=rng.randint(1, 16),
                    window=rng.randint(1, 160), **bits)
    H, ctx = rng.choice([1, 2, 4, 8, 16, 32]), _log(rng, 1, 20000)
    return dict(op=op, B=_log(rng, 1, max(1, min(16, 16 * 32 * 2000 // (H * ctx)))), H=H, ctx=ctx, n=_log(rng, 1, ctx),
                out=rng.choice(["fp16", "bf16", "fp32"]), **bits)


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda")


def _rope_table(max_ctx):
    freq = 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) * 2 / D)
    ang = torch.arange(max_ctx, device="cuda", dtype=torch.float64)[:, None] * freq
    return ang.cos().float(), ang.sin().float()


def _keys(g, *shape):
    """Keys with six large channels for each head (dimension 1), as the cache's quantizer expects them."""
    x = _randn(g, *shape)
    big = torch.rand((shape[1], D), generator=g, device="cuda").argsort(-1)[:, :6]
    gain = torch.ones((shape[1], D), device="cuda").scatter_(1, big, 20.0)
    return (x * gain[None, :, None]).half()


def _pack(q, bits):
    q = q.to(torch.uint8).unflatten(-1, (D * bits // 8, 8 // bits))
    shift = torch.arange(8 // bits, device=q.device, dtype=torch.uint8) * bits
    return (q << shift).sum(-1).to(torch.uint8)


def _quantize(x, dim, bits):
    """Codes, fp16 scale and fp16 zero-point of groups along ``dim``; every step one fp32 rounding."""
    x = x.float()
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = ((hi - lo) / float(2 ** bits - 1)).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = (-lo / s.float()).half()
    q = (x / s.float() + z.float()).round().clamp(0, 2 ** bits - 1)
    return q, s.squeeze(dim), z.squeeze(dim)


def _quantize_keys(k, bits):
    q, s, z = _quantize(k.unflatten(2, (-1, GROUP)), 3, bits)
    return _pack(q.flatten(2, 3), bits), s, z


def _quantize_values(v, bits):
    q, s, z = _quantize(v.unflatten(-1, (-1, GROUP)), -1, bits)
    return _pack(q.flatten(-2, -1), bits), s, z


def _cache(g, case, n_tok, room):
    """A KIVI cache of n_tok[b] tokens as a prefill and some decode steps leave it: keys of a
    multiple of the group quantized, values a little behind or level with them."""
    B, H, R = case["B"], case["H"], case["R"]
    n_tok = torch.tensor(n_tok)
    nqk = (n_tok - R).clamp(min=0).add(GROUP - 1) // GROUP * GROUP
    behind = torch.randint(0, GROUP, (B,), generator=torch.Generator().manual_seed(int(_randint(g, 0, 1 << 30, 1))))
    nqv = torch.minimum((nqk - behind).clamp(min=0), nqk).maximum(n_tok - R).clamp(min=0)
    T = (max(int(nqk.max()), GROUP) + room + GROUP - 1) // GROUP * GROUP
    lens = torch.zeros((3, (B + 3) // 4 * 4), dtype=torch.int32)
    lens[0, :B], lens[1, :B], lens[2, :B] = n_tok, nqk, nqv
    st = dict(H=H, R=R, T=T, kb=case["kb"], vb=case["vb"], lens=lens.cuda())
    st["k_codes"], st["k_scale"], st["k_zero"] = _quantize_keys(_keys(g, B, H, T, D), case["kb"])
    st["v_codes"], st["v_scale"], st["v_zero"] = _quantize_values(_randn(g, B, H, T, D).half(), case["vb"])
    st["k_resid"], st["v_resid"] = _keys(g, B, H, R, D), _randn(g, B, H, R, D).half()
    return st


def _handle(st, B, Hq):
    """The library's cache object over the buffers of ``st``."""
    from sub_bit_quantized_gb300 import kvq

    cfg = kvq.KiviConfig(n_heads=st["H"], n_q_heads=Hq, k_bits=st["kb"], v_bits=st["vb"], residual=st["R"],
                         max_batch=B, max_tokens=st["T"])
    cache = kvq.KiviCache(kvq.KiviConfig(n_heads=st["H"], k_bits=st["kb"], v_bits=st["vb"], residual=GROUP, max_batch=B))
    cache.cfg = cfg
    for name in ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "k_resid", "v_resid"):
        setattr(cache, name, st[name])
    cache.n_tok, cache.n_quant_k, cache.n_quant_v = st["lens"][0, :B], st["lens"][1, :B], st["lens"][2, :B]
    return cfg, cache


def _lengths(g, B, ctx):
    """Ragged context lengths, the longest of them ctx."""
    n = (ctx * (0.75 + 0.25 * torch.rand((B,), generator=g, device="cuda"))).ceil().int().clamp(1, ctx).tolist()
    n[0] = ctx
    return n


def _prepare_rows(case, g):
    B, N, Hq, H, x = case["B"], case["N"], case["Hq"], case["H"], DTYPES[case["x"]]
    st = dict(op="rows", eps=1e-6, cos=None, sin=None, pos=None)
    if case["fused"]:  # views of the projection's output [B][N][(Hq + 2 H) D]
        qkv = _randn(g, B, N, Hq + 2 * H, D).to(x)
        st["q"], st["k"], st["v"] = qkv.split([Hq, H, H], dim=2)
    else:
        st["q"], st["k"], st["v"] = (_randn(g, B, N, h, D).to(x) for h in (Hq, H, H))
    st["wq"], st["wk"] = ((1 + 0.2 * _randn(g, D)).to(x) for _ in range(2))
    if case["rope"]:
        first = _randint(g, 0, 16384, B, 1)
        st["pos"] = (first + torch.arange(N, device="cuda")).int()
        st["cos"], st["sin"] = _rope_table(32768)

    def out(h, t):
        if case["head_major"]:
            return torch.zeros((B, h, N, D), dtype=t, device="cuda").transpose(1, 2)
        return torch.zeros((B, N, h, D), dtype=t, device="cuda")

    # with rotation the keys go on to the KIVI cache (fp16), without it to one that holds them unrotated (bf16)
    kt = torch.float16 if case["rope"] else torch.bfloat16
    st["qo"], st["ko"], st["vo"] = out(Hq, torch.bfloat16), out(H, kt), out(H, kt)
    if own:
        from sub_bit_quantized_gb300 import kvq

        st["call"] = kvq.QkNormRopeCall(st["q"], st["k"], st["v"], st["wq"], st["wk"], st["eps"], st["cos"], st["sin"],
                                        st["pos"], st["qo"], st["ko"], st["vo"])
    return st


def _trees(seed, B, N):
    """Parents drawn at random (a few roots), as a bit for each visible drafted token; n_draft[b] of the N are real."""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand((B, N), generator=g).tolist()
    count = torch.randint(max(1, N - N // 4), N + 1, (B,), generator=g).tolist()
    masks = []
    for b in range(B):
        row = []
        for i in range(N):
            parent = int(u[b][i] * (i + 1)) - 1 if i else -1
            row.append((row[parent] if parent >= 0 else 0) | (1 << i))
        masks.append([m - (1 << 64) if m >> 63 else m for m in row])
    return torch.tensor(masks, dtype=torch.int64).cuda(), torch.tensor(count, dtype=torch.int32).cuda()


def _prepare_tree(case, g, seed):
    B, N, H, rep = case["B"], case["N"], case["H"], case["rep"]
    st = _cache(g, case, _lengths(g, B, case["ctx"]), 0)
    st.update(op="tree", rep=rep)
    st["q"] = _randn(g, B, N, H * rep, D).bfloat16()
    st["kd"] = _keys(g, B, H, N, D).transpose(1, 2).contiguous()
    st["vd"] = _randn(g, B, N, H, D).half()
    st["mask"], st["n_draft"] = _trees(seed, B, N)
    st["out"] = torch.zeros((B, N, H * rep, D), dtype=torch.bfloat16, device="cuda")
    if own:
        from sub_bit_quantized_gb300 import kvq

        cfg, cache = _handle(st, B, H * rep)
        st["ws"] = kvq.make_tree_workspace(cfg, B, N)
        st["call"] = kvq.TreeAttnCall(cfg, cache, st["q"], st["kd"], st["vd"], st["mask"], st["out"],
                                      n_draft=st["n_draft"], ws=st["ws"])
    return st


def _prepare_commit(case, g):
    B, N, H, R = case["B"], case["N"], case["H"], case["R"]
    n = (R + _randint(g, 1, R + 1, B)).tolist()  # every fill of the key residual
    st = _cache(g, case, n, 2 * R)
    st.update(op="commit", N=N)
    # the key residual holds what came since its last flush, the value window is full
    nqk = torch.tensor(n) - 1 - (torch.tensor(n) - 1) % R
    st["lens"][1, :B], st["lens"][2, :B] = nqk.int().cuda(), (torch.tensor(n) - R).int().cuda()
    st["lens0"] = st["lens"].clone()
    st["kd"] = _keys(g, B, H, N, D).transpose(1, 2).contiguous()
    st["vd"] = _randn(g, B, N, H, D).half()
    st["n_accept"] = _randint(g, 1, N + 1, B).int()
    some = torch.rand((B, N), generator=g, device="cuda").argsort(-1)  # ancestors come before their children
    some.masked_fill_(torch.arange(N, device="cuda") >= st["n_accept"][:, None], N)
    st["path"] = some.sort(-1)[0].clamp(max=N - 1).int()
    w = case["window"]
    st["begin"] = torch.tensor([max(0, x - w) for x in n], dtype=torch.int32).cuda()
    st["ko"], st["vo"] = (torch.zeros((B, H, w, D), dtype=torch.float16, device="cuda") for _ in range(2))
    if own:
        from sub_bit_quantized_gb300 import kvq

        cfg, cache = _handle(st, B, H)
        st["call"] = kvq.KiviCommitCall(cfg, cache, st["kd"], st["vd"], st["path"], st["n_accept"])
        st["read"] = kvq.KiviReadCall(cfg, cache, st["ko"], st["vo"], tok_begin=st["begin"])
    return st


def _prepare_read(case, g):
    B, H, n = case["B"], case["H"], case["n"]
    lens = _lengths(g, B, case["ctx"])
    st = _cache(g, case, lens, 0)
    st["op"] = "read"
    st["begin"] = torch.tensor([max(0, x - n) for x in lens], dtype=torch.int32).cuda()  # the newest n tokens
    st["ko"], st["vo"] = (torch.zeros((B, H, n, D), dtype=DTYPES[case["out"]], device="cuda") for _ in range(2))
    if own:
        from sub_bit_quantized_gb300 import kvq

        cfg, cache = _handle(st, B, H)
        st["read"] = kvq.KiviReadCall(cfg, cache, st["ko"], st["vo"], tok_begin=st["begin"])
    return st


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "rows":
        return _prepare_rows(case, g)
    if case["op"] == "tree":
        return _prepare_tree(case, g, seed)
    if case["op"] == "commit":
        return _prepare_commit(case, g)
    return _prepare_read(case, g)


# ------------------------------------------------------------------------------------ plain forms

def _unpack(codes, bits):
    shift = torch.arange(8 // bits, device=codes.device, dtype=torch.uint8) * bits
    return ((codes.unsqueeze(-1) >> shift) & (2 ** bits - 1)).flatten(-2, -1).float()


def _at(x, t):
    """Rows t[b][j] of x [B][H][rows][...]."""
    return x.gather(2, t[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3]))


def _cached(st, t):
    """Keys and values (fp32) of the cached tokens t [B][n]: dequantized, or from the fp16 residuals."""
    B = t.shape[0]
    nqk, nqv = (st["lens"][i, :B, None].long() for i in (1, 2))
    tq = t.clamp(0, st["T"] - 1)
    per_group = [_at(st[x], tq // GROUP).float() for x in ("k_scale", "k_zero")]
    k = (_unpack(_at(st["k_codes"], tq), st["kb"]) - per_group[1]) * per_group[0]
    spread = [_at(st[x], tq).float().repeat_interleave(GROUP, -1) for x in ("v_scale", "v_zero")]
    v = (_unpack(_at(st["v_codes"], tq), st["vb"]) - spread[1]) * spread[0]
    kr = _at(st["k_resid"], (t - nqk).clamp(0, st["R"] - 1)).float()
    vr = _at(st["v_resid"], t % st["R"]).float()
    return torch.where((t < nqk)[:, None, :, None], k, kr), torch.where((t < nqv)[:, None, :, None], v, vr)


def _plain_rows(st):
    def norm(x, w):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()

    def rotate(x):
        if st["cos"] is None:
            return x
        c, s = (st[t][st["pos"].long()].unsqueeze(2) for t in ("cos", "sin"))
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    st["qo"].copy_(rotate(norm(st["q"], st["wq"])))
    st["ko"].copy_(rotate(norm(st["k"], st["wk"])))
    st["vo"].copy_(st["v"].float())


def _plain_tree(st):
    B, N, Hq, _ = st["q"].shape
    H, rep = st["H"], st["rep"]
    S = int(st["T"]) + st["R"]
    t = torch.arange(S, device="cuda").expand(B, S)
    k, v = _cached(st, t)
    k = torch.cat([k, st["kd"].transpose(1, 2).float()], 2)
    v = torch.cat([v, st["vd"].transpose(1, 2).float()], 2)
    q = st["q"].float().view(B, N, H, rep, D).transpose(1, 2).reshape(B, H, N * rep, D)
    s = q @ k.transpose(2, 3) / math.sqrt(D)
    j = torch.arange(N, device="cuda")
    n_draft = st["n_draft"].long()
    among = ((st["mask"].unsqueeze(-1) >> j) & 1).bool() & (j < n_draft[:, None])[:, None]
    before = (t < st["lens"][0, :B, None])[:, None].expand(B, N, S)
    seen = torch.cat([before, among], 2).repeat_interleave(rep, 1)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(B, H, N, rep, D).transpose(1, 2).reshape(B, N, Hq, D)
    real = (j < n_draft[:, None])[:, :, None, None]
    st["out"].copy_(torch.where(real, o.to(st["out"].dtype), st["out"]))


def _put(x, t, new, keep):
    """x's rows t[b][j] become new where keep[b][j]; the others stay."""
    old = _at(x, t)
    x.scatter_(2, t[:, None, :, None].expand_as(old), torch.where(keep[:, None, :, None], new, old))


def _plain_commit(st):
    B, N = st["path"].shape
    R, T = st["R"], st["T"]
    n, nqk, nqv = (st["lens"][i, :B, None].long() for i in range(3))
    m = st["n_accept"].long()[:, None]
    pick = st["path"].long()
    kn, vn = _at(st["kd"].transpose(1, 2), pick), _at(st["vd"].transpose(1, 2), pick)
    held = n - nqk  # keys in the residual
    j = torch.arange(R + N, device="cuda")[None]
    line = torch.where((j < held)[:, None, :, None], _at(st["k_resid"], j.clamp(max=R - 1).expand(B, -1)),
                       _at(kn, (j - held).clamp(0, N - 1)))  # keys of tokens nqk + j
    flush = held + m > R
    codes, s, z = _quantize_keys(line[:, :, :R], st["kb"])
    jr = torch.arange(R, device="cuda")[None]
    jg = torch.arange(R // GROUP, device="cuda")[None]
    _put(st["k_codes"], (nqk + jr).clamp(max=T - 1), codes, flush.expand(B, R))
    _put(st["k_scale"], (nqk // GROUP + jg).clamp(max=T // GROUP - 1), s, flush.expand(B, R // GROUP))
    _put(st["k_zero"], (nqk // GROUP + jg).clamp(max=T // GROUP - 1), z, flush.expand(B, R // GROUP))
    left = held + m - R * flush
    _put(st["k_resid"], jr.expand(B, R), _at(line, (jr + R * flush).clamp(max=R + N - 1)), jr < left)
    i = torch.arange(N, device="cuda")[None]
    out = (n + m - R - nqv).clamp(min=0)  # values that leave the window
    codes, s, z = _quantize_values(_at(st["v_resid"], (nqv + i) % R), st["vb"])
    for x, y in (("v_codes", codes), ("v_scale", s), ("v_zero", z)):
        _put(st[x], (nqv + i).clamp(max=T - 1), y, i < out)
    _put(st["v_resid"], (n + i) % R, vn, i < m)
    st["lens"][:, :B] = torch.cat([n + m, nqk + R * flush, nqv + out], 1).T.int()


def _plain_read(st):
    B, _, n, _ = st["ko"].shape
    t = st["begin"].long()[:, None] + torch.arange(n, device="cuda")
    there = (t < st["lens"][0, :B, None])[:, None, :, None]
    for o, x in zip((st["ko"], st["vo"]), _cached(st, t)):
        o.copy_(torch.where(there, x.to(o.dtype), o))


def run(state):
    st = state
    if st["op"] == "rows":
        st["call"]() if own else _plain_rows(st)
        return dict(q=st["qo"], k=st["ko"], v=st["vo"])
    if st["op"] == "tree":
        st["call"]() if own else _plain_tree(st)
        return st["out"]
    if st["op"] == "commit":
        st["lens"].copy_(st["lens0"])  # each pass commits to the same lengths
        if own:
            st["call"]()
            st["read"]()
        else:
            _plain_commit(st)
            _plain_read(st)
        B = st["path"].shape[0]
        return dict(k=st["ko"], v=st["vo"], n_tok=st["lens"][0, :B], n_quant_k=st["lens"][1, :B], n_quant_v=st["lens"][2, :B])
    st["read"]() if own else _plain_read(st)
    return dict(k=st["ko"], v=st["vo"])


# ------------------------------------------------------------------------------------ work

def _token_bytes(case):
    """Bytes of a cached token of one head: codes, its share of the key scales, the value scales."""
    return D * (case["kb"] + case["vb"]) / 8 + 2 * D * 2 / GROUP + 2 * (D // GROUP) * 2


def _held(case, n):
    """(quantized, fp16) tokens of a context of n."""
    quant = max(0, n - case["R"])
    return quant, n - quant


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    B, H = case["B"], case["H"]
    if case["op"] == "rows":
        rows = B * case["N"] * (case["Hq"] + 2 * H)
        table = B * case["N"] * D * 4 if case["rope"] else 0
        return {"bytes": rows * D * 4 + table, "flops": B * case["N"] * (case["Hq"] + H) * D * (7 if case["rope"] else 4)}
    if case["op"] == "tree":
        n = 0.875 * case["ctx"]  # the mean of the ragged lengths
        quant, half = _held(case, n)
        rows = case["N"] * case["rep"]
        cache = B * H * (quant * _token_bytes(case) + half * 4 * D)
        return {"bytes": cache + B * H * (4 * rows * D + 4 * case["N"] * D) + 8 * B * case["N"],
                "flops": 4 * B * H * rows * D * (n + case["N"] / 2)}
    if case["op"] == "commit":
        N, w, R = case["N"], case["window"], case["R"]
        half = (N + 1) / 2  # accepted tokens
        flushed = half / R * R  # a flush of R keys falls on half / R of the passes
        written = 2 * half * 4 * D + flushed * (2 * D + D * case["kb"] / 8 + 8) + half * (2 * D + D * case["vb"] / 8 + 16)
        quant, kept = max(0, w - R), min(w, R)
        return {"bytes": B * H * (written + quant * _token_bytes(case) + kept * 4 * D + w * 4 * D) + 24 * B,
                "flops": B * H * (w + 2 * N) * 4 * D}
    n = min(case["n"], 0.9 * case["ctx"]) if case["n"] < case["ctx"] else 0.875 * case["ctx"]
    half = min(n, case["R"])
    return {"bytes": B * H * ((n - half) * _token_bytes(case) + half * 4 * D + n * 2 * D * size[case["out"]]),
            "flops": B * H * n * 4 * D}


# ------------------------------------------------------------------------------------ exact values

def _table_row(codes, scale, zero, bits):
    """X = s (q - z) in fp64 from the bytes of a row; scale and zero broadcast over it."""
    c = codes.long()
    parts = [(c // 2 ** (bits * i)) % 2 ** bits for i in range(8 // bits)]
    return scale.double() * (torch.stack(parts, -1).reshape(*c.shape[:-1], D).double() - zero.double())


def _whole(st, b):
    """Keys and values [H][n_tok][D] of request b in fp64."""
    n, nqk, nqv = (int(x) for x in st["lens"][:, b])
    k = torch.empty((st["H"], n, D), dtype=torch.float64, device="cuda")
    v = torch.empty_like(k)
    g = nqk // GROUP
    grouped = st["k_codes"][b, :, :nqk].reshape(st["H"], g, GROUP, D * st["kb"] // 8)
    k[:, :nqk] = _table_row(grouped, st["k_scale"][b, :, :g, None], st["k_zero"][b, :, :g, None],
                            st["kb"]).reshape(st["H"], nqk, D)
    per = [st[x][b, :, :nqv, :, None].expand(-1, -1, -1, GROUP).reshape(st["H"], nqv, D) for x in ("v_scale", "v_zero")]
    v[:, :nqv] = _table_row(st["v_codes"][b, :, :nqv], per[0], per[1], st["vb"])
    k[:, nqk:] = st["k_resid"][b, :, : n - nqk].double()
    for t in range(nqv, n):
        v[:, t] = st["v_resid"][b, :, t % st["R"]].double()
    return k, v


def _exact_rows(st):
    outs = {}
    for name, x, w, to in (("q", "q", "wq", "qo"), ("k", "k", "wk", "ko")):
        y = st[x].double()
        y = y / ((y ** 2).sum(-1, keepdim=True) / D + st["eps"]).sqrt() * st[w].double()
        if st["cos"] is not None:
            z = torch.complex(y[..., : D // 2], y[..., D // 2:])
            p = st["pos"].long()
            z = z * torch.complex(st["cos"][p].double(), st["sin"][p].double())[:, :, None]
            y = torch.cat([z.real, z.imag], -1)
        outs[name] = y
    outs["v"] = st["v"].double()
    return outs


def _exact_tree(st):
    B, N, Hq, _ = st["q"].shape
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        k, v = _whole(st, b)
        real = int(st["n_draft"][b])
        k = torch.cat([k, st["kd"][b, :real].double().transpose(0, 1)], 1)
        v = torch.cat([v, st["vd"][b, :real].double().transpose(0, 1)], 1)
        n = k.shape[1] - real
        bits = [m % (1 << 64) for m in st["mask"][b].tolist()]
        blind = torch.tensor([[not bits[i] >> j & 1 for j in range(real)] for i in range(real)], device="cuda")
        for h in range(st["H"]):
            heads = slice(h * st["rep"], (h + 1) * st["rep"])
            s = torch.einsum("nrd,td->nrt", st["q"][b, :real, heads].double(), k[h]) * D ** -0.5
            s[:, :, n:].masked_fill_(blind[:, None], -math.inf)
            out[b, :real, heads] = torch.softmax(s, -1) @ v[h]
    return out


def _exact_group(x, bits):
    """The values that a group x [..., 32] stands for once it is quantized, in fp64."""
    lo, hi = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
    s = ((hi - lo) / (2 ** bits - 1)).half().double()
    s[s == 0] = 1
    z = (-lo / s).half().double()
    return s * (torch.clamp(torch.round(x / s + z), 0, 2 ** bits - 1) - z)


def _exact_commit(st):
    B, R, w = st["path"].shape[0], st["R"], st["ko"].shape[2]
    outs = dict(k=torch.zeros(st["ko"].shape, dtype=torch.float64, device="cuda"),
                v=torch.zeros(st["ko"].shape, dtype=torch.float64, device="cuda"), n_tok=None, n_quant_k=None, n_quant_v=None)
    for b in range(B):
        n, nqk, nqv = (int(x) for x in st["lens"][:, b])
        path = st["path"][b, : int(st["n_accept"][b])].long()
        k, v = _whole(st, b)
        k = torch.cat([k, st["kd"][b, path].double().transpose(0, 1)], 1)
        v = torch.cat([v, st["vd"][b, path].double().transpose(0, 1)], 1)
        n += len(path)
        if n - nqk > R:
            block = k[:, nqk : nqk + R].reshape(st["H"], R // GROUP, GROUP, D).transpose(2, 3)
            k[:, nqk : nqk + R] = _exact_group(block, st["kb"]).transpose(2, 3).reshape(st["H"], R, D)
        if n - R > nqv:
            rows = v[:, nqv : n - R].reshape(st["H"], n - R - nqv, D // GROUP, GROUP)
            v[:, nqv : n - R] = _exact_group(rows, st["vb"]).reshape(st["H"], n - R - nqv, D)
        begin = int(st["begin"][b])
        rows = min(w, n - begin)
        outs["k"][b, :, :rows], outs["v"][b, :, :rows] = k[:, begin : begin + rows], v[:, begin : begin + rows]
    return outs


def _exact_read(st):
    B, H, n, _ = st["ko"].shape
    outs = dict(k=torch.zeros((B, H, n, D), dtype=torch.float64, device="cuda"),
                v=torch.zeros((B, H, n, D), dtype=torch.float64, device="cuda"))
    for b in range(B):
        begin = int(st["begin"][b])
        for name, x in zip("kv", _whole(st, b)):
            rows = min(n, x.shape[1] - begin)
            outs[name][b, :, :rows] = x[:, begin : begin + rows]
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    return dict(rows=_exact_rows, tree=_exact_tree, commit=_exact_commit, read=_exact_read)[case["op"]](st)
