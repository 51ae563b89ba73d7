"""Cases that measure the operators of serving many continuations of one prompt.

The prompt is cached once, and every request attends to it together with its own tokens (``prefix``);
samples and beams take over one another's cache slots (``fork``); drafted tokens are verified against
the target's probabilities, which yields the path to commit and the next token (``verify``).

``run`` computes a pass in elementary torch operations, or with ``own`` set through the library.
"""
import math

import numpy as np
import torch

own = False

D = 128
GROUP = 32
PAGE = 8
SINK = 8
KEEP, FREE = -1, -2
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PART = ("k_codes", "k_scale", "k_zero", "v_codes", "v_scale", "v_zero", "k_resid", "v_resid")


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a few chats under one system prompt, just begun: latency
        dict(name="prefix_chat", op="prefix", B=4, H=8, rep=4, N=1, ctx=1013, own=57, kb=2, vb=2, R=128),
        # samples of one prompt, multi-head, as many as the attention benchmark's batch
        dict(name="prefix_mha_2bit", op="prefix", B=16, H=32, rep=1, N=1, ctx=4096, own=512, kb=2, vb=2, R=128),
        # a full batch of grouped-query requests under a long instruction
        dict(name="prefix_gqa_4bit", op="prefix", B=64, H=8, rep=4, N=1, ctx=8191, own=640, kb=4, vb=4, R=128),
        # chains of drafts over one long document: the most rows and the most tokens
        dict(name="prefix_drafts", op="prefix", B=16, H=8, rep=4, N=8, ctx=32768, own=1024, kb=4, vb=2, R=128),
        # a prompt cached once goes to the slots of a multi-head batch, from another cache
        dict(name="fork_prompt", op="fork", fmt="kivi", B=16, H=32, ctx=4096, kb=2, vb=2, R=128, one=True),
        # a beam search drops some of its beams in favour of others, in place
        dict(name="fork_beams", op="fork", fmt="kivi", B=64, H=8, ctx=1531, kb=4, vb=4, R=128, one=False),
        # a few samples of a short context, in a cache of index pages: latency
        dict(name="fork_pages", op="fork", fmt="vq", B=8, H=16, ctx=701, L=2, T=4, recent=64, one=False),
        # one request, a chain of four drafts: latency
        dict(name="verify_one", op="verify", B=1, N=5, V=32768, tree=False, draft=True, greedy=False, x="fp32"),
        # a batch of chains, drawn from a smaller model's distributions
        dict(name="verify_chains", op="verify", B=64, N=8, V=131072, tree=False, draft=True, greedy=False, x="fp32"),
        # trees whose children are drawn from one distribution each, odd vocabulary
        dict(name="verify_trees", op="verify", B=16, N=24, V=50021, tree=True, draft=True, greedy=False, x="fp32"),
        # trees of the most likely tokens, a point mass each
        dict(name="verify_points", op="verify", B=16, N=48, V=50021, tree=True, draft=False, greedy=False, x="fp32"),
        # without sampling: the logits themselves
        dict(name="verify_greedy", op="verify", B=32, N=16, V=131072, tree=True, draft=False, greedy=True, x="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "fork", "verify"])
    bits = dict(kb=rng.choice([2, 4]), vb=rng.choice([2, 4]), R=rng.choice([32, 64, 128]))
    if op == "prefix":
        H = rng.choice([1, 2, 4, 8, 16, 32])
        rep = rng.choice([1, 2, 3, 4, 7, 8]) if H < 16 else 1
        room = 16 * 8 * 32 * 32768  # query rows times tokens of the largest case
        N = _log(rng, 1, 64) if rng.random() < 0.5 else 1
        ctx = _log(rng, 1, max(1, min(32768, room // (H * rep * N))))
        B = _log(rng, 1, max(1, min(128, room // (H * rep * N * ctx))))
        mine = _log(rng, 1, max(1, min(4096, room // (H * rep * N * B), 16 * 8 * 2048 // (B * H))))
        return dict(op=op, B=B, H=H, rep=rep, N=N, ctx=ctx, own=mine, **bits)
    if op == "fork":
        H = rng.choice([1, 2, 4, 8, 16, 32])
        if rng.random() < 0.3:
            T = rng.choice([1, 2, 4])
            L = rng.choice([1, 2, 4])
            ctx = _log(rng, 1, 4000)
            most = 16 * 32 * 4000 // (H * L * T * (ctx // 4 + 400))
            return dict(op=op, fmt="vq", B=_log(rng, 1, max(1, min(64, most))), H=H, ctx=ctx, L=L, T=T,
                        recent=rng.choice([64, 256]), one=rng.random() < 0.5)
        ctx = _log(rng, 1, 20000)
        return dict(op=op, fmt="kivi", B=_log(rng, 1, max(1, min(128, 16 * 32 * 2000 // (H * (ctx + 500))))), H=H, ctx=ctx,
                    one=rng.random() < 0.5, **bits)
    N, V = _log(rng, 1, 64), _log(rng, 500, 160000)
    B = _log(rng, 1, max(1, min(128, 64 * 8 * 131072 // (2 * N * V))))
    greedy = rng.random() < 0.3
    return dict(op=op, B=B, N=N, V=V, tree=rng.random() < 0.6, draft=not greedy and rng.random() < 0.6, greedy=greedy,
                x=rng.choice(["bf16", "fp16", "fp32"]) if greedy else "fp32")


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _keys(g, *shape):
    """Keys with six large channels for each head (dimension 1), as the cache's quantizer expects them."""
    x = _randn(g, *shape)
    big = _rand(g, shape[1], D).argsort(-1)[:, :6]
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


def _kivi(g, case, n_tok, behind):
    """A KIVI cache of n_tok[b] tokens as a prefill and some decode steps leave it: keys of a multiple of
    the group quantized, values up to ``behind`` tokens less far."""
    B, H, R = len(n_tok), case["H"], case["R"]
    n = torch.tensor(n_tok)
    nqk = (n - R).clamp(min=0).add(GROUP - 1) // GROUP * GROUP
    less = (_rand(g, B) * (behind + 1)).long().cpu()
    nqv = torch.minimum((nqk - less).clamp(min=0), nqk).maximum(n - R).clamp(min=0)
    T = max(int(nqk.max()), GROUP)
    lens = torch.zeros((3, (B + 3) // 4 * 4), dtype=torch.int32)
    lens[0, :B], lens[1, :B], lens[2, :B] = n, nqk, nqv
    st = dict(B=B, H=H, R=R, T=T, kb=case["kb"], vb=case["vb"], lens=lens.cuda())
    st["k_codes"], st["k_scale"], st["k_zero"] = _quantize_keys(_keys(g, B, H, T, D), case["kb"])
    st["v_codes"], st["v_scale"], st["v_zero"] = _quantize_values(_randn(g, B, H, T, D).half(), case["vb"])
    st["k_resid"], st["v_resid"] = _keys(g, B, H, R, D), _randn(g, B, H, R, D).half()
    return st


def _kivi_handle(c, Hq):
    """The library's cache object over the buffers of ``c``."""
    from sub_bit_quantized_gb300 import kvq

    cfg = kvq.KiviConfig(n_heads=c["H"], n_q_heads=Hq, k_bits=c["kb"], v_bits=c["vb"], residual=c["R"], max_batch=c["B"],
                         max_tokens=c["T"])
    cache = kvq.KiviCache(kvq.KiviConfig(n_heads=c["H"], k_bits=c["kb"], v_bits=c["vb"], residual=GROUP, max_batch=c["B"]))
    cache.cfg = cfg
    for name in PART:
        setattr(cache, name, c[name])
    cache.n_tok, cache.n_quant_k, cache.n_quant_v = (c["lens"][i, :c["B"]] for i in range(3))
    return cfg, cache


def _lengths(g, B, ctx):
    """Ragged context lengths, the longest of them ctx."""
    n = (ctx * (0.5 + 0.5 * _rand(g, B))).ceil().int().clamp(1, ctx).tolist()
    n[0] = ctx
    return n


def _prepare_prefix(case, g):
    B, N, H, rep = case["B"], case["N"], case["H"], case["rep"]
    st = dict(op="prefix", rep=rep)
    st["prefix"] = _kivi(g, case, [case["ctx"]], 0)   # as its prefill left it
    st["mine"] = _kivi(g, case, _lengths(g, B, case["own"]), GROUP - 1)
    st["q"] = _randn(g, B, N, H * rep, D).bfloat16()
    # the new token and its drafts, a chain: row i sees the first i + 1 of them
    st["kd"] = _keys(g, B, H, N, D).transpose(1, 2).contiguous()
    st["vd"] = _randn(g, B, N, H, D).half()
    chain = [(2 << i) - 1 for i in range(N)]
    st["mask"] = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in chain]] * B, dtype=torch.int64).cuda()
    st["n_draft"] = (N - (_rand(g, B) * (N // 4 + 1)).int()).int()
    st["out"] = torch.zeros((B, N, H * rep, D), dtype=torch.bfloat16, device="cuda")
    if own:
        from sub_bit_quantized_gb300 import kvq

        cfg, cache = _kivi_handle(st["mine"], H * rep)
        pcfg, prefix = _kivi_handle(st["prefix"], H * rep)
        st["ws"] = kvq.make_prefix_workspace(cfg, pcfg, B, N)
        st["call"] = kvq.PrefixAttnCall(cfg, cache, pcfg, prefix, 0, st["q"], st["out"], k_draft=st["kd"], v_draft=st["vd"],
                                        mask=st["mask"], n_draft=st["n_draft"], ws=st["ws"])
    return st


def _vq(g, case, n_tok):
    """A LoopVQ cache (8 channels of 2 loop steps a codeword, or of the only one) of n_tok[b] tokens."""
    B, H, L, T, recent = len(n_tok), case["H"], case["L"], case["T"], case["recent"]
    NB, NG = max(1, T // 2), D // 8
    n = torch.tensor(n_tok)
    pages = ((n - SINK - recent) // PAGE).clamp(min=0)
    P = max(1, int(pages.max()))
    lens = torch.zeros((2, (B + 3) // 4 * 4), dtype=torch.int32)
    lens[0, :B], lens[1, :B] = n, pages
    c = dict(B=B, H=H, L=L, T=T, recent=recent, P=P, lens=lens.cuda())
    c["idx_k"], c["idx_v"] = (torch.randint(0, 256, (L, NB, B, H, P, PAGE * NG), generator=g, device="cuda").to(torch.uint8)
                              for _ in range(2))
    c["win_k"], c["win_v"] = (_randn(g, L, T, B, H, SINK + recent + PAGE, D).bfloat16() for _ in range(2))
    return c


def _vq_handle(c):
    from sub_bit_quantized_gb300 import kvq

    def cfg(**kw):
        Tc = min(2, c["T"])
        return kvq.VqConfig(T=c["T"], Tc=Tc, G=8 * Tc, n_layers=c["L"], n_heads=c["H"], max_ctx=32768, **kw)

    cache = kvq.VqCache(cfg())
    cache.cfg = cfg(recent=c["recent"], max_pages=c["P"], max_batch=c["B"])
    for name in ("idx_k", "idx_v", "win_k", "win_v"):
        setattr(cache, name, c[name])
    cache.seq_len, cache.n_pages = c["lens"][0, :c["B"]], c["lens"][1, :c["B"]]
    return cache.cfg, cache


def _arrays(st):
    return PART if st["fmt"] == "kivi" else ("idx_k", "idx_v", "win_k", "win_v")


def _prepare_fork(case, g):
    B = case["B"]
    make = _kivi if case["fmt"] == "kivi" else _vq
    more = (GROUP - 1,) if case["fmt"] == "kivi" else ()
    st = dict(op="fork", fmt=case["fmt"])
    if case["one"]:  # every slot takes over the prompt in slot 0 of another cache
        st["src"] = make(g, case, [case["ctx"]], *more)
        st["dst"] = make(g, case, _lengths(g, B, max(1, case["ctx"] // 2)), *more)
        room = "T" if case["fmt"] == "kivi" else "P"
        if st["dst"][room] < st["src"][room]:
            st["dst"] = make(g, case, [case["ctx"]] * B, *more)
        source = [0] * B
    else:  # some slots go on, some take over one of those, some are freed
        st["dst"] = st["src"] = make(g, case, _lengths(g, B, case["ctx"]), *more)
        u, v = _rand(g, B).tolist(), _rand(g, B).tolist()
        live = [0] + [i for i in range(1, B) if u[i] < 0.4]
        source = [KEEP if i in live else FREE if u[i] > 0.95 else live[int(v[i] * len(live))] for i in range(B)]
    st["source"] = torch.tensor(source, dtype=torch.int32).cuda()
    if own:
        from sub_bit_quantized_gb300 import kvq

        handle = (lambda c: _kivi_handle(c, c["H"])) if case["fmt"] == "kivi" else _vq_handle
        cfg, cache = handle(st["dst"])
        other = handle(st["src"]) if case["one"] else (None, None)
        st["call"] = kvq.CacheForkCall(cfg, cache, st["source"], from_cfg=other[0], from_cache=other[1])
    return st


def _prepare_verify(case, g, seed):
    B, N, V, x = case["B"], case["N"], case["V"], DTYPES[case["x"]]
    st = dict(op="verify", p=None, q=None, u=None)
    logits = 3 * _randn(g, B, N, V)
    rng = np.random.default_rng(seed)
    parent = np.tile(np.arange(N) - 1, (B, 1))
    if case["tree"] and N > 1:  # a parent among the nodes before, the later ones more often
        parent[:, 1:] = (np.arange(1, N) * rng.random((B, N - 1)) ** 0.5).astype(np.int64)
    st["parent"] = torch.from_numpy(parent.astype(np.int32)).cuda()
    st["n_draft"] = torch.from_numpy((N - rng.integers(0, N // 4 + 1, B)).astype(np.int32)).cuda()
    at = st["parent"].long().clamp(min=0)
    b = torch.arange(B, device="cuda")[:, None]
    if case["greedy"]:
        st["p"] = logits.to(x)
        best = st["p"].float().argmax(-1)[b, at]
        st["token"] = torch.where(_rand(g, B, N) < 0.7, best, (_rand(g, B, N) * V).long().clamp(max=V - 1)).int()
    else:
        st["p"] = torch.softmax(logits, -1)
        if case["draft"]:  # a smaller model: other logits, near these; its children are drawn from what it says
            logits += 0.8 * _randn(g, B, N, V)
            st["q"] = torch.softmax(logits, -1)
            of, bar = st["q"][b, at], _rand(g, B, N, 1)
            st["token"] = torch.searchsorted(of.cumsum(-1), bar).clamp(max=V - 1)[..., 0].int()
        else:  # the k-th child is the k-th best of a node
            nth = [[sum(row[j] == row[i] for j in range(i)) for i in range(N)] for row in parent.tolist()]
            best = st["p"].topk(min(V, 64), -1)[1]
            st["token"] = best[b, at, torch.tensor(nth, device="cuda").clamp(max=min(V, 64) - 1)].int()
        st["u"] = _rand(g, B, N)
    del logits
    st["path"] = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    st["count"], st["next"] = (torch.zeros((B,), dtype=torch.int32, device="cuda") for _ in range(2))
    if own:
        from sub_bit_quantized_gb300 import kvq

        st["call"] = kvq.VerifyDraftCall(st["p"], st["q"], st["token"], st["parent"], st["u"], st["path"], st["count"],
                                         st["next"], n_draft=st["n_draft"])
    return st


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "prefix":
        return _prepare_prefix(case, g)
    if case["op"] == "fork":
        return _prepare_fork(case, g)
    return _prepare_verify(case, g, seed)


# ------------------------------------------------------------------------------------ plain forms

def _unpack(codes, bits):
    shift = torch.arange(8 // bits, device=codes.device, dtype=torch.uint8) * bits
    return ((codes.unsqueeze(-1) >> shift) & (2 ** bits - 1)).flatten(-2, -1).float()


def _at(x, t):
    """Rows t[b][j] of x [B][H][rows][...]."""
    return x.gather(2, t[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3]))


def _cached(c):
    """Keys and values (fp32) of the tokens 0 .. T + R - 1 of every slot, and which of them are there."""
    B, T, R = c["B"], c["T"], c["R"]
    n, nqk, nqv = (c["lens"][i, :B, None].long() for i in range(3))
    t = torch.arange(T + R, device="cuda").expand(B, -1)
    scale, zero = (c[x].float().repeat_interleave(GROUP, 2) for x in ("k_scale", "k_zero"))
    k = (_unpack(c["k_codes"], c["kb"]) - zero) * scale
    scale, zero = (c[x].float().repeat_interleave(GROUP, 3) for x in ("v_scale", "v_zero"))
    v = (_unpack(c["v_codes"], c["vb"]) - zero) * scale
    k = torch.where((t < nqk)[:, None, :, None], _at(k, t.clamp(max=T - 1)),
                    _at(c["k_resid"], (t - nqk).clamp(0, R - 1)).float())
    v = torch.where((t < nqv)[:, None, :, None], _at(v, t.clamp(max=T - 1)), _at(c["v_resid"], t % R).float())
    return k, v, t < n


def _plain_prefix(st):
    B, N, Hq, _ = st["q"].shape
    H, rep = st["mine"]["H"], st["rep"]
    q = st["q"].float().view(B, N, H, rep, D).permute(2, 0, 1, 3, 4).reshape(H, B * N * rep, D) / math.sqrt(D)
    kp, vp, there = _cached(st["prefix"])
    s0 = (q @ kp[0].transpose(1, 2)).masked_fill_(~there[0], -math.inf)  # the prefix: rows of all requests at once
    k, v, before = _cached(st["mine"])
    k = torch.cat([k, st["kd"].transpose(1, 2).float()], 2)
    v = torch.cat([v, st["vd"].transpose(1, 2).float()], 2)
    rows = q.view(H, B, N * rep, D).transpose(0, 1)
    s1 = rows @ k.transpose(2, 3)
    j = torch.arange(N, device="cuda")
    real = j < st["n_draft"].long()[:, None]
    among = ((st["mask"].unsqueeze(-1) >> j) & 1).bool() & real[:, None]
    seen = torch.cat([before[:, None].expand(-1, N, -1), among], 2).repeat_interleave(rep, 1)[:, None]
    s1 = s1.masked_fill_(~seen, -math.inf).transpose(0, 1).reshape(H, B * N * rep, -1)
    m = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s0, s1 = s0.sub_(m).exp_(), s1.sub_(m).exp_()
    total = s0.sum(-1, keepdim=True) + s1.sum(-1, keepdim=True)
    o = s0 @ vp[0] + (s1.view(H, B, N * rep, -1).transpose(0, 1) @ v).transpose(0, 1).reshape(H, B * N * rep, D)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(H, B, N, rep, D).permute(1, 2, 0, 3, 4).reshape(B, N, Hq, D)
    st["out"].copy_(torch.where(real[:, :, None, None], o.to(st["out"].dtype), st["out"]))


def _move(dst, src, slots, source, dim, rows, valid):
    """Slot i of dst (dimension ``dim``) gets the valid rows (dimension ``rows``) of slot source[i] of src."""
    n = min(dst.shape[rows], src.shape[rows])
    new = src.narrow(rows, 0, n).index_select(dim, source.clamp(min=0))
    shape = [1] * dst.dim()
    shape[dim], shape[rows] = slots, n
    to = dst.narrow(rows, 0, n)
    to.copy_(torch.where(valid[:, :n].reshape(shape), new, to))


def _plain_fork(st):
    dst, src, source = st["dst"], st["src"], st["source"].long()
    B = dst["B"]
    moved, freed = source >= 0, source == FREE
    lens = src["lens"][:, source.clamp(min=0)].long()
    held = lambda used, rows: (torch.arange(rows, device="cuda") < used[:, None]) & moved[:, None]
    if st["fmt"] == "kivi":
        n, nqk, nqv = lens
        ring = torch.zeros((B, dst["R"]), dtype=torch.bool, device="cuda")
        t = nqv[:, None] + torch.arange(dst["R"], device="cuda")  # tokens of the value window
        ring.scatter_(1, t % dst["R"], (t < n[:, None]) & moved[:, None])
        for name in PART:
            used = dict(k_codes=nqk, k_scale=nqk // GROUP, k_zero=nqk // GROUP, k_resid=n - nqk).get(name, nqv)
            valid = ring if name == "v_resid" else held(used, src[name].shape[2])
            _move(dst[name], src[name], B, source, 0, 2, valid)
    else:
        n, pages = lens
        slots = SINK + dst["recent"] + PAGE
        first = SINK + PAGE * pages  # the first position behind the pages
        t = first[:, None] + torch.arange(slots - SINK, device="cuda")
        win = torch.zeros((B, slots), dtype=torch.bool, device="cuda")
        win.scatter_(1, SINK + (t - SINK) % (slots - SINK), (t < n[:, None]) & moved[:, None])
        win[:, :SINK] = held(n, SINK)
        for x in "kv":
            _move(dst["idx_" + x], src["idx_" + x], B, source, 2, 4, held(pages, src["idx_" + x].shape[4]))
            _move(dst["win_" + x], src["win_" + x], B, source, 2, 4, win)
    now = dst["lens"][:, :B]
    dst["lens"][:, :B] = torch.where(moved, lens.int(), torch.where(freed, torch.zeros_like(now), now))


def _plain_verify(st):
    p, q, u, parent, n_draft = st["p"], st["q"], st["u"], st["parent"].long(), st["n_draft"].long()
    B, N, V = p.shape
    b = torch.arange(B, device="cuda")
    node = torch.zeros(B, dtype=torch.long, device="cuda")
    count = torch.ones_like(node)
    st["path"][:, 0] = 0

    def step(i, taken):
        nonlocal node, count
        st["path"][b, count.clamp(max=N - 1)] = torch.where(taken, i, st["path"][b, count.clamp(max=N - 1)].long()).int()
        node, count = torch.where(taken, i, node), count + taken

    if u is None:
        best = p.float().argmax(-1)
        lowest = (p == p.gather(-1, best[..., None])).int().argmax(-1)  # of equal values the first
        for i in range(1, N):
            step(i, (parent[:, i] == node) & (i < n_draft) & (st["token"][:, i].long() == lowest[b, node]))
        st["next"].copy_(lowest[b, node])
        st["count"].copy_(count)
        return
    one = torch.ones(B, dtype=torch.float64, device="cuda")
    a, z = torch.zeros_like(one), one
    gone = torch.zeros((B, V), dtype=torch.bool, device="cuda")
    left = lambda: (p[b, node].double() - a[:, None] * q[b, node] if q is not None else p[b, node].double().masked_fill(gone, 0)).clamp(min=0)
    for i in range(1, N):
        tried = (parent[:, i] == node) & (i < n_draft)
        x = st["token"][:, i].long()
        w = left()
        wx = w[b, x]
        of = q[b, node, x].double() if q is not None else one
        taken = tried & (u[:, i].double() * z * of < wx)
        failed = tried & ~taken
        if q is not None:
            a = torch.where(failed, a + z, a)
            z = torch.where(failed, left().sum(-1), z)
        else:
            z = torch.where(failed, z - wx, z)
            gone[b, x] |= failed
        step(i, taken)
        a, z = a.masked_fill(taken, 0), z.masked_fill(taken, 1)
        gone &= ~taken[:, None]
    w = left()
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p[b, node].double())
    upto = w.cumsum(-1)
    passed = upto > u[:, :1].double() * upto[:, -1:]
    st["next"].copy_(passed.int().argmax(-1))
    st["count"].copy_(count)


def run(state):
    st = state
    if own:
        st["call"]()
    else:
        dict(prefix=_plain_prefix, fork=_plain_fork, verify=_plain_verify)[st["op"]](st)
    if st["op"] == "prefix":
        return st["out"]
    if st["op"] == "verify":
        return dict(path=st["path"], n_accept=st["count"], next=st["next"])
    c = st["dst"]
    return dict({name: c[name] for name in _arrays(st)}, lens=c["lens"])


# ------------------------------------------------------------------------------------ work

def _token_bytes(case):
    """Bytes of a cached token of one head: codes, its share of the key scales, the value scales."""
    return D * (case["kb"] + case["vb"]) / 8 + 2 * D * 2 / GROUP + 2 * (D // GROUP) * 2


def _cache_bytes(case, n):
    quant = max(0, n - case["R"])
    return case["H"] * (quant * _token_bytes(case) + (n - quant) * 4 * D)


def work(case):
    B = case["B"]
    if case["op"] == "prefix":
        H, N, rep, mine = case["H"], case["N"], case["rep"], 0.75 * case["own"]
        cached = _cache_bytes(case, case["ctx"]) + B * _cache_bytes(case, mine)
        return {"bytes": cached + B * H * N * (4 * rep * D + 4 * D) + 8 * B * N,
                "flops": 4 * B * H * N * rep * D * (case["ctx"] + mine + (N + 1) / 2)}
    if case["op"] == "fork":
        if case["fmt"] == "kivi":
            slot = _cache_bytes(case, case["ctx"] if case["one"] else 0.75 * case["ctx"])
        else:
            n = case["ctx"] if case["one"] else 0.75 * case["ctx"]
            held = min(n, SINK + case["recent"] + PAGE / 2)
            slot = case["L"] * case["H"] * (case["T"] * held * 4 * D + max(1, case["T"] // 2) * (n - held) * 2 * D // 8)
        read, written = (1, B) if case["one"] else (min(0.4 * B, 0.55 * B), 0.55 * B)  # distinct sources, slots that move
        return {"bytes": slot * (read + written), "flops": 0}
    # a row of the target at the path's end, one of the draft where something was rejected there; without sampling a
    # row for each node of the path
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["x"]]
    rows = 2 if case["draft"] else 1
    if case["greedy"]:
        rows = min(case["N"], 2.5)
    return {"bytes": B * case["V"] * size * rows + 12 * B * case["N"], "flops": B * case["V"] * rows * 2}


# ------------------------------------------------------------------------------------ exact values

def _table(codes, scale, zero, bits):
    """X = s (q - z) in fp64 from the bytes of rows; scale and zero broadcast over them."""
    c = codes.long()
    parts = [(c // 2 ** (bits * i)) % 2 ** bits for i in range(8 // bits)]
    return scale.double() * (torch.stack(parts, -1).reshape(*c.shape[:-1], D).double() - zero.double())


def _whole(c, b):
    """Keys and values [H][n_tok][D] of slot b in fp64."""
    n, nqk, nqv = (int(x) for x in c["lens"][:, b])
    H, g = c["H"], nqk // GROUP
    k = torch.empty((H, n, D), dtype=torch.float64, device="cuda")
    v = torch.empty_like(k)
    grouped = c["k_codes"][b, :, :nqk].reshape(H, g, GROUP, D * c["kb"] // 8)
    k[:, :nqk] = _table(grouped, c["k_scale"][b, :, :g, None], c["k_zero"][b, :, :g, None], c["kb"]).reshape(H, nqk, D)
    per = [c[x][b, :, :nqv, :, None].expand(-1, -1, -1, GROUP).reshape(H, nqv, D) for x in ("v_scale", "v_zero")]
    v[:, :nqv] = _table(c["v_codes"][b, :, :nqv], per[0], per[1], c["vb"])
    k[:, nqk:] = c["k_resid"][b, :, : n - nqk].double()
    for t in range(nqv, n):
        v[:, t] = c["v_resid"][b, :, t % c["R"]].double()
    return k, v


def _exact_prefix(st):
    B, N, Hq, _ = st["q"].shape
    rep = st["rep"]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    k0, v0 = _whole(st["prefix"], 0)
    for b in range(B):
        k1, v1 = _whole(st["mine"], b)
        for i in range(int(st["n_draft"][b])):
            sees = [j for j in range(int(st["n_draft"][b])) if int(st["mask"][b, i]) >> j & 1]
            k = torch.cat([k0, k1, st["kd"][b, sees].double().transpose(0, 1)], 1)
            v = torch.cat([v0, v1, st["vd"][b, sees].double().transpose(0, 1)], 1)
            q = st["q"][b, i].double().view(-1, rep, D)
            s = torch.einsum("hrd,htd->hrt", q, k) * D ** -0.5
            out[b, i] = (torch.softmax(s, -1) @ v).view(Hq, D)
    return out


def _exact_fork(st):
    """Slot by slot, from copies of what was there."""
    old = {name: x.clone() for name, x in st["src"].items() if torch.is_tensor(x)}
    new = {name: x.clone() for name, x in st["dst"].items() if torch.is_tensor(x)}
    for i, s in enumerate(st["source"].tolist()):
        if s == FREE:
            new["lens"][:, i] = 0
        if s < 0:
            continue
        new["lens"][:, i] = old["lens"][:, s]
        lens = old["lens"][:, s].tolist()
        if st["fmt"] == "kivi":
            n, nqk, nqv = lens
            for name, rows in (("k_codes", nqk), ("k_scale", nqk // GROUP), ("k_zero", nqk // GROUP), ("v_codes", nqv),
                               ("v_scale", nqv), ("v_zero", nqv), ("k_resid", n - nqk)):
                new[name][i, :, :rows] = old[name][s, :, :rows]
            for t in range(nqv, n):
                new["v_resid"][i, :, t % st["dst"]["R"]] = old["v_resid"][s, :, t % st["dst"]["R"]]
        else:
            n, pages = lens
            ring = st["dst"]["recent"] + PAGE
            rows = list(range(min(n, SINK))) + [SINK + (t - SINK) % ring for t in range(SINK + PAGE * pages, n)]
            for x in "kv":
                new["idx_" + x][:, :, i, :, :pages] = old["idx_" + x][:, :, s, :, :pages]
                new["win_" + x][:, :, i, :, rows] = old["win_" + x][:, :, s, :, rows]
    return dict({name: new[name] for name in _arrays(st)}, lens=new["lens"])


def _exact_verify(st):
    """Request by request with the distributions themselves: a rejected draw leaves max(0, r - q), normalised."""
    B, N = st["token"].shape
    path, count, nxt = np.zeros((B, N), np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    token, parent, real = (st[x].cpu().numpy() for x in ("token", "parent", "n_draft"))
    u = None if st["u"] is None else st["u"].double().cpu().numpy()
    for b in range(B):
        row = lambda x, i: st[x][b, i].double().cpu().numpy()
        node, found = 0, [0]
        r = row("p", 0)
        total, rejected = 1.0, False
        for i in range(1, real[b]):
            if parent[b, i] != node:
                continue
            x = token[b, i]
            if u is None:
                taken = x == int(np.argmax(r))
            elif st["q"] is not None:
                qx = float(st["q"][b, node, x])
                taken = u[b, i] * total * qx < r[x]
                if not taken:
                    r = np.maximum(r - total * row("q", node), 0)
                    total = r.sum()
            else:
                taken = u[b, i] * total < r[x]
                if not taken:
                    total -= r[x]
                    r[x] = 0
            if taken:
                node = i
                found.append(i)
                r, total = row("p", i), 1.0
        if u is None:
            nxt[b] = np.argmax(r)
        else:
            r = r if r.sum() > 0 else row("p", node)
            upto = np.cumsum(r)
            nxt[b] = np.argmax(upto > u[b, 0] * upto[-1])
        path[b, : len(found)], count[b] = found, len(found)
    return {name: torch.from_numpy(x) for name, x in dict(path=path, n_accept=count, next=nxt).items()}


def exact(case, seed):
    st = prepare(case, seed)
    return dict(prefix=_exact_prefix, fork=_exact_fork, verify=_exact_verify)[case["op"]](st)
