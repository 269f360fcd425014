"""Cases and plain forms of the linear-attention serving operators.

Four operators that a serving step of a linear-attention layer uses together: the chunked
and the recurrent form of linear attention with a decay for each head (``op`` "chunk" and
"token"), the block plan built from request lengths ("plan") and the group norm with an
activation ("norm"). ``run`` makes the library's calls where ``own`` is true and computes
the same in elementary torch operations, in 32 bits, where it is false; ``exact`` computes
it from the definitions in 64 bits, token by token.
"""
from __future__ import annotations

import math

import torch
import torch.nn.functional as F

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
CHUNK = 64  # tokens per chunk of the plain chunked form


def listed():
    return [
        # one short prompt: the latency of a prefill call
        dict(name="prompt_short", op="chunk", B=1, T=37, H=16, HV=16, K=128, V=128, dtype="bf16",
             decay="token", packed=False),
        # a dense prefill batch at the library's own prefill sizes, with carried-in states
        dict(name="prompt_batch", op="chunk", B=2, T=4096, H=16, HV=16, K=128, V=128,
             dtype="bf16", decay="token", packed=False),
        # more value heads than key heads at the library's own sizes: the largest prefill
        dict(name="prompt_gva", op="chunk", B=4, T=8192, H=8, HV=32, K=128, V=256, dtype="bf16",
             decay="head", packed=False),
        # one long document with few heads, q, k and v views of one fused projection
        dict(name="prompt_long", op="chunk", B=1, T=16384, H=4, HV=4, K=64, V=64, dtype="fp16",
             decay="token", packed=True),
        # full precision at odd sizes, key heads shared by three value heads
        dict(name="prompt_odd", op="chunk", B=3, T=333, H=2, HV=6, K=48, V=80, dtype="fp32",
             decay="token", packed=False),
        # a packed batch of ragged prompts that continue cached prefixes, states in pages
        dict(name="prompt_paged", op="paged", n=16, low=64, high=2048, H=32, HV=32, K=128, V=128,
             block=256, dtype="bf16", decay="token"),
        # one request decoding: the latency of a single token
        dict(name="token_one", op="token", n=1, S=1, H=16, HV=16, K=128, V=128, dtype="bf16",
             decay="token", block=0),
        # a full decode batch with paged states, some entries padding
        dict(name="token_batch", op="token", n=256, S=1, H=32, HV=32, K=128, V=128, dtype="bf16",
             decay="token", block=256),
        # the plan of a decode step: every request one token
        dict(name="plan_tokens", op="plan", n=256, block=64, context=8192, query=1, spare=1.5),
        # the plan of a prefill step: ragged prompts of up to 2048 tokens
        dict(name="plan_prompts", op="plan", n=64, block=16, context=4096, query=2048, spare=1.5),
        # a layer's output norm and gate: statistics per token and head
        dict(name="norm_tokens", op="norm", N=8192, L=1, C=4096, G=32, gate=True, dtype="bf16"),
        # statistics over all positions of a sample, channels not a power of two
        dict(name="norm_positions", op="norm", N=4, L=4096, C=320, G=32, gate=False, dtype="fp16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "paged", "token", "plan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    H = rng.choice([1, 2, 4, 8, 16])
    HV = H * rng.choice([1, 1, 1, 2, 3, 4])
    K = rng.choice([32, 48, 64, 96, 128, 128, 128])
    V = rng.choice([32, 64, 80, 128, 128, 128, 256])
    decay = rng.choice(["token", "token", "head", "none"])
    if op == "chunk":
        B = _log(rng, 1, 8)
        T = _log(rng, 1, max(2, min(16384, (1 << 26) // (B * HV * (K + V)))))
        return dict(op=op, B=B, T=T, H=H, HV=HV, K=K, V=V, dtype=dtype,
                    decay=decay if T <= 2048 else "token", packed=rng.random() < 0.5)
    if op == "paged":
        n = _log(rng, 1, 24)
        high = _log(rng, 2, 2048)
        return dict(op=op, n=n, low=0 if rng.random() < 0.3 else 1, high=high, H=min(H, 8),
                    HV=min(H, 8) * (HV // H), K=K, V=min(V, 128),
                    block=rng.choice([64, 128, 256, 512]), dtype=dtype, decay="token")
    if op == "token":
        return dict(op=op, n=_log(rng, 1, 300), S=rng.choice([1, 1, 1, 2, 4]), H=H, HV=HV, K=K,
                    V=min(V, 128), dtype=dtype, decay=decay,
                    block=rng.choice([0, 1, 16, 64, 256]))
    if op == "plan":
        query = rng.choice([1, 1, 7, 64, 512, 2048])
        return dict(op=op, n=_log(rng, 1, 1024 if query <= 64 else 96),
                    block=rng.choice([1, 16, 24, 64, 128, 256]),
                    context=_log(rng, 1, 16384), query=query, spare=rng.choice([0.5, 1.2, 2.0]))
    G = rng.choice([1, 2, 4, 8, 16, 32])
    C = G * rng.choice([3, 8, 10, 16, 32, 64, 80, 128])
    if rng.random() < 0.5:
        L, N = 1, _log(rng, 1, max(2, (1 << 25) // C))
    else:
        L = _log(rng, 2, 16384)
        N = _log(rng, 1, max(2, min(32, (1 << 25) // (C * L))))
    return dict(op=op, N=N, L=L, C=C, G=G, gate=rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _decay(gen, kind, lead, HV):
    """Log decays. Per token: -A softplus(a + bias) with A in [1, 16] and the bias such that
    softplus(bias) is spread over [0.001, 0.1]; per head: log(1 - 2^-(5 + 8 h / HV))."""
    if kind == "none":
        return None
    if kind == "head":
        h = torch.arange(HV, device="cuda", dtype=torch.float32)
        return torch.log1p(-torch.exp2(-5.0 - 8.0 * h / HV)).contiguous()
    A = 1.0 + 15.0 * torch.rand(HV, generator=gen, device="cuda")
    dt = torch.exp(torch.rand(HV, generator=gen, device="cuda") * math.log(100.0)
                   + math.log(0.001))
    a = torch.randn(*lead, HV, generator=gen, device="cuda")
    return -A * F.softplus(0.5 * a + dt + torch.log(-torch.expm1(-dt)))


def _qkv(gen, lead, H, HV, K, V, dtype, packed):
    """q and k as they leave a convolution with SiLU, v ~ N(0, 1); `packed`: views of one
    projection [.., H K + H K + HV V]."""
    dt = DTYPES[dtype]
    x = torch.randn(*lead, 2 * H * K + HV * V, generator=gen, device="cuda")
    x[..., :2 * H * K] = F.silu(x[..., :2 * H * K])
    x = x.to(dt)
    q, k, v = x.split([H * K, H * K, HV * V], dim=-1)
    q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (HV, V))
    return (q, k, v) if packed else (q.contiguous(), k.contiguous(), v.contiguous())


def _lengths(case, seed):
    """Host-side request lengths (the same for every seed, so that shapes are) and contexts of a
    packed batch."""
    n = case["n"]
    gen = torch.Generator().manual_seed(n * 7919 + case["high"])
    lens = torch.randint(case["low"], case["high"] + 1, (n,), generator=gen)
    lens[0] = case["high"]
    gen.manual_seed(seed * 7 + 1)
    ctx = torch.randint(0, 4 * case["block"], (n,), generator=gen)
    ctx[torch.rand(n, generator=gen) < 0.3] = 0
    return lens, ctx


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, seed, gen)


def _prepare_chunk(c, seed, gen):
    q, k, v = _qkv(gen, (c["B"], c["T"]), c["H"], c["HV"], c["K"], c["V"], c["dtype"], c["packed"])
    s0 = torch.randn(c["B"], c["HV"], c["K"], c["V"], generator=gen, device="cuda")
    return dict(op="chunk", q=q, k=k, v=v, s0=s0, scale=c["K"] ** -0.5,
                g=_decay(gen, c["decay"], (c["B"], c["T"]), c["HV"]))


def _tables(gen, used, width, n_pages=0):
    """Block tables [n, width] with used[r] distinct pages of n_pages (0: just as many) in row
    r, -1 past them."""
    total = int(used.sum())
    pages = torch.randperm(max(total, n_pages), generator=gen, device="cuda").to(torch.int32)
    used = used.cuda()
    first = torch.cumsum(used, 0) - used
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j).clamp_(max=max(total - 1, 0))
    return torch.where(j < used[:, None], pages[at] if total else at.int(), -1).contiguous()


def _prepare_paged(c, seed, gen):
    lens, ctx = _lengths(c, seed)
    bs = c["block"]
    T = int(lens.sum())
    q, k, v = _qkv(gen, (1, T), c["H"], c["HV"], c["K"], c["V"], c["dtype"], False)
    cu = torch.zeros(c["n"] + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(lens, 0)
    used = (ctx + lens + bs - 1) // bs
    n_pages = int(((lens + bs - 1) // bs + 4).sum())
    tables = _tables(gen, used, max(1, int(used.max())), n_pages)
    pool = torch.randn(n_pages, c["HV"], c["K"], c["V"], generator=gen, device="cuda")
    # what the scheduler knows on the host: each block that the step ends or reaches
    req, blk = [], []
    for r in range(c["n"]):
        if lens[r]:
            b = torch.arange(int(ctx[r]) // bs, int(used[r]))
            req.append(torch.full_like(b, r))
            blk.append(b)
    cat = lambda p: (torch.cat(p) if p else torch.zeros(0, dtype=torch.int64)).cuda()  # noqa: E731
    return dict(op="paged", q=q, k=k, v=v, g=_decay(gen, c["decay"], (1, T), c["HV"]), pool=pool,
                tables=tables, cu=cu.to(torch.int32).cuda(), ctx=ctx.to(torch.int32).cuda(),
                block=bs, scale=c["K"] ** -0.5, longest=int(lens.max()), req=cat(req), blk=cat(blk))


def _prepare_token(c, seed, gen):
    n, S, bs = c["n"], c["S"], c["block"]
    q, k, v = _qkv(gen, (n, S), c["H"], c["HV"], c["K"], c["V"], c["dtype"], False)
    s = dict(op="token", q=q, k=k, v=v, g=_decay(gen, c["decay"], (n, S), c["HV"]),
             scale=c["K"] ** -0.5, block=bs)
    if bs == 0:
        s["state"] = torch.randn(n, c["HV"], c["K"], c["V"], generator=gen, device="cuda")
        return s
    host = torch.Generator().manual_seed(seed * 7 + 2)
    ctx = torch.randint(0, 4 * bs, (n,), generator=host)
    pad = torch.rand(n, generator=host) < 0.06
    # only the blocks that the step reads or writes need pages of their own here
    lo = (ctx - 1).clamp(min=0) // bs
    hi = (ctx + S - 1) // bs
    count = torch.where(pad, 0, hi - lo + 1)
    total = n * (S // bs + 2)
    width = int(hi.max()) + 1
    perm = torch.randperm(total, generator=host).to(torch.int32)
    first = torch.cumsum(count, 0) - count
    j = torch.arange(width)[None] - lo[:, None]
    inside = (j >= 0) & (j < count[:, None])
    tables = torch.where(inside, perm[(first[:, None] + j).clamp(0, total - 1)], -1)
    s["tables"] = tables.to(torch.int32).contiguous().cuda()
    s["ctx"] = ctx.to(torch.int32).cuda()
    s["pool"] = torch.randn(total, c["HV"], c["K"], c["V"], generator=gen, device="cuda")
    # what the scheduler knows on the host: the steps after which a state is kept
    t = torch.arange(S)[None]
    keep = (((ctx[:, None] + t + 1) % bs == 0) | (t + 1 == S)) & ~pad[:, None]
    s["req"], s["step"] = (x.cuda() for x in keep.nonzero(as_tuple=True))
    return s


def _prepare_plan(c, seed, gen):
    n, bs = c["n"], c["block"]
    host = torch.Generator().manual_seed(seed * 7 + 3)
    ctx = torch.randint(0, c["context"] + 1, (n,), generator=host)
    ctx[torch.rand(n, generator=host) < 0.1] = 0
    qry = torch.randint(1, c["query"] + 1, (n,), generator=host)
    qry[torch.rand(n, generator=host) < 0.1] = 0  # requests that sit this step out
    have = (ctx + bs - 1) // bs
    need = (ctx + qry + bs - 1) // bs - have
    width = (c["context"] + c["query"] + bs - 1) // bs
    tables = _tables(gen, have, width)
    spare = int(c["spare"] * int(need.sum())) + 2
    free = (torch.randperm(spare, generator=gen, device="cuda") + int(have.sum())).to(torch.int32)
    return dict(op="plan", ctx=ctx.to(torch.int32).cuda(), qry=qry.to(torch.int32).cuda(),
                tables=tables, free=free, used=torch.ones(1, dtype=torch.int32, device="cuda"),
                block=bs, tokens=n * c["query"])


def _prepare_norm(c, seed, gen):
    dt = DTYPES[c["dtype"]]
    shape = (c["N"], c["L"], c["C"])
    x = torch.randn(*shape, generator=gen, device="cuda")
    x = (x * 2.0 + torch.randn(c["C"], generator=gen, device="cuda")).to(dt)
    gate = torch.randn(*shape, generator=gen, device="cuda").to(dt) if c["gate"] else None
    w = 1.0 + 0.1 * torch.randn(c["C"], generator=gen, device="cuda")
    b = 0.1 * torch.randn(c["C"], generator=gen, device="cuda")
    return dict(op="norm", x=x, gate=gate, w=w, b=b, groups=c["G"], eps=1e-5)


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_chunk(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    return gdp.gdp_linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"],
                                    initial_state=s["s0"])


def _own_paged(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    o = gdp.gdp_linear_chunk_fwd_paged(s["q"], s["k"], s["v"], s["g"], s["cu"], s["pool"],
                                       s["tables"], s["ctx"], s["block"], scale=s["scale"])
    return o, s["pool"]


def _own_token(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    if s["block"] == 0:
        return gdp.gdp_linear_recurrent_update(s["q"], s["k"], s["v"], s["g"], s["state"],
                                               scale=s["scale"]), s["state"]
    o = gdp.gdp_linear_recurrent_update_paged(s["q"], s["k"], s["v"], s["g"], s["pool"],
                                              s["tables"], s["ctx"], s["block"], scale=s["scale"])
    return o, s["pool"]


def _own_plan(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    return (*gdp.gdp_block_plan(s["ctx"], s["qry"], s["tables"], s["free"], s["used"], s["block"],
                                s["tokens"]), s["tables"])


def _own_norm(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    return gdp.gdp_group_norm(s["x"], s["groups"], s["w"], s["b"], gate=s["gate"], eps=s["eps"],
                              activation="silu")


def _segment_sums(x):
    """[.., n] -> [.., n, n]: entry (t, i) is the sum of x over i < j <= t, -inf for i > t."""
    n = x.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    s = torch.where(low, x[..., :, None], 0.0).cumsum(-2)
    return torch.where(low | torch.eye(n, dtype=torch.bool, device=x.device), s, -torch.inf)


def _chunked(q, k, v, g, s0, scale):
    """q, k [N, L, HV, K], v [N, L, HV, V], g [N, L, HV], s0 [N, HV, K, V] in 32 bits, L whole
    chunks. Returns o [N, L, HV, V] and the states at the chunk boundaries
    [N, HV, L / CHUNK + 1, K, V]."""
    N, L, HV, K = q.shape
    V, n = v.shape[-1], L // CHUNK
    q, k, v = (x.reshape(N, n, CHUNK, HV, -1).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    g = g.reshape(N, n, CHUNK, HV).permute(0, 3, 1, 2)
    d = torch.exp(_segment_sums(g))
    o = ((q @ k.transpose(-1, -2)) * d) @ v
    u = k.transpose(-1, -2) @ (v * d[..., -1, :, None])
    total = torch.cat([torch.zeros_like(g[..., :1, 0]), g.sum(-1)], -1)
    s = torch.exp(_segment_sums(total)) @ torch.cat([s0[:, :, None], u], 2).reshape(N, HV, n + 1, K * V)
    s = s.reshape(N, HV, n + 1, K, V)
    o = o + (q * torch.exp(g.cumsum(-1))[..., None]) @ s[:, :, :n]
    return (o * scale).permute(0, 2, 3, 1, 4).reshape(N, L, HV, V), s


def _full_decay(g, lead, HV, device):
    if g is None:
        return torch.zeros(*lead, HV, device=device)
    return g.float().expand(*lead, HV)


def _plain_chunk(s):
    q, k, v = (s[x].float() for x in "qkv")
    B, T, H, _ = q.shape
    HV = v.shape[2]
    g = _full_decay(s["g"], (B, T), HV, q.device)
    q, k = (x.repeat_interleave(HV // H, 2) for x in (q, k))
    more = -T % CHUNK
    q, k, v = (F.pad(x, (0, 0, 0, 0, 0, more)) for x in (q, k, v))
    o, st = _chunked(q, k, v, F.pad(g, (0, 0, 0, more)), s["s0"], s["scale"])
    return o[:, :T].to(s["q"].dtype), st[:, :, -1].contiguous()


def _plain_paged(s):
    cu, ctx, bs, HV = s["cu"].long(), s["ctx"].long(), s["block"], s["v"].shape[2]
    H, T = s["q"].shape[2], s["q"].shape[1]
    lens = cu[1:] - cu[:-1]
    # each request in a row of its own, its chunks ending where its blocks do
    L = -(-(s["longest"] + CHUNK - 1) // CHUNK) * CHUNK
    j = torch.arange(L, device=cu.device)[None] - (ctx % CHUNK)[:, None]
    inside = (j >= 0) & (j < lens[:, None])
    at = torch.where(inside, cu[:-1, None] + j, 0)
    take = lambda x: torch.where(inside[..., None, None], x[0][at].float(), 0.0)  # noqa: E731
    q, k, v = (take(s[x]) for x in "qkv")
    q, k = (x.repeat_interleave(HV // H, 2) for x in (q, k))
    g = torch.where(inside[..., None], s["g"][0][at], 0.0)
    page = s["tables"].long().gather(1, ((ctx - 1).clamp(min=0) // bs)[:, None])[:, 0]
    s0 = torch.where((ctx > 0)[:, None, None, None], s["pool"][page.clamp(min=0)], 0.0)
    o, st = _chunked(q, k, v, g, s0, s["scale"])
    out = torch.zeros(1, T + 1, HV, v.shape[-1], device=cu.device)
    out[0, torch.where(inside, at, T)] = o
    end = ((s["blk"] + 1) * bs - ctx[s["req"]] // CHUNK * CHUNK) // CHUNK
    pages = s["tables"].long()[s["req"], s["blk"]]
    s["pool"][pages] = st[s["req"], :, end.clamp(max=L // CHUNK)]
    return out[:, :T].to(s["q"].dtype), s["pool"]


def _plain_token(s):
    q, k, v = (s[x].float() for x in "qkv")
    n, S, H, K = q.shape
    HV = v.shape[2]
    g = _full_decay(s["g"], (n, S), HV, q.device)
    q, k = (x.repeat_interleave(HV // H, 2) for x in (q, k))
    # all S steps at once: o_t = q_t (e^(G_t) S0 + sum_{i <= t} e^(G_t - G_i) k_i v_i^T)
    q, k, v, g = q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), g.transpose(1, 2)
    d = torch.exp(_segment_sums(g))                             # [n, HV, S, S]
    first = torch.exp(g.cumsum(-1))                             # [n, HV, S]
    inner = (((q @ k.transpose(-1, -2)) * d) @ v)
    if s["block"] == 0:
        o = inner + (q * first[..., None]) @ s["state"]
        s["state"].copy_(first[..., -1, None, None] * s["state"]
                         + k.transpose(-1, -2) @ (v * d[..., -1, :, None]))
        return (o * s["scale"]).transpose(1, 2).to(s["q"].dtype).contiguous(), s["state"]
    bs, ctx, pool, tables = s["block"], s["ctx"].long(), s["pool"], s["tables"].long()
    page = tables.gather(1, ((ctx - 1).clamp(min=0) // bs)[:, None])[:, 0]
    written = tables.gather(1, (ctx[:, None] + torch.arange(S, device=ctx.device)) // bs)
    live = (written[:, -1] >= 0)[:, None, None, None]
    s0 = torch.where((ctx > 0)[:, None, None, None], pool[page.clamp(min=0)], 0.0)
    o = torch.where(live, inner + (q * first[..., None]) @ s0, 0.0)
    # the states after the steps that end a block or the call
    r, t = s["req"], s["step"]
    after = (d[r, :, t, :, None] * k[r]).transpose(-1, -2) @ v[r]
    pool[written[r, t]] = after + first[r, :, t, None, None] * s0[r]
    return (o * s["scale"]).transpose(1, 2).to(s["q"].dtype).contiguous(), pool


def _plain_plan(s):
    ctx, qry, bs, N = s["ctx"].long(), s["qry"].long(), s["block"], s["tokens"]
    n, width = s["tables"].shape
    have = (ctx + bs - 1) // bs
    need = (ctx + qry + bs - 1) // bs - have
    fits = (s["used"] + need.cumsum(0) <= s["free"].numel()) & (qry.cumsum(0) <= N)
    qry, need = torch.where(fits, qry, 0), torch.where(fits, need, 0)
    cu = torch.cat([torch.zeros_like(qry[:1]), qry.cumsum(0)])
    first = need.cumsum(0) - need + s["used"]
    j = torch.arange(width, device=ctx.device)[None] - have[:, None]
    new = (j >= 0) & (j < need[:, None])
    at = torch.where(new, first[:, None] + j, 0)
    s["tables"].copy_(torch.where(new, s["free"][at], s["tables"]))
    t = torch.arange(N, device=ctx.device)
    req = (t[:, None] >= cu[None, 1:]).sum(1) if n * N <= 1 << 27 else torch.searchsorted(cu[1:], t, right=True)
    inside = t < cu[-1]
    req = torch.where(inside, req, 0)
    pos = ctx[req] + t - cu[req]
    page = s["tables"].long()[req, torch.where(inside, pos // bs, 0)]
    slot = torch.where(page >= 0, page * bs + pos % bs, -1)
    req, pos, slot = (torch.where(inside, x, -1) for x in (req, pos, slot))
    used = s["used"] + need.sum().int()
    return cu.int(), req.int(), pos.int(), slot, used, s["tables"]


def _plain_norm(s):
    x = s["x"].float()
    N, L, C = x.shape
    y = x.reshape(N, L, s["groups"], C // s["groups"])
    mean = y.mean((1, 3), keepdim=True)
    y = y - mean
    rstd = torch.rsqrt((y * y).mean((1, 3), keepdim=True) + s["eps"])
    y = (y * rstd).reshape(N, L, C) * s["w"] + s["b"]
    a = y if s["gate"] is None else s["gate"].float()
    act = a / (1.0 + torch.exp(-a))
    return (act if s["gate"] is None else y * act).to(s["x"].dtype)


_own = dict(chunk=_own_chunk, paged=_own_paged, token=_own_token, plan=_own_plan, norm=_own_norm)
_plain = dict(chunk=_plain_chunk, paged=_plain_paged, token=_plain_token, plan=_plain_plan,
              norm=_plain_norm)


# ------------------------------------------------------------------ work

def work(c):
    op = c["op"]
    if op == "plan":
        tokens = c["n"] * c["query"]
        return {"bytes": 8 * c["n"] + 4 * (c["n"] + 1) + 16 * tokens
                + 4 * (tokens * 0.45 // c["block"]), "flops": 0}
    if op == "norm":
        e = c["N"] * c["L"] * c["C"]
        return {"bytes": e * SIZES[c["dtype"]] * (3 if c["gate"] else 2) + 8 * c["C"],
                "flops": e * (12 if c["gate"] else 10)}
    H, HV, K, V, esz = c["H"], c["HV"], c["K"], c["V"], SIZES[c["dtype"]]
    if op == "chunk":
        rows, states = c["B"] * c["T"], 2 * c["B"]
    elif op == "paged":
        rows = c["n"] * (c["low"] + c["high"]) // 2
        states = c["n"] + rows // c["block"] + c["n"] // 2  # read, written at block ends and at the end
    else:
        rows, states = c["n"] * c["S"], 2 * c["n"]
    per_token = esz * (2 * H * K + 2 * HV * V) + (4 * HV if c["decay"] == "token" else 0)
    # the recurrence itself (decay, rank-one update, read-out) is the least arithmetic
    return {"bytes": rows * per_token + states * HV * K * V * 4, "flops": rows * HV * 5 * K * V}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _walk(q, k, v, g, state, scale, seen=None):
    """S <- e^g S + k v^T, o = scale S^T q, one token after another; q, k [n, T, H, K]."""
    n, T, H, K = q.shape
    HV = v.shape[2]
    q, k, v = q.double(), k.double(), v.double()
    q, k = (x.repeat_interleave(HV // H, 2) for x in (q, k))
    o = torch.zeros(n, T, HV, v.shape[-1], dtype=torch.float64, device=q.device)
    w = None if g is None else torch.exp(g.double()).expand(n, T, HV)
    for t in range(T):
        if w is not None:
            state = state * w[:, t, :, None, None]
        state = state + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * (q[:, t, :, None, :] @ state)[:, :, 0]
        if seen is not None:
            seen(t, state)
    return o, state


def _exact_chunk(s):
    return _walk(s["q"], s["k"], s["v"], s["g"], s["s0"].double(), s["scale"])


def _exact_paged(s):
    cu, ctx, bs = s["cu"].tolist(), s["ctx"].tolist(), s["block"]
    n, HV, V = len(ctx), s["v"].shape[2], s["v"].shape[3]
    tables = s["tables"].tolist()
    pool = s["pool"].double()
    lens = [cu[r + 1] - cu[r] for r in range(n)]
    T = max(max(lens), 1)
    dev = pool.device

    def rows(x):
        p = torch.zeros(n, T, *x.shape[2:], dtype=torch.float64, device=dev)
        for r in range(n):
            p[r, :lens[r]] = x[0, cu[r]:cu[r + 1]].double()
        return p

    s0 = torch.stack([pool[tables[r][(ctx[r] - 1) // bs]] if ctx[r] else torch.zeros_like(pool[0])
                      for r in range(n)])

    def seen(t, state):
        for r in range(n):
            end = ctx[r] + t + 1
            if t < lens[r] and (end % bs == 0 or t + 1 == lens[r]):
                pool[tables[r][(end - 1) // bs]] = state[r]

    o, _ = _walk(rows(s["q"]), rows(s["k"]), rows(s["v"]), rows(s["g"]), s0, s["scale"], seen)
    flat = torch.zeros(1, cu[-1], HV, V, dtype=torch.float64, device=dev)
    for r in range(n):
        flat[0, cu[r]:cu[r + 1]] = o[r, :lens[r]]
    return flat, pool


def _exact_token(s):
    if s["block"] == 0:
        return _walk(s["q"], s["k"], s["v"], s["g"], s["state"].double(), s["scale"])
    bs, ctx, tables, pool = s["block"], s["ctx"].tolist(), s["tables"].tolist(), s["pool"].double()
    n, S = s["q"].shape[:2]
    live = [tables[r][(ctx[r] + S - 1) // bs] >= 0 for r in range(n)]
    s0 = torch.stack([pool[tables[r][(ctx[r] - 1) // bs]] if live[r] and ctx[r]
                      else torch.zeros_like(pool[0]) for r in range(n)])

    def seen(t, state):
        for r in range(n):
            end = ctx[r] + t + 1
            if live[r] and (end % bs == 0 or t + 1 == S):
                pool[tables[r][(end - 1) // bs]] = state[r]

    o, _ = _walk(s["q"], s["k"], s["v"], s["g"], s0, s["scale"], seen)
    o[[r for r in range(n) if not live[r]]] = 0.0
    return o, pool


def _exact_plan(s):
    return None


def _exact_norm(s):
    x = s["x"].double()
    N, L, C = x.shape
    y = x.reshape(N, L, s["groups"], -1)
    var, mean = torch.var_mean(y, (1, 3), correction=0, keepdim=True)
    y = ((y - mean) / torch.sqrt(var + s["eps"])).reshape(N, L, C)
    y = y * s["w"].double() + s["b"].double()
    if s["gate"] is None:
        return y * torch.sigmoid(y)
    return y * (s["gate"].double() * torch.sigmoid(s["gate"].double()))
