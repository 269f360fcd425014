"""Cases and plain forms of the operators of attention layers over a paged cache.

Models that keep linear-attention states in most layers keep keys and values in the others, so
these three stand beside the block plan, whose positions and slots they take: the position rotation
of heads ("rotary"), appending keys and values to a paged cache with the rotation on the way
("append"), and attention of new tokens, single ones, trees of drafted ones or pieces of prompts,
over that cache ("attend"). ``run`` makes the library's calls where ``own`` is true and computes the
same in elementary torch operations, in 32 bits (angles in 64), where it is false; ``exact`` computes
it from the definitions in 64 bits, one request after another.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one token's query heads: the latency of a call
        dict(name="rotary_one", op="rotary", T=1, H=16, D=128, R=128, offset=0, inter=False, scaling="none",
             far=5000, backward=False, dtype="bf16", fused=False),
        # the query heads of a prefill step, views of a fused projection
        dict(name="rotary_prompt", op="rotary", T=8192, H=32, D=128, R=128, offset=0, inter=False, scaling="none",
             far=8192, backward=False, dtype="bf16", fused=True),
        # the gradient's pass at odd sizes: neighbours as pairs, part of the head, far positions
        dict(name="rotary_far", op="rotary", T=1001, H=6, D=80, R=48, offset=16, inter=True, scaling="ramp",
             far=1 << 20, backward=True, dtype="fp32", fused=False),
        # a decode step's new keys and values, some entries padding, its queries rotated in the same call
        dict(name="append_step", op="append", n=256, low=1, high=1, context=8192, H=32, HKV=8, D=128, DV=128, R=128,
             inter=False, scaling="none", block=256, dtype="bf16", fused=True, pad=0.06),
        # ragged prompts of a prefill step
        dict(name="append_prompts", op="append", n=16, low=64, high=1024, context=2048, H=32, HKV=8, D=128, DV=128,
             R=128, inter=False, scaling="wavelength", block=64, dtype="bf16", fused=True, pad=0.0),
        # odd sizes in full precision, no queries, half of the head rotated
        dict(name="append_odd", op="append", n=7, low=1, high=90, context=500, H=0, HKV=3, D=72, DV=40, R=36,
             inter=True, scaling="linear", block=24, dtype="fp32", fused=False, pad=0.0),
        # one request decoding at a short context: the latency of a single token
        dict(name="token_one", op="attend", n=1, low=1, high=1, tree=False, least=300, most=300, H=16, HKV=4, D=128,
             DV=128, block=64, dtype="bf16", pad=0.0),
        # a full decode batch, contexts of up to 8192 tokens, some entries padding
        dict(name="token_batch", op="attend", n=256, low=1, high=1, tree=False, least=64, most=8192, H=32, HKV=8,
             D=128, DV=128, block=256, dtype="bf16", pad=0.06),
        # trees of drafted tokens of a verification step, ragged
        dict(name="tree_batch", op="attend", n=16, low=16, high=64, tree=True, least=1024, most=8192, H=32, HKV=8,
             D=128, DV=128, block=64, dtype="bf16", pad=0.0),
        # a few drafted tokens of one request after a long document, small pages
        dict(name="tree_long", op="attend", n=1, low=8, high=8, tree=True, least=131000, most=131000, H=16, HKV=2,
             D=64, DV=64, block=16, dtype="fp16", pad=0.0),
        # pieces of prompts that continue cached prefixes: the largest
        dict(name="prompt_pieces", op="attend", n=8, low=256, high=1024, tree=False, least=0, most=4096, H=16, HKV=4,
             D=128, DV=128, block=128, dtype="bf16", pad=0.0),
        # full precision at odd sizes, three query heads a key head
        dict(name="tree_odd", op="attend", n=5, low=1, high=13, tree=True, least=0, most=2000, H=6, HKV=2, D=80,
             DV=48, block=24, dtype="fp32", pad=0.2),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    HKV = rng.choice([1, 2, 3, 4, 8])
    H = HKV * rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([32, 48, 64, 64, 72, 80, 96, 128, 128, 128, 128, 256])
    scaling = rng.choice(["none", "none", "linear", "ramp", "wavelength"])
    if op == "rotary":
        R = 2 * rng.randint(1, D // 2) if rng.random() < 0.4 else D
        return dict(op=op, T=_log(rng, 1, max(2, (1 << 25) // (H * D))), H=H, D=D, R=R,
                    offset=rng.choice([0, 0, D - R]), inter=rng.random() < 0.5, scaling=scaling,
                    far=_log(rng, 16, 1 << 21), backward=rng.random() < 0.3, dtype=dtype, fused=rng.random() < 0.5)
    DV = D if rng.random() < 0.7 else rng.choice([32, 40, 64, 128])
    block = rng.choice([1, 8, 16, 24, 32, 64, 128, 256])
    context = _log(rng, 16, 8192)
    if op == "append":
        high = rng.choice([1, 1, 5, 64, 512, 1024])
        n = _log(rng, 1, max(2, min(512, (1 << 23) // (high * HKV * D), (1 << 26) // ((context + high) * HKV * D))))
        return dict(op=op, n=n, low=rng.choice([0, 1]) if high > 1 else 1, high=high, context=context,
                    H=H if rng.random() < 0.7 else 0, HKV=HKV, D=D, DV=DV,
                    R=2 * rng.randint(1, D // 2) if rng.random() < 0.4 else D, inter=rng.random() < 0.5,
                    scaling=scaling, block=block, dtype=dtype, fused=rng.random() < 0.5,
                    pad=rng.choice([0.0, 0.1]))
    kind = rng.choice(["token", "token", "tree", "tree", "piece"])
    high = 1 if kind == "token" else rng.randint(2, 64) if kind == "tree" else _log(rng, 3, 700)
    most = _log(rng, 1, 65536 if kind != "piece" else 4096)
    room = min(256, (1 << 28) // ((most + high) * HKV * (D + DV)), (1 << 27) // ((most + high) * H * high),
               (1 << 34) // ((most + high) * H * high * (D + DV)))
    return dict(op=op, n=_log(rng, 1, max(2, room)), low=1 if high == 1 else rng.randint(0, high), high=high,
                tree=kind == "tree", least=rng.choice([0, most // 2, most]), most=most, H=H, HKV=HKV, D=D, DV=DV,
                block=block, dtype=dtype, pad=rng.choice([0.0, 0.0, 0.1]))


# ------------------------------------------------------------------ inputs

def _frequencies(R, scaling):
    """Angles per position of the R / 2 pairs, fp64, and the amplitude: base 10000, or scaled from
    an original length of 4096 by 8 (linear: all; ramp: from the pairs that turn 32 times within
    the length to those that turn once, amplitude 1 + 0.1 ln 8; wavelength: from wavelengths of a
    quarter of the length to the whole)."""
    i = torch.arange(R // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / R)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling == "ramp":
        at = [R * math.log(4096.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(10000.0)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        t = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - t) + f / 8.0 * t, 0.1 * math.log(8.0) + 1.0
    t = ((4096.0 * f / (2.0 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
    return f * t + f / 8.0 * (1.0 - t), 1.0


def _heads(gen, T, sizes, dtype, fused):
    """Tensors [T, H, D] of N(0, 1) for each (H, D) of `sizes`: views of one projection, or apart."""
    dt = DTYPES[dtype]
    if not fused:
        return [torch.randn(T, H, D, generator=gen, device="cuda").to(dt) for H, D in sizes]
    x = torch.randn(T, sum(H * D for H, D in sizes), generator=gen, device="cuda").to(dt)
    return [y.unflatten(-1, s) for y, s in zip(x.split([H * D for H, D in sizes], dim=-1), sizes)]


def _lengths(n, low, high, least, most):
    """Host-side lengths of the requests' new tokens and of their contexts, the same for every seed."""
    gen = torch.Generator().manual_seed(n * 7919 + high * 31 + most)
    lens = torch.randint(low, high + 1, (n,), generator=gen)
    lens[0] = high
    ctx = torch.randint(least, most + 1, (n,), generator=gen)
    ctx[0] = most
    return lens, ctx


def _tables(gen, used, pad):
    """Block tables with used[r] pages of their own in row r, in random order, -1 past them; rows of
    -1 alone for padding requests. Returns the tables on the device and the number of pages."""
    total, width = int(used.sum()), max(1, int(used.max()))
    pages = torch.randperm(total, generator=gen).to(torch.int32)
    first = torch.cumsum(used, 0) - used
    j = torch.arange(width)
    at = (first[:, None] + j).clamp_(max=max(total - 1, 0))
    tables = torch.where(j < used[:, None], pages[at] if total else -1, -1)
    tables[torch.rand(used.numel(), generator=gen) < pad] = -1
    return tables.to(torch.int32).contiguous().cuda(), max(total, 1)


def _cache(gen, pages, block, H, D, dtype):
    x = torch.empty(pages, block, H, D, dtype=DTYPES[dtype], device="cuda")
    return x.normal_(generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, seed, gen)


def _prepare_rotary(c, seed, gen):
    f, amplitude = _frequencies(c["R"], c["scaling"])
    D = [(c["H"], c["D"])] * (3 if c["fused"] else 1)
    pos = torch.randint(0, c["far"], (c["T"],), generator=gen, device="cuda", dtype=torch.int32)
    return dict(op="rotary", x=_heads(gen, c["T"], D, c["dtype"], c["fused"])[0], pos=pos, f=f.cuda(),
                amplitude=amplitude, offset=c["offset"], inter=c["inter"], backward=c["backward"])


def _prepare_append(c, seed, gen):
    lens, ctx = _lengths(c["n"], c["low"], c["high"], 0, c["context"])
    host = torch.Generator().manual_seed(seed * 7 + 1)
    bs = c["block"]
    tables, pages = _tables(host, (ctx + lens + bs - 1) // bs, c["pad"])
    T = int(lens.sum())
    q, k, v = _heads(gen, T, [(c["H"], c["D"]), (c["HKV"], c["D"]), (c["HKV"], c["DV"])], c["dtype"], c["fused"])
    # as the block plan gives them: each token's position and slot, -1 where there is no page
    req = torch.repeat_interleave(torch.arange(c["n"]), lens)
    pos = ctx[req] + torch.arange(T) - (torch.cumsum(lens, 0) - lens)[req]
    page = tables[req.cuda(), (pos // bs).cuda()].long()
    slot = torch.where(page >= 0, page * bs + (pos % bs).cuda(), -1)
    f, amplitude = _frequencies(c["R"], c["scaling"])
    return dict(op="append", q=q if c["H"] else None, k=k, v=v, pos=pos.to(torch.int32).cuda(), slot=slot, f=f.cuda(),
                amplitude=amplitude, inter=c["inter"], kc=_cache(gen, pages, bs, c["HKV"], c["D"], c["dtype"]),
                vc=_cache(gen, pages, bs, c["HKV"], c["DV"], c["dtype"]))


def _trees(host, n, S):
    """Ancestors' bits [n, S] of random trees: a token's parent is one of the eight before it, or
    the context; every token sees itself."""
    bits = torch.zeros(n, S + 1, dtype=torch.int64)  # the last column: no parent
    for i in range(S):
        parent = torch.randint(max(-1, i - 8), i, (n,), generator=host)
        bits[:, i] = bits[torch.arange(n), parent] | (1 << i if i < 63 else -1 << 63)
    return bits[:, :S]


def _prepare_attend(c, seed, gen):
    lens, ctx = _lengths(c["n"], c["low"], c["high"], c["least"], c["most"])
    host = torch.Generator().manual_seed(seed * 7 + 2)
    bs = c["block"]
    tables, pages = _tables(host, (ctx + lens + bs - 1) // bs, c["pad"])
    T = int(lens.sum())
    # queries twice as long as keys: scores of standard deviation 2
    q = (2.0 * torch.randn(1, T, c["H"], c["D"], generator=gen, device="cuda")).to(DTYPES[c["dtype"]])
    cu = torch.zeros(c["n"] + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(lens, 0)
    tree = None
    if c["tree"]:
        bits = _trees(host, c["n"], c["high"])
        tree = bits[torch.arange(c["high"])[None] < lens[:, None]][None].cuda()
    return dict(op="attend", q=q, kc=_cache(gen, pages, bs, c["HKV"], c["D"], c["dtype"]),
                vc=_cache(gen, pages, bs, c["HKV"], c["DV"], c["dtype"]), tables=tables, tree=tree,
                ctx=ctx.to(torch.int32).cuda(), cu=cu.to(torch.int32).cuda(), scale=c["D"] ** -0.5,
                most_tokens=int(lens.max()), most_keys=int((ctx + lens).max()))


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_rotary(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    return gdp.gdp_rotary(s["x"], s["pos"], s["f"], offset=s["offset"], interleaved=s["inter"],
                          amplitude=s["amplitude"], backward=s["backward"])


def _own_append(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    q = gdp.gdp_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["slot"], positions=s["pos"], frequencies=s["f"],
                             interleaved=s["inter"], amplitude=s["amplitude"], q=s["q"])
    return [x for x in (q, s["kc"], s["vc"]) if x is not None]


def _own_attend(s):
    import linear_attention_ssm_gdp_gb300 as gdp
    return gdp.gdp_attention_paged(s["q"], s["kc"], s["vc"], s["tables"], s["ctx"], cu_seqlens=s["cu"],
                                   tree_mask=s["tree"], scale=s["scale"])


def _rotate(x, pos, f, amplitude, offset, inter, backward):
    """x [T, H, D] in 32 bits with the pairs of [offset, offset + R) turned; angles in 64 bits."""
    angle = pos.double()[:, None] * f * (-1.0 if backward else 1.0)
    c = (amplitude * torch.cos(angle)).float()[:, None]
    s = (amplitude * torch.sin(angle)).float()[:, None]
    y = x.float().clone()
    part = y[..., offset:offset + 2 * f.numel()]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else part.chunk(2, dim=-1)
    turned = a * c - b * s, a * s + b * c
    part.copy_(torch.stack(turned, -1).flatten(-2) if inter else torch.cat(turned, -1))
    return y


def _plain_rotary(s):
    y = _rotate(s["x"], s["pos"], s["f"], s["amplitude"], s["offset"], s["inter"], s["backward"])
    return y.to(s["x"].dtype)


def _plain_append(s):
    turn = (s["pos"], s["f"], s["amplitude"], 0, s["inter"], False)
    keep = s["slot"] >= 0
    slot = s["slot"][keep]
    s["kc"].flatten(0, 1)[slot] = _rotate(s["k"], *turn).to(s["k"].dtype)[keep]
    s["vc"].flatten(0, 1)[slot] = s["v"][keep]
    q = [] if s["q"] is None else [_rotate(s["q"], *turn).to(s["q"].dtype)]
    return q + [s["kc"], s["vc"]]


def _plain_attend(s):
    q, ctx, cu, bs = s["q"][0], s["ctx"].long(), s["cu"].long(), s["kc"].shape[1]
    T, H, D = q.shape
    HKV, S, L = s["kc"].shape[2], s["most_tokens"], s["most_keys"]
    n, dev = ctx.numel(), q.device
    lens = cu[1:] - cu[:-1]
    # each request in a row of its own
    i, j = torch.arange(S, device=dev)[None], torch.arange(L, device=dev)[None]
    token = torch.where(i < lens[:, None], cu[:-1, None] + i, T)
    rows = torch.cat([q.float(), torch.zeros_like(q[:1]).float()])[token]           # [n, S, H, D]
    page = s["tables"].long().gather(1, (j // bs).expand(n, L).clamp(max=s["tables"].shape[1] - 1))
    there = (j < (ctx + lens)[:, None]) & (page >= 0)
    page = torch.where(there, page, 0)
    k = s["kc"][page, j % bs].float().permute(0, 2, 3, 1)                           # [n, HKV, D, L]
    v = torch.where(there[..., None, None], s["vc"][page, j % bs], 0.0).float().permute(0, 2, 1, 3)
    sees = j[:, None] <= (ctx[:, None] + i)[..., None]                              # [n, S, L]
    if s["tree"] is not None:
        bits = torch.cat([s["tree"][0], torch.zeros_like(s["tree"][0, :1])])[token]  # [n, S]
        back = j - ctx[:, None]                                                     # [n, L]
        own_bit = (bits[..., None] >> back.clamp(0, 63)[:, None]) & 1
        sees = torch.where(back[:, None] < 0, True, (own_bit == 1) & (back[:, None] < 64))
    sees = sees & there[:, None]
    rows = rows.unflatten(2, (HKV, H // HKV)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n, HKV, S G, D]
    x = (rows @ k) * s["scale"]
    x = torch.where(sees.repeat_interleave(H // HKV, 1)[:, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0.0, 1.0, total)
    o = o.unflatten(2, (S, H // HKV)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [n, S, H, DV]
    out = torch.zeros(T + 1, H, o.shape[-1], device=dev)
    out[token] = o
    return out[None, :T].to(s["q"].dtype)


_own = dict(rotary=_own_rotary, append=_own_append, attend=_own_attend)
_plain = dict(rotary=_plain_rotary, append=_plain_append, attend=_plain_attend)


# ------------------------------------------------------------------ work

def work(c):
    esz = SIZES[c["dtype"]]
    if c["op"] == "rotary":
        e = c["T"] * c["H"]
        return {"bytes": 2 * e * c["D"] * esz + 4 * c["T"] + 4 * c["R"], "flops": 3 * e * c["R"]}
    if c["op"] == "append":
        lens, _ = _lengths(c["n"], c["low"], c["high"], 0, c["context"])
        T = int(lens.sum())
        kept = T * (1.0 - c["pad"])
        return {"bytes": int(2 * T * c["H"] * c["D"] * esz + 2 * kept * c["HKV"] * (c["D"] + c["DV"]) * esz + 12 * T
                             + 4 * c["R"]),
                "flops": int(3 * T * c["R"] * (c["H"] + c["HKV"]))}
    lens, ctx = _lengths(c["n"], c["low"], c["high"], c["least"], c["most"])
    keep = 1.0 - c["pad"]
    T, keys = int(lens.sum()), int(torch.where(lens > 0, ctx + lens, 0).sum()) * keep
    # what the tokens see: the context, and of the new tokens half (a chain), or a few (a tree: itself at least)
    pairs = float((lens * ctx).sum() + (lens if c["tree"] else lens * (lens + 1) // 2).sum()) * keep
    return {"bytes": int(keys * c["HKV"] * (c["D"] + c["DV"]) * esz + T * c["H"] * (c["D"] + c["DV"]) * esz
                         + 4 * keys / c["block"] + 8 * c["n"] + (8 * T if c["tree"] else 0)),
            "flops": int(2 * pairs * c["H"] * (c["D"] + c["DV"]))}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _turned(x, pos, f, amplitude, offset, inter, sign):
    """Each pair as a complex number times amplitude e^(i pos f), in 64 bits."""
    y = x.double().clone()
    m = f.numel()
    first = offset + torch.arange(m, device=x.device) * (2 if inter else 1)
    second = first + (1 if inter else m)
    z = torch.complex(y[..., first], y[..., second])
    angle = sign * pos.double()[:, None, None] * f
    z = z * torch.polar(torch.full_like(angle, amplitude), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotary(s):
    return _turned(s["x"], s["pos"], s["f"], s["amplitude"], s["offset"], s["inter"], -1.0 if s["backward"] else 1.0)


def _exact_append(s):
    turn = (s["pos"], s["f"], s["amplitude"], 0, s["inter"], 1.0)
    bs, slot = s["kc"].shape[1], s["slot"]
    kc, vc = s["kc"].double(), s["vc"].double()
    t = torch.nonzero(slot >= 0)[:, 0]
    kc[slot[t] // bs, slot[t] % bs] = _turned(s["k"], *turn)[t]
    vc[slot[t] // bs, slot[t] % bs] = s["v"][t].double()
    return ([] if s["q"] is None else [_turned(s["q"], *turn)]) + [kc, vc]


def _exact_attend(s):
    q, cu, ctx, tables = s["q"][0], s["cu"].tolist(), s["ctx"].tolist(), s["tables"]
    bs, HKV, DV = s["kc"].shape[1], s["kc"].shape[2], s["vc"].shape[3]
    T, H, _ = q.shape
    out = torch.zeros(1, T, H, DV, dtype=torch.float64, device=q.device)
    for r in range(len(ctx)):
        a, b = cu[r], cu[r + 1]
        at = torch.arange(ctx[r] + b - a, device=q.device)
        page = tables[r, at // bs].long()
        if a == b or not bool((page >= 0).any()):
            continue
        at, page = at[page >= 0], page[page >= 0]
        k, v = s["kc"][page, at % bs].double(), s["vc"][page, at % bs].double()
        back = at - ctx[r]
        i = torch.arange(b - a, device=q.device)
        sees = back[None] <= i[:, None]
        if s["tree"] is not None:
            sees = (back < 0) | ((s["tree"][0, a:b, None] >> back.clamp(0, 63)) & 1 == 1)
        for h in range(H):
            x = (q[a:b, h].double() @ k[:, h // (H // HKV)].T) * s["scale"]
            p = torch.softmax(x.masked_fill(~sees, -math.inf), -1).nan_to_num(0.0)
            out[0, a:b, h] = p @ v[:, h // (H // HKV)]
    return out
