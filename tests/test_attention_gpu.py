"""Attention over a paged cache against its formula in 64 bits.

Tolerances, per element of o, with A = sum p |v| / sum p and n the keys of the longest request:
  the output's rounding             u |ref|, u = 2^-8 (bf16), 2^-11 (fp16), 2^-24 (fp32)
  weights rounded to a 16-bit type  u A (none for fp32)
  a score's error e changes its weight by a factor 1 + e, top and bottom: 2 max_j e_j A, with
    e_j = (D + 4) 2^-24 scale sum_d |q_d k_jd| (a sum of D products in any order, each addition
    rounded or, on the tensor cores, cut off at 2^-23 once per 16 products, and the scale's product)
  2^x by the hardware               2^-22 each, top and bottom: 2^-20 A with the factors of joins
  sums of n weights                 (80 + n / 16) 2^-23 A
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF: 2.0 ** -8, HF: 2.0 ** -11, FP: 2.0 ** -24}


def make_cache(gen, pages, block, H, D, dtype, kind):
    if kind == "heads":
        return torch.randn(pages, H, block, D, generator=gen, device=DEV).to(dtype).transpose(1, 2)
    if kind == "pair":
        return torch.randn(pages, 2, block, H, D, generator=gen, device=DEV).to(dtype)[:, 1]
    if kind == "odd":                              # rows off the 16-byte grid
        return torch.randn(pages, block, H, D + 1, generator=gen, device=DEV).to(dtype)[..., 1:]
    return torch.randn(pages, block, H, D, generator=gen, device=DEV).to(dtype)


def problem(lens, ctx, H, HKV, D, DV, block, dtype, layout="plain", tree=False, seed=0, packed=True, loud=2.0,
            holes=()):
    """Inputs of one call. holes: (request, block) pairs whose table entries are -1."""
    gen = torch.Generator(device=DEV).manual_seed(seed + 13 * D + len(lens))
    host = torch.Generator().manual_seed(seed)
    n, T = len(lens), sum(lens)
    used = [-(-(c + s) // block) for c, s in zip(ctx, lens)]
    pages = max(sum(used), 1) + 2
    perm = torch.randperm(pages, generator=host).tolist()
    tables = torch.full((n, max(max(used), 1) + 1), -1, dtype=torch.int32)
    for r in range(n):
        for b in range(used[r]):
            tables[r, b] = perm.pop()
    for r, b in holes:
        tables[r, b] = -1
    x = (loud * torch.randn(1, T, H + 2, D, generator=gen, device=DEV)).to(dtype)
    q = x[:, :, 1:-1] if layout != "plain" else x[:, :, 1:-1].contiguous()
    mask = None
    if tree:
        rows = []
        for s in lens:
            bits = []
            for i in range(s):
                parent = int(torch.randint(max(-1, i - 4), i, (1,), generator=host)) if i else -1
                b = (bits[parent] if parent >= 0 else 0) | 1 << i
                bits.append(b)
            rows += bits
        mask = torch.tensor([b - (1 << 64) if b >= 1 << 63 else b for b in rows], dtype=torch.int64, device=DEV)[None]
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)
    d = dict(q=q, k_cache=make_cache(gen, pages, block, HKV, D, dtype, layout),
             v_cache=make_cache(gen, pages, block, HKV, DV, dtype, layout), block_tables=tables.to(DEV),
             context_lens=torch.tensor(ctx, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV), tree_mask=mask)
    if not packed:
        d["q"] = q.reshape(n, lens[0], H, D)
        d["cu_seqlens"] = None
        d["tree_mask"] = None if mask is None else mask.view(n, lens[0])
    return d


def reference(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, tree_mask, scale=None):
    """(o, tolerance) [T, H, DV] in fp64."""
    dt, D = q.dtype, q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    n = context_lens.numel()
    cu = cu_seqlens.tolist() if cu_seqlens is not None else [r * q.shape[1] for r in range(n + 1)]
    q = q.flatten(0, 1)
    T, H = q.shape[:2]
    block, HKV, DV = k_cache.shape[1], k_cache.shape[2], v_cache.shape[3]
    mask = None if tree_mask is None else tree_mask.flatten()
    o = torch.zeros(T, H, DV, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    u = UNIT[dt]
    for r in range(n):
        a, b, c = cu[r], cu[r + 1], int(context_lens[r])
        if a == b:
            continue
        at = torch.arange(c + b - a, device=DEV)
        page = block_tables[r][at // block].long()
        at, page = at[page >= 0], page[page >= 0]
        i, back = torch.arange(b - a, device=DEV)[:, None], at[None] - c
        sees = back <= i
        if mask is not None:
            sees = (back < 0) | ((mask[a:b, None] >> back.clamp(0, 63)) & 1 == 1)
        if at.numel() == 0:
            continue
        for h in range(H):
            g = h // (H // HKV)
            k, v = k_cache[page, at % block, g].double(), v_cache[page, at % block, g].double()
            x = (q[a:b, h].double() @ k.T * scale).masked_fill(~sees, -torch.inf)
            p = torch.softmax(x, -1).nan_to_num(0.0)
            size = abs(scale) * (q[a:b, h].double().abs() @ k.abs().T).masked_fill(~sees, 0.0).amax(-1, keepdim=True)
            A = p @ v.abs()
            e = (D + 4) * 2.0 ** -24 * size
            o[a:b, h] = p @ v
            tol[a:b, h] = u * o[a:b, h].abs() + A * ((u if dt != FP else 0.0) + 2 * e + 2.0 ** -20
                                                     + (80 + at.numel() / 16) * 2.0 ** -23)
    return o, tol


def check(gdp, d, scale=None, status=0):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = gdp.gdp_attention_paged(**d, scale=scale, status=st)
    assert int(st) == status
    o, tol = reference(**d, scale=scale)
    bad = (got.flatten(0, 1).double() - o).abs() - tol
    assert bool((bad <= 0).all()), (float(bad.max()), int((bad > 0).sum()), bad.numel())
    return got


SIZES = [
    # lens, ctx, H, HKV, D, DV, block, layout
    ([1], [0], 1, 1, 64, 64, 16, "plain"),
    ([1], [299], 16, 4, 128, 128, 64, "plain"),
    ([1, 0, 3, 1, 64], [127, 50, 128, 0, 255], 8, 2, 128, 128, 16, "pair"),
    ([1] * 40, list(range(0, 800, 20)), 8, 8, 64, 64, 32, "heads"),
    ([5, 1, 33], [1000, 64, 3], 6, 2, 80, 48, 24, "plain"),          # pages that end inside a tile
    ([2, 9], [700, 31], 4, 4, 96, 128, 8, "heads"),
    ([2, 9], [70, 31], 4, 4, 128, 64, 1, "plain"),                   # a page a token
    ([7], [400], 32, 1, 128, 128, 128, "plain"),                     # 224 rows a key head
    ([64, 13], [900, 2000], 16, 2, 128, 128, 256, "pair"),           # two tiles of rows and more
    ([3, 2], [90, 210], 3, 1, 33, 17, 10, "plain"),                  # odd sizes
    ([3, 2], [90, 210], 3, 1, 64, 64, 16, "odd"),                    # rows off the 16-byte grid
    ([4, 2], [300, 210], 2, 2, 256, 256, 64, "plain"),
    ([1, 1], [1500, 2], 4, 4, 256, 200, 16, "heads"),
]


@pytest.mark.parametrize("lens,ctx,H,HKV,D,DV,block,layout", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("tree", [False, True])
def test_attention(gdp, lens, ctx, H, HKV, D, DV, block, layout, dtype, tree):
    check(gdp, problem(lens, ctx, H, HKV, D, DV, block, dtype, layout, tree))


@pytest.mark.parametrize("D,DV", [(100, 36), (50, 250), (33, 64), (64, 33), (4, 2), (1, 1), (255, 256)])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("layout", ["plain", "pair", "odd"])
def test_rows_of_any_width(gdp, D, DV, dtype, layout):
    """Rows that are whole copies of 16, 8 or 4 bytes, or none, on grids of as many; NaN in the slots not in use."""
    d = problem([1, 6, 2], [130, 31, 0], 6, 2, D, DV, 12, dtype, layout, tree=True)
    used = d["block_tables"][d["block_tables"] >= 0].long()
    for name in ("k_cache", "v_cache"):
        free = torch.ones(d[name].shape[0], dtype=torch.bool, device=DEV)
        free[used] = False
        d[name][free] = float("nan")
    check(gdp, d)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_prompts(gdp, dtype):
    """Pieces of prompts: a chain longer than 64 tokens, more rows than a tile."""
    check(gdp, problem([300, 0, 129, 1], [0, 5, 700, 33], 4, 2, 64, 64, 16, dtype))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_long_context(gdp, dtype):
    """One request over all CTAs: every piece of an item joins."""
    check(gdp, problem([3], [20011], 4, 2, 64, 64, 64, dtype, tree=True))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("tree", [False, True])
def test_dense_batch(gdp, dtype, tree):
    check(gdp, problem([4] * 6, [10, 0, 300, 7, 129, 64], 8, 2, 128, 128, 32, dtype, tree=tree, packed=False))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_scales(gdp, dtype, scale):
    check(gdp, problem([3, 1], [200, 77], 4, 2, 64, 64, 16, dtype, loud=0.5), scale=scale)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_blocks_that_are_not_there(gdp, dtype):
    """Holes in a context, a padding request, a request with none of its blocks but the last."""
    d = problem([2, 1, 3, 1], [300, 64, 200, 31], 4, 2, 128, 128, 16, dtype,
                holes=[(0, 0), (0, 7), (0, 8), (0, 9), (0, 10), (0, 11), (0, 12), (0, 13), (0, 14), (0, 15), (0, 16)]
                + [(1, b) for b in range(5)] + [(2, b) for b in range(12)])
    got = check(gdp, d)
    assert float(got[0, 2].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_that_see_nothing(gdp, dtype):
    d = problem([3, 2], [0, 40], 4, 2, 64, 64, 16, dtype, tree=True)
    d["tree_mask"][0, 1] = 0
    d["tree_mask"][0, 4] = 0                       # sees the context only
    got = check(gdp, d)
    assert float(got[0, 1].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_what_is_not_the_requests_is_not_read(gdp, dtype):
    """NaN in unused pages, behind the last token, and in the slots of absent blocks."""
    d = problem([2, 1], [133, 64], 4, 2, 128, 128, 16, dtype, holes=[(0, 3)])
    want = gdp.gdp_attention_paged(**d)
    for c in (d["k_cache"], d["v_cache"]):
        used = torch.zeros(c.shape[:2], dtype=torch.bool, device=DEV)
        for r, L in enumerate((135, 65)):
            for p in range(L):
                page = int(d["block_tables"][r, p // 16])
                if page >= 0:
                    used[page, p % 16] = True
        c[~used] = torch.nan
    got = gdp.gdp_attention_paged(**d)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_values_that_are_not_finite_stay_with_their_request(gdp, dtype):
    d = problem([2, 2, 1], [40, 100, 30], 4, 2, 64, 64, 16, dtype)
    want = gdp.gdp_attention_paged(**d)
    page = int(d["block_tables"][1, 2])
    d["v_cache"][page, 5] = torch.inf
    d["k_cache"][page, 6] = torch.nan
    got = gdp.gdp_attention_paged(**d)
    assert torch.equal(got[:, :2], want[:, :2]) and torch.equal(got[:, 4:], want[:, 4:])
    assert not bool(torch.isfinite(got[:, 2:4]).any())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_refused_on_the_device(gdp, dtype):
    d = problem([2, 1, 3], [40, 30, 20], 4, 2, 64, 64, 16, dtype)
    want = gdp.gdp_attention_paged(**d)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = dict(d, context_lens=torch.tensor([40, -1, 20], dtype=torch.int32, device=DEV))
    got = gdp.gdp_attention_paged(**bad, status=st)          # a negative context
    assert int(st) == 1 and float(got[0, 2].abs().max()) == 0
    assert torch.equal(got[0, :2], want[0, :2]) and torch.equal(got[0, 3:], want[0, 3:])
    for c in (10 ** 6, 2 ** 31 - 1):                          # a table too short for it
        st.zero_()
        bad = dict(d, context_lens=torch.tensor([40, 30, c], dtype=torch.int32, device=DEV))
        got = gdp.gdp_attention_paged(**bad, status=st)
        assert int(st) == 1 and float(got[0, 3:].abs().max()) == 0 and torch.equal(got[0, :3], want[0, :3])
    for page in (d["k_cache"].shape[0], 2 ** 31 - 1):         # a page outside the pool: as if not there
        st.zero_()
        t = d["block_tables"].clone()
        t[1, 0] = page
        got = gdp.gdp_attention_paged(**dict(d, block_tables=t), status=st)
        t[1, 0] = -1
        assert int(st) == 1 and torch.equal(got, gdp.gdp_attention_paged(**dict(d, block_tables=t)))
    out = torch.full_like(want, 7.0)
    for cu in ([0, 2, 1, 6], [1, 2, 3, 6], [0, 2, 3, 7], [0, -1, 3, 6]):  # bad offsets: o is left alone
        st.zero_()
        gdp.gdp_attention_paged(**dict(d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV)), status=st,
                                out=out)
        assert int(st) == 1 and bool((out == 7.0).all())
    long = problem([65, 2], [3, 4], 2, 2, 64, 64, 16, dtype)  # a tree has at most 64 tokens
    long["tree_mask"] = torch.full((1, 67), -1, dtype=torch.int64, device=DEV)
    st.zero_()
    got = gdp.gdp_attention_paged(**long, status=st)
    assert int(st) == 1 and float(got[0, :65].abs().max()) == 0 and float(got[0, 65:].abs().max()) > 0


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_past_the_last_request_stay(gdp, dtype):
    d = problem([2, 3], [40, 30], 4, 2, 64, 64, 16, dtype)
    want = gdp.gdp_attention_paged(**d)
    more = dict(d, q=torch.cat([d["q"], torch.full_like(d["q"][:, :3], torch.nan)], 1))
    out = torch.full((1, 8, 4, 64), 5.0, device=DEV, dtype=dtype)
    gdp.gdp_attention_paged(**more, out=out)
    assert torch.equal(out[:, :5], want) and bool((out[:, 5:] == 5.0).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_captured_replayed_and_on_another_stream(gdp, dtype):
    d = problem([1] * 5, [10, 200, 3, 64, 127], 8, 2, 128, 128, 16, dtype)
    d["block_tables"] = torch.where(d["block_tables"] < 0, 0, d["block_tables"])
    out = torch.empty(1, 5, 8, 128, device=DEV, dtype=dtype)
    need = gdp.gdp_attention_paged_workspace_size(1, 5, 5, 8, 2, 128, 128, dtype)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gdp.gdp_attention_paged(**d, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    first = out.clone()
    assert torch.equal(first, gdp.gdp_attention_paged(**d))
    graphs = []
    for _ in range(2):                             # two graphs that share the workspace, one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdp.gdp_attention_paged(**d, out=out, workspace=ws)
        graphs.append(g)
    for step in range(3):
        d["context_lens"].add_(1)
        out.zero_()
        ws.fill_(255)                              # nothing in the workspace is kept between calls
        graphs[step % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gdp.gdp_attention_paged(**d))
        o, tol = reference(**d)
        assert bool(((out.flatten(0, 1).double() - o).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_the_same_bits_twice(gdp, dtype):
    d = problem([4, 1, 9], [3000, 100, 7], 8, 2, 128, 128, 64, dtype, tree=True)
    a = gdp.gdp_attention_paged(**d)
    for _ in range(3):
        assert torch.equal(a, gdp.gdp_attention_paged(**d))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_requests(gdp, dtype):
    """More requests than threads, most of them without tokens."""
    lens = [1 if r % 7 == 0 else 0 for r in range(3000)]
    ctx = [r % 50 for r in range(3000)]
    check(gdp, problem(lens, ctx, 2, 1, 64, 64, 16, dtype))


def test_empty_calls(gdp):
    kc = torch.zeros(4, 16, 2, 64, device=DEV, dtype=BF)
    i32 = dict(dtype=torch.int32, device=DEV)
    o = gdp.gdp_attention_paged(torch.zeros(1, 0, 4, 64, device=DEV, dtype=BF), kc, kc, torch.zeros(2, 3, **i32),
                                torch.zeros(2, **i32), cu_seqlens=torch.zeros(3, **i32))
    assert o.shape == (1, 0, 4, 64)
    o = gdp.gdp_attention_paged(torch.zeros(0, 1, 4, 64, device=DEV, dtype=BF), kc, kc, torch.zeros(0, 3, **i32),
                                torch.zeros(0, **i32))
    assert o.shape == (0, 1, 4, 64)
    # tables without blocks, a cache without pages: rows that see nothing
    st = torch.zeros(1, **i32)
    o = gdp.gdp_attention_paged(torch.ones(2, 1, 4, 64, device=DEV, dtype=BF), kc[:0], kc[:0], torch.zeros(2, 0, **i32),
                                torch.zeros(2, **i32), status=st)
    assert int(st) == 1 and float(o.abs().max()) == 0


def test_step_of_a_server(gdp):
    """Plan, append and attention together, a tree verified and its accepted path appended again."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    i32 = dict(dtype=torch.int32, device=DEV)
    n, H, HKV, D, block = 3, 8, 2, 64, 16
    free, used = torch.randperm(40, generator=gen, device=DEV).to(torch.int32), torch.zeros(1, **i32)
    tables, ctx = torch.full((n, 8), -1, **i32), torch.zeros(n, **i32)
    kc, vc = (torch.full((40, block, HKV, D), torch.nan, device=DEV, dtype=BF) for _ in range(2))
    f, _ = gdp.gdp_rotary_frequencies(D)
    keys, values = [[] for _ in range(n)], [[] for _ in range(n)]

    def step(lens, mask=None, depth=None, keep=None):
        nonlocal used
        T = sum(lens)
        q, k, v = (torch.randn(1, T, h, D, generator=gen, device=DEV).to(BF) for h in (H, HKV, HKV))
        query = torch.tensor(lens, **i32)
        cu, req, pos, slot, used = gdp.gdp_block_plan(ctx, query, tables, free, used, block, T)
        at = pos if depth is None else ctx[req.long()] + depth
        q = gdp.gdp_cache_append(k, v, kc, vc, slot[None], positions=at[None], frequencies=f, q=q)
        o = gdp.gdp_attention_paged(q, kc, vc, tables, ctx, cu_seqlens=cu, tree_mask=mask)
        turned = gdp.gdp_rotary(k, at[None], f)
        r0 = cu.tolist()
        for r in range(n):
            kk = torch.stack(keys[r] + list(turned[0, r0[r]:r0[r + 1]])).double()
            vv = torch.stack(values[r] + list(v[0, r0[r]:r0[r + 1]])).double()
            for i in range(lens[r]):
                c = len(keys[r])
                see = [j for j in range(lens[r]) if (mask is None and j <= i)
                       or (mask is not None and int(mask[0, r0[r] + i]) >> j & 1)]
                idx = list(range(c)) + [c + j for j in see]
                for h in range(H):
                    p = torch.softmax(kk[idx, h // 4] @ q[0, r0[r] + i, h].double() * D ** -0.5, 0)
                    want = p @ vv[idx, h // 4]
                    A = p @ vv[idx, h // 4].abs()
                    tol = UNIT[BF] * (want.abs() + A) + 1e-4 * A  # the terms of reference(), at these sizes
                    assert bool(((o[0, r0[r] + i, h].double() - want).abs() <= tol).all())
        path = [list(range(m)) for m in lens] if keep is None else keep
        if keep is not None:  # the accepted tokens move to the front
            first = ctx[req.long()].long()
            place = torch.full((T,), -1, dtype=torch.int64, device=DEV)
            for r in range(n):
                for d, i in enumerate(path[r]):
                    p = int(first[r0[r] + i]) + d
                    place[r0[r] + i] = int(tables[r, p // block]) * block + p % block
            gdp.gdp_cache_append(k, v, kc, vc, place[None], positions=at[None], frequencies=f)
        for r in range(n):
            for i in path[r]:
                keys[r].append(turned[0, r0[r] + i])
                values[r].append(v[0, r0[r] + i])
        ctx.add_(torch.tensor([len(p) for p in path], **i32))

    step([37, 5, 16])
    step([1, 1, 1])
    bits = [0b1, 0b11, 0b101, 0b1011]
    step([4, 4, 4], torch.tensor([bits * 3], device=DEV), torch.tensor([0, 1, 1, 2] * 3, **i32),
         [[0, 2], [0, 1, 3], [0]])
    step([1, 1, 1])


@pytest.mark.parametrize("lens,ctx", [([1] * 96, list(range(40, 4840, 50))), ([64, 33, 64, 50], [3000, 700, 64, 2000]),
                                      ([500, 260], [100, 900])])
def test_many_pieces_many_times(gdp, lens, ctx):
    """Many pieces on every CTA, launched back to back and from idle with cold caches: the same bits."""
    d = problem(lens, ctx, 32, 8, 128, 128, 64, BF)
    want = gdp.gdp_attention_paged(**d)
    flush = torch.empty(400 << 20, dtype=torch.uint8, device=DEV)
    got = []
    for i in range(30):
        if i % 3 == 1:
            flush.zero_()
        if i % 5 == 1:
            torch.cuda.synchronize()
        got.append(gdp.gdp_attention_paged(**d))
    assert all(torch.equal(x, want) for x in got)
    check(gdp, d)


@pytest.mark.parametrize("block", [1, 3, 12, 100, 520])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,DV", [(64, 64), (128, 96)])
def test_block_sizes(gdp, block, dtype, D, DV):
    """Pages that are not whole boxes: other loads than for multiples of 8, holes among them."""
    d = problem([3, 1, 40, 0, 2], [500, 64, 1300, 9, 31], 8, 2, D, DV, block, dtype,
                holes=[(0, 0), (2, 1)] if block > 1 else [(0, 7), (0, 64), (2, 1000)])
    check(gdp, d)
    dead = dict(d, k_cache=d["k_cache"].clone(), v_cache=d["v_cache"].clone())
    last = int(d["block_tables"][0, 502 // block])  # NaN behind the request's last token
    for c in (dead["k_cache"], dead["v_cache"]):
        c[last, 502 % block + 1:] = torch.nan
    assert torch.equal(gdp.gdp_attention_paged(**dead), gdp.gdp_attention_paged(**d))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,DV", [(256, 256), (136, 64), (64, 192), (192, 128)])
@pytest.mark.parametrize("block,tree", [(64, False), (8, True), (5, True)])
def test_heads_above_128(gdp, dtype, D, DV, block, tree):
    """One slot of 128 rows: more rows than that, one token, holes, rows behind the last token."""
    d = problem([50, 1, 3, 64], [900, 2000, 31, 0], 8, 2, D, DV, block, dtype, tree=tree, holes=[(0, 1), (1, 3)])
    check(gdp, d)
    for c in (d["k_cache"], d["v_cache"]):
        c[int(d["block_tables"][1, 2000 // block]), 2000 % block + 1:] = torch.nan
    check(gdp, d)


def test_heads_above_128_many_times(gdp):
    d = problem([40, 1, 64, 7] * 8, [2000, 900, 64, 3000] * 8, 8, 2, 256, 256, 64, BF)
    want = gdp.gdp_attention_paged(**d)
    flush = torch.empty(400 << 20, dtype=torch.uint8, device=DEV)
    got = []
    for i in range(30):
        if i % 3 == 1:
            flush.zero_()
        if i % 5 == 1:
            torch.cuda.synchronize()
        got.append(gdp.gdp_attention_paged(**d))
    assert all(torch.equal(x, want) for x in got)
    check(gdp, d)


@pytest.mark.parametrize("D,DV,layout", [(197, 197, "plain"), (207, 207, "heads"), (238, 150, "plain"), (256, 143, "pair"),
                                         (160, 238, "plain"), (256, 136, "odd"), (129, 129, "odd"), (1, 256, "plain")])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_sizes_with_the_most_shared_memory(gdp, D, DV, layout, dtype):
    """As many stages as fit: what a size takes does not grow with it."""
    check(gdp, problem([1, 0, 9], [90, 7, 31], 6, 2, D, DV, 24, dtype, layout))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("far", [14.3, 18.7, 20.6])
def test_many_small_weights(gdp, far, dtype):
    """One key of weight 1 and value 0, thousands of weights near 2^-far, all the same, so that their roundings do not
    average out: weights this far below the largest keep their type's full precision. (Many requests of the same pages: a
    CTA has whole ones.)"""
    n, D = 8192, 64
    d = problem([1], [n - 1], 1, 1, D, D, 64, dtype)
    for name in ("q", "k_cache", "v_cache"):
        d[name].zero_()
    d["q"][0, 0, 0, 0] = 1.0
    first = int(d["block_tables"][0, 0])
    d["k_cache"][first, 0, 0, 0] = far * 0.6931471806
    d["v_cache"].fill_(1.0)
    d["v_cache"][first, 0] = 0.0
    R = 320
    d.update(q=d["q"].expand(1, R, 1, D), block_tables=d["block_tables"].expand(R, -1).contiguous(),
             context_lens=d["context_lens"].expand(R).contiguous(),
             cu_seqlens=torch.arange(R + 1, dtype=torch.int32, device=DEV))
    check(gdp, d, scale=1.0)


def test_another_current_device_is_refused(gdp, monkeypatch):
    d = problem([2, 3], [40, 7], 4, 2, 64, 64, 16, BF)
    k, v = d["q"][0, :, :2].contiguous(), d["q"][0, :, 2:4].contiguous()
    slot = torch.full((5,), -1, dtype=torch.int64, device=DEV)
    pos = torch.zeros(5, dtype=torch.int32, device=DEV)
    f = torch.ones(32, dtype=torch.float64, device=DEV)
    monkeypatch.setattr(gdp, "_current_device", lambda: 1)
    for call in (lambda: gdp.gdp_attention_paged(**d), lambda: gdp.gdp_rotary(k, pos, f),
                 lambda: gdp.gdp_cache_append(k, v, d["k_cache"], d["v_cache"], slot)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
