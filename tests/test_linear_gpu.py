"""Linear attention with a decay for each head: the chunked form, the recurrent form and
their paged states against the recurrence itself, token by token in 64 bits.

Tolerances, from the roundings that are made (u: the type's unit roundoff, 2^-8 for bf16,
2^-11 for fp16; RMS: of the reference):
  states, fp32: every decay factor, product and sum rounds at 2^-24 relative to terms
    that add up like a random walk; with at most a few hundred terms of weight near
    one, 2^-24 * sqrt(300) * (a peak of ~6 RMS) is below 1e-5 RMS.
  o in fp32: the same, 1e-5 RMS (the read-out sums K products of such terms).
  o in bf16 / fp16: u |o| for the output's own rounding, and 12 u RMS for the operands
    that are rounded to the type on the way (scores and states, each u / sqrt(3) of
    terms that add up like a random walk: sqrt(2 / 3) u of the row's RMS, five of them
    at the peak, and rows up to three times the overall RMS).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TOL_S = 1e-5


def err(got, want):
    if want.numel() == 0:
        return 0.0
    want, got = want.double().cpu(), got.double().cpu()
    rms = want.pow(2).mean().sqrt().item()
    return (got - want).abs().max().item() / max(rms, 1e-30)


def o_ok(got, want):
    """Whether every element of o is inside the bound above."""
    if want.numel() == 0:
        return True
    if got.dtype == torch.float32:
        return err(got, want) <= 1e-5
    u, want = UNIT[got.dtype], want.double().cpu()
    rms = want.pow(2).mean().sqrt()
    return bool(((got.double().cpu() - want).abs() <= u * want.abs() + 12 * u * rms).all())


def walk(q, k, v, g, s0, scale):
    """[B, T, ..] token by token; returns o and the state after every token."""
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    q, k, v = (x.double().cpu() for x in (q, k, v))
    q, k = (x.repeat_interleave(HV // H, 2) for x in (q, k))
    s = torch.zeros(B, HV, K, V, dtype=torch.float64) if s0 is None else s0.double().cpu()
    gg = torch.zeros(B, T, HV, dtype=torch.float64) if g is None else g.double().cpu().expand(B, T, HV)
    o, after = torch.zeros(B, T, HV, V, dtype=torch.float64), []
    for t in range(T):
        s = torch.exp(gg[:, t])[..., None, None] * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * torch.einsum("bhk,bhkv->bhv", q[:, t], s)
        after.append(s)
    return o, after


def inputs(B, T, H, HV, K, V, dtype, decay, seed=0, packed=False, state=True):
    gen = torch.Generator().manual_seed(seed + 31 * T + K)
    x = torch.randn(B, T, 2 * H * K + HV * V, generator=gen).to(dtype).to(DEV)
    q, k, v = x.split([H * K, H * K, HV * V], -1)
    q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (HV, V))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    g = {"none": None, "head": -torch.rand(HV, generator=gen) * 0.1,
         "token": -torch.rand(B, T, HV, generator=gen) * torch.rand(HV, generator=gen),
         "strong": -40.0 * torch.rand(B, T, HV, generator=gen)}[decay]
    s0 = torch.randn(B, HV, K, V, generator=gen).to(DEV) if state else None
    return q, k, v, None if g is None else g.to(DEV), s0


BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32

CHUNK = [
    # B, T, H, HV, K, V, dtype, decay
    (2, 1, 2, 2, 128, 128, BF, "token"), (1, 63, 2, 2, 128, 128, BF, "token"),
    (1, 64, 1, 2, 128, 128, BF, "head"), (2, 65, 2, 2, 128, 64, BF, "none"),
    (2, 130, 2, 4, 64, 128, BF, "token"), (1, 200, 1, 1, 128, 256, BF, "strong"),
    (3, 500, 2, 6, 64, 64, BF, "token"), (1, 1000, 1, 3, 128, 128, BF, "head"),
    (1, 1500, 2, 2, 128, 256, BF, "token"), (2, 333, 1, 2, 96, 80, BF, "token"),
    (1, 257, 2, 2, 64, 64, FP16, "token"), (1, 100, 1, 2, 128, 128, FP16, "none"),
    (2, 129, 3, 3, 40, 24, FP16, "strong"), (1, 700, 2, 4, 128, 128, FP16, "token"),
    (3, 77, 2, 6, 48, 80, F32, "token"), (1, 65, 1, 1, 1, 1, F32, "token"),
    (2, 300, 1, 2, 256, 32, F32, "head"), (1, 90, 2, 2, 33, 7, F32, "none"),
    (1, 640, 1, 1, 128, 128, F32, "token"), (1, 40, 1, 1, 17, 1024, BF, "token"),
]


@pytest.mark.parametrize("B,T,H,HV,K,V,dtype,decay", CHUNK)
@pytest.mark.parametrize("packed", [False, True])
def test_chunk(gdp, B, T, H, HV, K, V, dtype, decay, packed):
    q, k, v, g, s0 = inputs(B, T, H, HV, K, V, dtype, decay, packed=packed, state=packed)
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, scale=K ** -0.5, initial_state=s0)
    ro, after = walk(q, k, v, g, s0, K ** -0.5)
    assert o.dtype == dtype and o_ok(o, ro)
    assert err(fs, after[-1]) <= TOL_S


@pytest.mark.parametrize("B,T,H,HV,K,V", [(10, 1100, 8, 16, 128, 128), (170, 700, 1, 1, 64, 64), (1, 9000, 1, 2, 128, 128)])
def test_chunk_long(gdp, B, T, H, HV, K, V):
    """Many chunks per sequence, more sequences than SMs, several items per CTA: the last
    tokens and the final states against the walk over the last stretch from the state that
    the call itself gives there, and the first tokens against the walk."""
    q, k, v, g, s0 = inputs(B, T, H, HV, K, V, BF, "token", seed=1)
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0)
    cut = T - 40  # inside a chunk
    o1, mid = gdp.gdp_linear_chunk_fwd(q[:, :cut], k[:, :cut], v[:, :cut], g[:, :cut].contiguous(), initial_state=s0)
    few = [0, B // 2, B - 1]
    ro, _ = walk(*(x[few, :70] for x in (q, k, v, g)), s0[few], K ** -0.5)
    assert o_ok(o[few, :70], ro) and o_ok(o1[few, :70], ro)
    ro, after = walk(*(x[few, cut:] for x in (q, k, v, g)), mid[few], K ** -0.5)
    assert o_ok(o[few, cut:], ro) and err(fs[few], after[-1]) <= TOL_S
    assert torch.equal(o[:, :cut - cut % 64], o1[:, :cut - cut % 64]) or o_ok(o1, o[:, :cut])


@pytest.mark.parametrize("K,V,dtype", [(128, 128, BF), (64, 64, BF), (32, 48, F32), (64, 64, FP16)])
def test_chunk_packed_sequences(gdp, K, V, dtype):
    """Empty, one-token and ragged sequences; tokens outside every sequence stay
    untouched, and a NaN in one sequence reaches no other."""
    H, HV = 2, 4
    lens = [0, 1, 70, 0, 129, 64, 300, 5]
    T = sum(lens) + 9
    q, k, v, g, _ = inputs(1, T, H, HV, K, V, dtype, "token", seed=3)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    s0 = torch.randn(len(lens), HV, K, V, generator=torch.Generator().manual_seed(9)).to(DEV)
    bad = 4  # this sequence's last token, next to the following sequence's first, is NaN
    for x in (q, k, v):
        x[0, cu[bad + 1] - 1] = float("nan")
        x[0, cu[-1]:] = float("inf")
    g[0, cu[bad + 1] - 1] = float("nan")
    g[0, cu[-1]:] = float("nan")
    o = torch.full((1, T, HV, V), 7.0, dtype=dtype, device=DEV)
    fs = torch.empty_like(s0)
    gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu.to(DEV), initial_state=s0, out=(o, fs))
    assert (o[0, cu[-1]:] == 7.0).all()
    for i, n in enumerate(lens):
        a, b = int(cu[i]), int(cu[i + 1])
        if i == bad:
            b -= 1
        ro, after = walk(q[:, a:b], k[:, a:b], v[:, a:b], g[:, a:b], s0[i:i + 1], K ** -0.5)
        assert o_ok(o[:, a:b], ro), i
        if i != bad:
            assert err(fs[i:i + 1], after[-1] if n else s0[i:i + 1]) <= TOL_S, i


@pytest.mark.parametrize("K,V,dtype", [(128, 128, BF), (64, 128, F32), (64, 64, FP16)])
def test_chunk_resets_and_zero_rows(gdp, K, V, dtype):
    """g = -inf drops the state; zero keys leave it; huge decays underflow to zero."""
    q, k, v, g, s0 = inputs(1, 200, 2, 2, K, V, dtype, "token", seed=5)
    g[0, 0, 0] = g[0, 64, 1] = g[0, 100] = float("-inf")
    g[0, 150, 0] = -1e30
    g[0, 170:180] = -90.0
    k[0, 20:40] = 0
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0)
    ro, after = walk(q, k, v, g, s0, K ** -0.5)
    assert o_ok(o, ro) and err(fs, after[-1]) <= TOL_S


@pytest.mark.parametrize("K,V,dtype", [(128, 128, BF), (32, 48, F32)])
def test_chunk_bad_offsets(gdp, K, V, dtype):
    q, k, v, g, _ = inputs(1, 100, 1, 2, K, V, dtype, "token")
    s0 = torch.randn(3, 2, K, V, device=DEV)
    for cu in ([0, 50, 40, 100], [0, 10, 20, 101], [-1, 10, 20, 30]):
        ws = torch.empty(gdp.gdp_linear_chunk_fwd_workspace_size(1, 100, 3, 1, 2, K, V, dtype),
                         dtype=torch.uint8, device=DEV)
        o = torch.full((1, 100, 2, V), 7.0, dtype=dtype, device=DEV)
        fs = torch.empty_like(s0)
        gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                                 initial_state=s0, workspace=ws, out=(o, fs))
        assert gdp.gdp_read_status(ws) == 1
        assert (o == 7.0).all() and torch.equal(fs, s0)


def paged_case(lens, ctx, bs, HV, K, V, seed=0):
    """Block tables over a pool of random pages, every block up to the last token paged."""
    gen = torch.Generator().manual_seed(seed)
    used = [-(-(c + n) // bs) for c, n in zip(ctx, lens)]
    width = max(max(used), 1)
    perm = torch.randperm(sum(used) + 3, generator=gen).tolist()
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    for r, u in enumerate(used):
        for j in range(u):
            tables[r, j] = perm.pop()
    pool = torch.randn(sum(used) + 3, HV, K, V, generator=gen)
    return tables, pool


def paged_reference(q, k, v, g, cu, ctx, tables, pool, bs, scale):
    want, o = pool.double().clone(), torch.zeros(v.shape, dtype=torch.float64)
    for r in range(len(ctx)):
        a, b = cu[r], cu[r + 1]
        if a == b:
            continue
        s0 = pool[tables[r, (ctx[r] - 1) // bs]][None] if ctx[r] else None
        o[:, a:b], after = walk(q[:, a:b], k[:, a:b], v[:, a:b], g[:, a:b], s0, scale)
        for t, s in enumerate(after):
            end = ctx[r] + t + 1
            if end % bs == 0 or t == b - a - 1:
                want[tables[r, (end - 1) // bs]] = s[0]
    return o, want


@pytest.mark.parametrize("K,V,dtype,bs", [(128, 128, BF, 64), (128, 128, BF, 128), (64, 64, BF, 128),
                                          (48, 32, F32, 64), (64, 64, FP16, 192)])
def test_chunk_paged(gdp, K, V, dtype, bs):
    H, HV = 1, 2
    lens = [1, 0, 64, 200, 130, 63, 300, 7]
    ctx = [0, 5, 64, 1, bs, bs - 1, 70, 3 * bs]
    cu = [0] + torch.tensor(lens).cumsum(0).tolist()
    q, k, v, g, _ = inputs(1, cu[-1], H, HV, K, V, dtype, "token", seed=11)
    tables, pool = paged_case(lens, ctx, bs, HV, K, V)
    ro, want = paged_reference(q, k, v, g, cu, ctx, tables, pool, bs, K ** -0.5)
    got = pool.to(DEV)
    o = gdp.gdp_linear_chunk_fwd_paged(q, k, v, g, torch.tensor(cu, dtype=torch.int32, device=DEV), got,
                                       tables.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), bs)
    assert o_ok(o, ro)
    assert err(got, want) <= TOL_S
    touched = {int(tables[r, (ctx[r] + t) // bs]) for r in range(len(lens)) for t in range(lens[r])}
    for pg in range(pool.shape[0]):
        if pg not in touched:
            assert torch.equal(got[pg].cpu(), pool[pg])


def test_chunk_paged_bad_tables(gdp):
    """A sequence with a page outside the pool, or a negative context, is skipped alone."""
    K = V = 128
    lens, ctx, bs, HV = [100, 100, 100, 100], [0, 64, 5, 0], 64, 2
    cu = torch.tensor([0, 100, 200, 300, 400], dtype=torch.int32)
    q, k, v, g, _ = inputs(1, 400, 2, HV, K, V, BF, "token")
    tables, pool = paged_case(lens, ctx, bs, HV, K, V)
    ctx[2] = -1
    tables[1, 2] = pool.shape[0]
    tables[3, 1] = -1
    got, o = pool.to(DEV), torch.full((1, 400, HV, V), 7.0, dtype=BF, device=DEV)
    ws = torch.empty(gdp.gdp_linear_chunk_fwd_workspace_size(1, 400, 4, 2, HV, K, V, BF),
                     dtype=torch.uint8, device=DEV)
    gdp.gdp_linear_chunk_fwd_paged(q, k, v, g, cu.to(DEV), got, tables.to(DEV),
                                   torch.tensor(ctx, dtype=torch.int32, device=DEV), bs, workspace=ws, out=o)
    assert gdp.gdp_read_status(ws) == 1
    assert (o[0, 100:] == 7.0).all()
    ro, after = walk(q[:, :100], k[:, :100], v[:, :100], g[:, :100], None, K ** -0.5)
    assert o_ok(o[:, :100], ro)
    want = pool.double()
    want[tables[0, 0]], want[tables[0, 1]] = after[63][0], after[99][0]
    assert err(got, want) <= TOL_S


TOKEN = [
    # n, S, H, HV, K, V, dtype, decay
    (1, 1, 2, 2, 128, 128, BF, "token"), (5, 1, 2, 4, 64, 64, FP16, "head"),
    (3, 4, 1, 3, 128, 256, BF, "token"), (2, 16, 2, 2, 48, 80, F32, "none"),
    (40, 1, 4, 8, 128, 128, BF, "token"), (2, 2, 1, 1, 256, 32, F32, "strong"),
    (3, 3, 2, 2, 33, 7, F32, "token"), (2, 1, 1, 2, 1, 1, FP16, "token"),
    (2, 5, 1, 1, 200, 9, BF, "token"), (300, 1, 1, 2, 32, 16, F32, "token"),
]


@pytest.mark.parametrize("n,S,H,HV,K,V,dtype,decay", TOKEN)
def test_recurrent(gdp, n, S, H, HV, K, V, dtype, decay):
    q, k, v, g, s0 = inputs(n, S, H, HV, K, V, dtype, decay, packed=True)
    ro, after = walk(q, k, v, g, s0, 0.3)
    o = gdp.gdp_linear_recurrent_update(q, k, v, g, s0, scale=0.3)
    assert o.dtype == dtype and o_ok(o, ro)
    assert err(s0, after[-1]) <= TOL_S


@pytest.mark.parametrize("bs,S", [(1, 1), (1, 4), (16, 1), (16, 5), (256, 2)])
def test_recurrent_paged(gdp, bs, S):
    H, HV, K, V, n = 1, 2, 128, 64, 9
    gen = torch.Generator().manual_seed(bs + S)
    ctx = torch.randint(0, 5 * bs, (n,), generator=gen).tolist()
    ctx[0], ctx[1] = 0, bs
    tables, pool = paged_case([S] * n, ctx, bs, HV, K, V)
    pad = 3
    tables[pad] = -1
    q, k, v, g, _ = inputs(n, S, H, HV, K, V, BF, "token", seed=2)
    want, ro = pool.double().clone(), torch.zeros(v.shape, dtype=torch.float64)
    for r in range(n):
        if r == pad:
            continue
        s0 = pool[tables[r, (ctx[r] - 1) // bs]][None] if ctx[r] else None
        ro[r:r + 1], after = walk(q[r:r + 1], k[r:r + 1], v[r:r + 1], g[r:r + 1], s0, K ** -0.5)
        for t, s in enumerate(after):
            end = ctx[r] + t + 1
            if end % bs == 0 or t == S - 1:
                want[tables[r, (end - 1) // bs]] = s[0]
    got, status = pool.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    o = gdp.gdp_linear_recurrent_update_paged(q, k, v, g, got, tables.to(DEV),
                                              torch.tensor(ctx, dtype=torch.int32, device=DEV), bs,
                                              status=status)
    assert int(status) == 0 and (o[pad] == 0).all()
    assert o_ok(o, ro) and err(got, want) <= TOL_S


def test_recurrent_paged_refuses_clashes(gdp):
    """Requests that write one page, write a page that another reads, or name a page outside the
    pool are skipped like padding; two requests that only read one page are not."""
    HV, K, V, bs = 2, 64, 64, 4
    #            writes 0 twice | reads+writes 2 | reads 2, writes 3 | both read 4, write 5, 6 | outside
    tables = torch.tensor([[0, -1], [0, -1], [2, -1], [2, 3], [4, 5], [4, 6], [99, -1], [7, -1]],
                          dtype=torch.int32)
    ctx = [1, 2, 3, 4, 4, 4, 0, -2]
    n = len(ctx)
    pool = torch.randn(8, HV, K, V)
    q, k, v, g, _ = inputs(n, 1, 1, HV, K, V, F32, "token")
    got, status = pool.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    o = gdp.gdp_linear_recurrent_update_paged(q, k, v, g, got, tables.to(DEV),
                                              torch.tensor(ctx, dtype=torch.int32, device=DEV), bs,
                                              status=status)
    assert int(status) == 1
    want = pool.double().clone()
    for r in range(n):
        if r in (0, 1, 2, 6, 7):
            assert (o[r] == 0).all(), r
            continue
        ro, after = walk(q[r:r + 1], k[r:r + 1], v[r:r + 1], g[r:r + 1],
                         pool[tables[r, (ctx[r] - 1) // bs]][None], K ** -0.5)
        assert o_ok(o[r:r + 1], ro)
        want[tables[r, ctx[r] // bs]] = after[0][0]
    assert err(got, want) <= TOL_S


def test_chunk_then_recurrent_continue_one_stream(gdp):
    """A prompt through the chunked form and tokens through the recurrent form, states in
    pages, give the one walk."""
    K = V = 128
    H, HV, bs, T, S = 2, 4, 64, 190, 6
    q, k, v, g, _ = inputs(1, T + S, H, HV, K, V, BF, "token", seed=8)
    tables = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device=DEV)
    pool = torch.full((4, HV, K, V), float("nan"), device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    o = [gdp.gdp_linear_chunk_fwd_paged(q[:, :T], k[:, :T], v[:, :T], g[:, :T].contiguous(),
                                        torch.tensor([0, T], **i32), pool, tables,
                                        torch.zeros(1, **i32), bs)]
    for t in range(T, T + S):
        o.append(gdp.gdp_linear_recurrent_update_paged(
            q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], g[:, t:t + 1].contiguous(), pool, tables,
            torch.tensor([t], **i32), bs))
    ro, after = walk(q, k, v, g, None, K ** -0.5)
    assert o_ok(torch.cat(o, 1), ro)
    for b, page in enumerate(tables[0].tolist()):
        assert err(pool[page], after[min((b + 1) * bs, T + S) - 1][0]) <= TOL_S


def test_side_stream(gdp):
    q, k, v, g, s0 = inputs(1, 300, 2, 2, 128, 128, BF, "token")
    ref, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        o, f2 = gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0)
    st.synchronize()
    assert torch.equal(o, ref) and torch.equal(fs, f2)


def test_binding_refuses(gdp):
    q, k, v, g, s0 = inputs(1, 8, 2, 4, 32, 32, BF, "token")
    ok = dict(initial_state=s0)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q.cpu(), k, v, g, **ok)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q, k[:, :4], v, g, **ok)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q, k, v.float(), g, **ok)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q, k, v, g.half(), **ok)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q, k, v, g[:, :4], **ok)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q.transpose(2, 3), k.transpose(2, 3), v, g, **ok)
    with pytest.raises(ValueError):
        gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0.half())
    with pytest.raises(ValueError):
        gdp.gdp_linear_recurrent_update(q, k, v, g, s0[:, :2])
    with pytest.raises(gdp.GDPError):  # three value heads over two key heads
        gdp.gdp_linear_chunk_fwd(q, k, v[:, :, :3], g[..., :3].contiguous())
    with pytest.raises(gdp.GDPError):  # too many tokens for a decode step
        gdp.gdp_linear_recurrent_update(*(x.repeat(1, 4, 1, 1) for x in (q, k, v)), None, s0)
    with pytest.raises(gdp.GDPError):  # block size not a multiple of the chunk
        i32 = dict(dtype=torch.int32, device=DEV)
        gdp.gdp_linear_chunk_fwd_paged(q, k, v, g, torch.tensor([0, 8], **i32), s0,
                                       torch.zeros(1, 1, **i32), torch.zeros(1, **i32), 48)
