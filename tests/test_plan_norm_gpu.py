"""The block plan against a plain walk over the requests (integers, exact) and the group norm
against its formula in 64 bits.

Group norm tolerances: the fp32 sums, the two-pass variance and the exponential leave a few
2^-23 of the value; with values up to ~8 RMS(ref), 1e-5 RMS(ref). A 16-bit output adds its
own rounding, u |ref| with u = 2^-8 (bf16) or 2^-11 (fp16).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}


def plan_reference(ctx, qry, tables, free, used, bs, N):
    n, width = tables.shape
    tables, status, out = tables.clone(), 0, []
    cu, req, pos, slot, full = [0], [], [], [], False
    for r in range(n):
        c, m = ctx[r], qry[r]
        have, need = -(-c // bs), -(-(c + m) // bs) - -(-c // bs)
        if c < 0 or m < 0 or c + m > width * bs:
            status |= 1
            m = need = 0
        if full or (need and used + need > len(free)) or len(req) + m > N:
            full, m, need = True, 0, 0
            status |= 2
        for j in range(need):
            tables[r, have + j] = free[used + j]
        used += need
        for p in range(c, c + m):
            pg = int(tables[r, p // bs])
            req.append(r)
            pos.append(p)
            slot.append(pg * bs + p % bs if pg >= 0 else -1)
        cu.append(len(req))
    fill = [-1] * (N - len(req))
    return cu, req + fill, pos + fill, slot + fill, used, tables, status


def run_plan(gdp, ctx, qry, tables, free, used, bs, N):
    i32 = dict(dtype=torch.int32, device=DEV)
    t, status = tables.to(DEV), torch.full((1,), 77, **i32)
    cu, req, pos, slot, u = gdp.gdp_block_plan(torch.tensor(ctx, **i32), torch.tensor(qry, **i32), t,
                                               torch.tensor(free, **i32), torch.tensor([used], **i32),
                                               bs, N, status=status)
    return cu.tolist(), req.tolist(), pos.tolist(), slot.tolist(), int(u), t.cpu(), int(status)


def check_plan(gdp, *a):
    got, want = run_plan(gdp, *a), plan_reference(*a)
    assert got[:5] == want[:5] and got[6] == want[6]
    assert torch.equal(got[5], want[5])


@pytest.mark.parametrize("n,bs,context,query,spare", [
    (1, 16, 0, 1, 5), (1, 1, 10, 7, 20), (3, 16, 100, 1, 9), (40, 24, 500, 64, 400),
    (256, 64, 8192, 1, 300), (600, 16, 64, 3, 900), (33, 128, 4000, 700, 400), (2000, 16, 50, 2, 3000),
    (5, 64, 1, 5000, 1000),
])
def test_plan(gdp, n, bs, context, query, spare):
    gen = torch.Generator().manual_seed(n + bs)
    ctx = torch.randint(0, context + 1, (n,), generator=gen).tolist()
    qry = torch.randint(0, query + 1, (n,), generator=gen).tolist()
    width = -(-(context + query) // bs)
    tables = torch.randint(0, 1 << 20, (n, width), generator=gen, dtype=torch.int32)
    free = torch.randperm(spare, generator=gen).tolist()
    check_plan(gdp, ctx, qry, tables, free, 2, bs, n * query + 3)


def test_plan_runs_out_of_pages_and_tokens(gdp):
    t = torch.arange(80, dtype=torch.int32).reshape(4, 20)
    check_plan(gdp, [3, 16, 40, 0], [20, 1, 30, 5], t, list(range(100, 104)), 1, 16, 200)  # pages
    check_plan(gdp, [3, 16, 40, 0], [20, 1, 30, 5], t, list(range(100, 140)), 0, 16, 40)   # tokens
    check_plan(gdp, [3, 16, 40, 0], [20, 0, 0, 0], t, [], 0, 16, 8)
    check_plan(gdp, [3, 17, 40, 1], [1, 1, 1, 1], t, [], 0, 16, 8)      # no new page needed


def test_plan_invalid_requests_are_empty(gdp):
    t = torch.arange(80, dtype=torch.int32).reshape(4, 20)
    t[1, 0] = -1  # a token whose block has no page
    check_plan(gdp, [-1, 4, 300, 2**31 - 1], [5, 2, 30, 2**31 - 1], t, list(range(100, 140)), 0, 16, 64)
    check_plan(gdp, [0, 4, 310, 0], [-5, 2, 10, 320], t, list(range(100, 140)), 0, 16, 400)


def test_plan_empty(gdp):
    check_plan(gdp, [], [], torch.empty(0, 4, dtype=torch.int32), [1, 2], 1, 16, 4)
    check_plan(gdp, [3], [0], torch.zeros(1, 4, dtype=torch.int32), [1, 2], 1, 16, 0)


def test_plan_refuses(gdp):
    i32 = dict(dtype=torch.int32, device=DEV)
    l1, t, f, u = torch.zeros(2, **i32), torch.zeros(2, 4, **i32), torch.zeros(3, **i32), torch.zeros(1, **i32)
    with pytest.raises(ValueError):
        gdp.gdp_block_plan(l1.long(), l1, t, f, u, 16, 8)
    with pytest.raises(ValueError):
        gdp.gdp_block_plan(l1, l1[:1], t, f, u, 16, 8)
    with pytest.raises(ValueError):
        gdp.gdp_block_plan(l1, l1, t.cpu(), f, u, 16, 8)
    with pytest.raises(gdp.GDPError):
        gdp.gdp_block_plan(l1, l1, t, f, u, 0, 8)
    with pytest.raises(gdp.GDPError):
        gdp.gdp_block_plan(l1, l1, t, f, u, 1 << 30, 8)


def norm_reference(x, G, w, b, gate, eps, act):
    x = x.double().cpu()
    N, L, C = x.shape
    y = x.reshape(N, L, G, C // G)
    var, mean = torch.var_mean(y, (1, 3), correction=0, keepdim=True)
    z = ((y - mean) / torch.sqrt(var + eps)).reshape(N, L, C)
    z = z * (1 if w is None else w.double().cpu()) + (0 if b is None else b.double().cpu())
    u = z if gate is None else gate.double().cpu()
    a = u * torch.sigmoid(u) if act == "silu" else u
    return a if gate is None else z * a


def check_norm(gdp, N, L, C, G, dt, out, gate, act="silu", affine=True, strided=False, offset=0.0):
    gen = torch.Generator().manual_seed(N + L + C)
    wide = C + 16 if strided else C
    x = (torch.randn(N, L, wide, generator=gen) * 2 + offset).to(dt).to(DEV)[..., wide - C:]
    gt = torch.randn(N, L, wide, generator=gen).to(out).to(DEV)[..., :C] if gate else None
    w = (1 + 0.1 * torch.randn(C, generator=gen)).to(DEV) if affine else None
    b = (0.1 * torch.randn(C, generator=gen)).to(DEV) if affine else None
    y = gdp.gdp_group_norm(x, G, w, b, gate=gt, activation=act, out_dtype=out)
    ref = norm_reference(x, G, w, b, gt, 1e-5, act)
    rms = ref.pow(2).mean().sqrt().item()
    assert y.dtype == out
    assert ((y.double().cpu() - ref).abs() <= UNIT[out] * ref.abs() + 1e-5 * rms).all()


BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("N,L,C,G,dt,out", [
    (1, 1, 4096, 32, BF, BF), (77, 1, 2048, 16, BF, BF), (300, 1, 512, 8, F32, BF), (5, 1, 80, 1, F32, F32),
    (9, 1, 320, 32, FP16, FP16), (3, 1, 21, 7, F32, F32), (2, 1, 5, 5, F32, F32), (4, 1, 16384, 1, BF, BF),
    (7, 1, 1200, 2, F32, FP16), (130, 1, 64, 8, BF, BF), (2, 1, 40000, 1, F32, F32), (3, 1, 6000, 3, FP16, FP16),
    (2, 4096, 320, 32, FP16, FP16), (1, 1000, 64, 4, BF, BF), (3, 7, 24, 8, F32, F32), (2, 50, 21, 3, F32, BF),
    (1, 5000, 8, 1, F32, F32), (4, 33, 3200, 2, BF, BF), (2, 300, 2002, 2, FP16, FP16), (1, 20000, 96, 3, BF, BF),
    (1, 2, 130, 130, F32, F32), (20, 64, 128, 16, F32, FP16), (1, 3, 17, 1, BF, BF), (1, 700, 4000, 2, F32, F32),
])
@pytest.mark.parametrize("gate", [False, True])
def test_group_norm(gdp, N, L, C, G, dt, out, gate):
    check_norm(gdp, N, L, C, G, dt, out, gate)


@pytest.mark.parametrize("L", [1, 40])
def test_group_norm_variants(gdp, L):
    check_norm(gdp, 6, L, 256, 4, BF, BF, True, act="none")
    check_norm(gdp, 6, L, 256, 4, F32, F32, False, act="none", affine=False)
    check_norm(gdp, 6, L, 256, 4, F32, F32, True, strided=True)
    check_norm(gdp, 6, L, 256, 4, BF, BF, True, strided=True, affine=False)


def test_group_norm_large_offset(gdp):
    """A mean 1000 times the spread: the two-pass variance keeps its digits. The inputs' own
    ulp at 1000 is 6e-5, which is the data's, the same on both sides; (x - mean) is exact to an
    ulp of the mean, 6e-5 / 2 of a spread of 2: the tolerance is 1e-4."""
    for N, L in ((9, 1), (2, 500)):
        gen = torch.Generator().manual_seed(3)
        x = (torch.randn(N, L, 96, generator=gen) * 2 + 1000.0).to(DEV)
        y = gdp.gdp_group_norm(x, 3, activation="none")
        ref = norm_reference(x, 3, None, None, None, 1e-5, "none")
        assert (y.double().cpu() - ref).abs().max().item() <= 1e-4


def test_group_norm_constant_rows_and_two_dims(gdp):
    x = torch.full((4, 64), 3.0, device=DEV)
    b = torch.randn(64, device=DEV)
    assert torch.equal(gdp.gdp_group_norm(x, 4, None, b, activation="none"), b.expand(4, 64))
    y = torch.randn(4, 64, device=DEV)
    assert torch.equal(gdp.gdp_group_norm(y, 4), gdp.gdp_group_norm(y[:, None], 4)[:, 0])
    assert gdp.gdp_group_norm(y[:0], 4).shape == (0, 64)


def test_group_norm_refuses(gdp):
    x = torch.randn(4, 2, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    for kw in (dict(weight=w.half()), dict(weight=w[:32]), dict(gate=x[:2]), dict(gate=x.half()),
               dict(activation="tanh"), dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            gdp.gdp_group_norm(x, 4, **kw)
    with pytest.raises(ValueError):
        gdp.gdp_group_norm(x.transpose(1, 2), 4)
    with pytest.raises(gdp.GDPError):
        gdp.gdp_group_norm(x, 5)
    with pytest.raises(gdp.GDPError):
        gdp.gdp_group_norm(x.half(), 4, out_dtype=torch.float32)
    with pytest.raises(gdp.GDPError):
        gdp.gdp_group_norm(x, 4, eps=-1.0)
