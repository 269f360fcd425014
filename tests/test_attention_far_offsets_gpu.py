"""Rotation, append and paged attention where elements lie more than 2^31 apart: pools of more than 2^32 bytes and
rows of more than 2^31 elements. Tolerances are test_attention_gpu's and test_rotary_gpu's."""
import pytest
import torch

import test_rotary_gpu
from test_attention_gpu import BF, DEV, FP, check, problem, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    yield
    torch.cuda.empty_cache()


# pages of 16 by TMA, of 12 by cp.async; heads off the grid of 8 and fp32 by the kernel for any size
@pytest.mark.parametrize("dtype,block,D", [(BF, 16, 64), (BF, 12, 64), (BF, 16, 60), (FP, 16, 64)])
def test_pools(gdp, dtype, block, D):
    lens, ctx, HKV = [3, 1, 40], [500, 64, 1300], 4
    d = problem(lens, ctx, 8, HKV, D, D, block, dtype)
    small, pages = d["k_cache"].shape[0], (1 << 31) // (block * HKV * D) + 200
    far = [pages - small, pages // 2]              # the pages' new places: the last ones, and half of them in the middle
    to = torch.arange(small, device=DEV) // 2 + torch.tensor(far, device=DEV)[torch.arange(small, device=DEV) % 2]
    for name in ("k_cache", "v_cache"):
        pool = torch.empty(pages, block, HKV, D, device=DEV, dtype=dtype)
        pool[to] = d[name]
        d[name] = pool
    t = d["block_tables"]
    d["block_tables"] = torch.where(t >= 0, to[t.clamp(min=0).long()].int(), -1)
    assert int(d["block_tables"].max()) * d["k_cache"].stride(0) > 1 << 31
    check(gdp, d)
    # new tokens appended to the last page: those that attention reads
    r = 2
    p = torch.arange(ctx[r], ctx[r] + lens[r], device=DEV)
    page, at = d["block_tables"][r, p // block].long(), p % block
    k, v = (torch.randn(lens[r], HKV, D, device=DEV, generator=torch.Generator(DEV).manual_seed(s)).to(dtype) for s in (1, 2))
    gdp.gdp_cache_append(k, v, d["k_cache"], d["v_cache"], page * block + at)
    assert torch.equal(d["k_cache"][page, at], k) and torch.equal(d["v_cache"][page, at], v)
    check(gdp, d)


def test_rows(gdp):
    """Queries of more than 2^31 elements, turned in place and attended from their end."""
    T, H, D = 270000, 64, 128
    x = torch.empty(T, H, D, device=DEV, dtype=BF)
    rows = torch.tensor([0, 1, 131071, 131072, 262143, 262144, T - 1], device=DEV)
    x[rows] = torch.randn(rows.numel(), H, D, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(BF)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f, _ = gdp.gdp_rotary_frequencies(D)
    want = test_rotary_gpu.turned(x[rows], pos[rows], f, 1.0, 0, False)
    gdp.gdp_rotary(x, pos, f, out=x)
    test_rotary_gpu.check(x[rows], want)
    # a request whose tokens are the last ones, after one without keys that has all the others
    d = problem([0, 5], [0, 70], H, 8, D, D, 16, BF)
    x[-5:] = torch.randn(5, H, D, device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(BF)
    i32 = dict(dtype=torch.int32, device=DEV)
    out = torch.empty(1, T, H, D, device=DEV, dtype=BF)
    gdp.gdp_attention_paged(**dict(d, q=x[None], cu_seqlens=torch.tensor([0, T - 5, T], **i32)), out=out)
    o, tol = reference(**dict(d, q=x[None, -5:], cu_seqlens=torch.tensor([0, 0, 5], **i32)))
    assert bool(((out[0, -5:].double() - o).abs() <= tol).all())
    assert float(out[0, ::30000].abs().max()) == 0
