"""Paged prompts around the lengths at which sequences are cut into segments: contexts off the chunk
grid, the page that the first segment starts from written by the last one, whole blocks kept on the
way. Against the walk in 64 bits, with the tolerances of the other linear-attention tests."""
import pytest
import torch

from test_linear_gpu import BF, DEV, F32, FP16, TOL_S, err, inputs, o_ok, paged_case, paged_reference

pytestmark = pytest.mark.gpu


def check(gdp, lens, ctx, bs, H, HV, K, V, dtype, seed=0):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v, g, _ = inputs(1, cu[-1], H, HV, K, V, dtype, "token", seed=seed)
    g = g * 0.05  # states last over the segments
    tables, pool = paged_case(lens, ctx, bs, HV, K, V, seed=seed)
    ro, want = paged_reference(q, k, v, g, cu, ctx, tables, pool, bs, K ** -0.5)
    got = pool.to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    o = gdp.gdp_linear_chunk_fwd_paged(q, k, v, g, torch.tensor(cu, **i32), got, tables.to(DEV), torch.tensor(ctx, **i32),
                                       bs)
    assert o_ok(o, ro)
    assert err(got, want) <= TOL_S
    touched = {int(tables[r, (ctx[r] + t) // bs]) for r in range(len(lens)) for t in range(lens[r])}
    for pg in range(pool.shape[0]):
        if pg not in touched:
            assert torch.equal(got[pg].cpu(), pool[pg])


@pytest.mark.parametrize("K,V,dtype", [(64, 128, BF), (48, 32, F32), (64, 64, FP16)])
@pytest.mark.parametrize("T,ctx", [(449, 63), (450, 63), (500, 50), (511, 1), (512, 0), (512, 63), (513, 63)])
def test_one_prompt_near_a_segment(gdp, K, V, dtype, T, ctx):
    check(gdp, [T], [ctx], 128, 1, 1, K, V, dtype)


@pytest.mark.parametrize("K,V,dtype", [(64, 128, BF), (48, 32, F32), (64, 64, FP16)])
@pytest.mark.parametrize("bs", [64, 192, 4096])
def test_cut_prompts(gdp, K, V, dtype, bs):
    """Segments of 512 positions: two sequences in several of them, among ones in one or none."""
    check(gdp, [1100, 3, 0, 577, 480], [37, 64, 5, 100, 63], bs, 1, 2, K, V, dtype)


def test_cut_at_a_larger_share(gdp):
    """As many heads as SMs: segments are as long as an SM's share of the batch."""
    check(gdp, [1000, 200], [45, 130], 256, 2, 152, 16, 8, BF)


@pytest.mark.parametrize("K,V,dtype", [(64, 128, BF), (48, 32, F32), (64, 64, FP16)])
@pytest.mark.parametrize("before", [100, 64, 700])
def test_context_past_31_bits(gdp, K, V, dtype, before):
    """Positions that pass 2^31, in blocks of 2^30 tokens, through both forms."""
    ctx, bs, S = 2 ** 31 - before, 2 ** 30, 3
    check(gdp, [650], [ctx], bs, 1, 2, K, V, dtype)
    q, k, v, g, _ = inputs(1, S, 1, 2, K, V, dtype, "token")
    at = 2 ** 31 - 2
    tables, pool = paged_case([S], [at], bs, 2, K, V)
    ro, want = paged_reference(q, k, v, g, [0, S], [at], tables, pool, bs, K ** -0.5)
    got = pool.to(DEV)
    o = gdp.gdp_linear_recurrent_update_paged(q, k, v, g, got, tables.to(DEV),
                                              torch.tensor([at], dtype=torch.int32, device=DEV), bs)
    assert o_ok(o, ro) and err(got, want) <= TOL_S
