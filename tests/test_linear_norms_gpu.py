"""Linear attention, chunked form, held to a bound on the 2-norm, which a systematic error of a few
tenths of a percent does not pass, over types and sizes, those with K above 128 among them.

Rounding o to p bits alone costs at most u / sqrt(3) of its norm (errors uniform in half an ulp, every
mantissa 1). With K <= 128 in bf16 the scores and the read-out's copy of the state are rounded to bf16
as well: each is off like o itself, they add to different terms, and the terms' sum is off by as much
relative to itself: sqrt(2) of that. Otherwise the operands have 22 bits or more. fp32 outputs and all states: 2^-24
per rounding, at the chunks' ends and in the sums, a few of them: 1e-6."""
import pytest
import torch

from test_linear_gpu import BF, DEV, F32, FP16, TOL_S, UNIT, err, inputs, o_ok, paged_case, paged_reference, walk

pytestmark = pytest.mark.gpu


def off(got, want):
    want, got = want.double().cpu(), got.double().cpu()
    return float((got - want).norm() / want.norm())


def bound(dtype, K, V):
    if dtype == F32:
        return 1e-6
    return (2 if dtype == BF and K <= 128 and K % 8 == 0 and V % 8 == 0 else 1) ** 0.5 * UNIT[dtype] / 3 ** 0.5


SIZES = [
    (2, 300, 1, 2, 256, 128), (1, 200, 2, 2, 192, 80), (1, 129, 1, 3, 136, 64), (2, 65, 1, 1, 250, 33), (1, 64, 1, 1, 129, 7),
    (1, 700, 1, 1, 256, 256), (2, 500, 2, 4, 128, 128), (1, 333, 1, 2, 64, 64), (1, 37, 2, 2, 128, 256), (1, 1, 2, 2, 200, 40),
]


@pytest.mark.parametrize("B,T,H,HV,K,V", SIZES)
@pytest.mark.parametrize("dtype", [BF, FP16, F32])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_dense(gdp, B, T, H, HV, K, V, dtype, decay):
    q, k, v, g, s0 = inputs(B, T, H, HV, K, V, dtype, decay, packed=True)
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0)
    ro, after = walk(q, k, v, g, s0, K ** -0.5)
    assert off(fs, after[-1]) <= 1e-6 and err(fs, after[-1]) <= TOL_S
    if B * T * HV * V >= 5000:  # a norm of few elements is a draw
        assert off(o, ro) <= bound(dtype, K, V)
    assert o_ok(o, ro)


@pytest.mark.parametrize("K,V", [(256, 64), (200, 40)])
@pytest.mark.parametrize("dtype", [BF, FP16, F32])
def test_wide_keys_packed_and_paged(gdp, K, V, dtype):
    H, HV, bs, lens, ctx = 1, 2, 64, [1, 0, 130, 600], [0, 5, 70, 37]
    cu = [0, 1, 1, 131, 731]
    i32 = dict(dtype=torch.int32, device=DEV)
    q, k, v, g, _ = inputs(1, 731, H, HV, K, V, dtype, "token", seed=4)
    tables, pool = paged_case(lens, ctx, bs, HV, K, V)
    ro, want = paged_reference(q, k, v, g, cu, ctx, tables, pool, bs, K ** -0.5)
    got = pool.to(DEV)
    o = gdp.gdp_linear_chunk_fwd_paged(q, k, v, g, torch.tensor(cu, **i32), got, tables.to(DEV), torch.tensor(ctx, **i32),
                                       bs)
    assert off(o, ro) <= bound(dtype, K, V) and o_ok(o, ro) and err(got, want) <= TOL_S
    s0 = torch.randn(4, HV, K, V, generator=torch.Generator().manual_seed(1)).to(DEV)
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=torch.tensor(cu, **i32), initial_state=s0)
    for r, n in enumerate(lens):
        ro, after = walk(*(x[:, cu[r]:cu[r + 1]] for x in (q, k, v, g)), s0[r:r + 1], K ** -0.5)
        assert o_ok(o[:, cu[r]:cu[r + 1]], ro)
        assert err(fs[r], after[-1][0] if n else s0[r]) <= TOL_S
