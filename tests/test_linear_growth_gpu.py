"""Decay factors at the end of fp32's range (a positive g is a growth): one token multiplies a state of
powers of two by e^g, so the state's relative error is the factor's, 2^-23 for the pair of floats
rounded to one; 4e-7 with the product's and the sum's roundings, which below the normal range are half
of the smallest float, 2^-149, each."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("K,V,dtype", [(128, 128, torch.bfloat16), (8, 8, torch.bfloat16), (4, 4, torch.float32)])
@pytest.mark.parametrize("form", ["recurrent", "chunk"])
def test_factor_near_the_top(gdp, K, V, dtype, form):
    g = torch.tensor([-87.0, -80.0, -1.0, 0.0, 1.0, 80.0, 87.9, 88.02, 88.3, 88.37, 88.38, 88.5, 88.69, 88.7, 88.71, 88.722])
    n = g.numel()
    q, k, v = (torch.zeros(n, 1, 1, c, dtype=dtype, device=DEV) for c in (K, K, V))
    s0 = torch.full((n, 1, K, V), 2.0 ** -10, device=DEV)
    s0[:, :, ::2] *= -2.0
    want = torch.exp(g.double())[:, None, None, None] * s0.double().cpu()
    gd = g.to(DEV)[:, None, None].contiguous()
    if form == "recurrent":
        got = s0.clone()
        gdp.gdp_linear_recurrent_update(q, k, v, gd, got)
    else:
        got = gdp.gdp_linear_chunk_fwd(q, k, v, gd, initial_state=s0)[1]
    off = ((got.double().cpu() - want).abs() / (4e-7 * want.abs() + 2.0 ** -149)).amax((1, 2, 3))
    assert (off <= 1).all(), dict(zip(g.tolist(), off.tolist()))


def test_factor_past_the_top(gdp):
    """Past ln of the largest float the factor is infinite, as e^g rounded to fp32 is."""
    q = k = v = torch.zeros(2, 1, 1, 8, device=DEV)
    s = torch.ones(2, 1, 8, 8, device=DEV)
    gdp.gdp_linear_recurrent_update(q, k, v, torch.tensor([88.73, 1000.0], device=DEV)[:, None, None], s)
    assert torch.isinf(s).all()
