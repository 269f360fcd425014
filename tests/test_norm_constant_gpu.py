"""Group norm of groups of equal and of nearly equal values. The mean of n values is off by a few
roundings, (log2 n + 2) 2^-24 of it, 7e-5 at 100; the rest of the mean that is taken out is good to as
many roundings of itself, 5e-11; times 1 / sqrt(eps) = 316: 2e-8. Equal values give z = 0 within
1e-6 (a mean that keeps its rounding gives up to 2.4e-3). Values a few ulps apart are held to the other
norm tests' tolerance: their distances from the rounded mean are whole ulps, whose sums are exact."""
import pytest
import torch

from test_plan_norm_gpu import BF, DEV, F32, FP16, norm_reference

pytestmark = pytest.mark.gpu
SIZES = [
    (300, 1, 96, 1), (64, 1, 480, 4), (9, 1, 1200, 2), (30, 1, 3600, 3), (7, 1, 1536, 2), (40, 1, 30, 6),  # tokens
    (50, 1, 560, 10), (20, 1, 720, 6), (6, 1, 1792, 2),
    (5, 1, 40000, 1), (6, 7, 24, 2), (3, 500, 96, 3), (2, 4097, 12, 1), (1, 700, 4000, 2), (4, 33, 600, 5),  # positions
    (1, 16383, 30, 1), (2, 9000, 48, 1), (1, 30000, 56, 1),                                               # slices
]


def levels(N, L, C, G, dtype):
    level = (100.0 + 50.0 * torch.rand(N, 1, G, 1, generator=torch.Generator().manual_seed(C))).to(dtype)
    return level.expand(N, L, G, C // G).reshape(N, L, C).contiguous()


@pytest.mark.parametrize("N,L,C,G", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF, FP16])
def test_equal_values(gdp, N, L, C, G, dtype):
    y = gdp.gdp_group_norm(levels(N, L, C, G, dtype).to(DEV), G, activation="none")
    assert y.float().abs().max().item() <= 1e-6


@pytest.mark.parametrize("N,L,C,G", SIZES)
def test_a_few_ulps_apart(gdp, N, L, C, G):
    ulps = torch.randint(0, 4, (N, L, C), generator=torch.Generator().manual_seed(1))
    x = (levels(N, L, C, G, F32) + ulps * 2.0 ** -17).to(DEV)  # an ulp between 64 and 128; a half of one up to 256
    y = gdp.gdp_group_norm(x, G, activation="none")
    ref = norm_reference(x, G, None, None, None, 1e-5, "none")
    assert ((y.double().cpu() - ref).abs() <= 1e-5 * ref.pow(2).mean().sqrt()).all()


@pytest.mark.parametrize("N,L,C,G", SIZES + [(300, 1, 2864, 4), (300, 1, 4000, 4), (2000, 1, 1000, 1), (3000, 1, 896, 1)])
@pytest.mark.parametrize("at", ["first", "second", "last"])
def test_an_outlier_costs_the_others_nothing(gdp, N, L, C, G, at):
    """One value 1000 times the others': sums and distances round to a few 2^-24 of the outlier's
    sqrt(n) stds or of the value itself, 1e-6 of it; the others are held to 4e-6, a few dozen 2^-24."""
    x = torch.randn(N, L, G, C // G, generator=torch.Generator().manual_seed(L + C))
    l, c = {"first": (0, 0), "second": (0, 1), "last": (L - 1, C // G - 1)}[at]
    x[:, l, :, c] *= 1000.0
    x = x.reshape(N, L, C).to(DEV)
    ref = norm_reference(x, G, None, None, None, 1e-5, "none")
    y = gdp.gdp_group_norm(x, G, activation="none").double().cpu()
    assert ((y - ref).abs() <= 1e-6 * ref.abs() + 4e-6 * ref.pow(2).mean().sqrt()).all()
