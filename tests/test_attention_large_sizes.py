"""Sizes past 31 bits are refused by the bindings of rotation, append and paged attention: the library takes 32-bit
sizes, and a larger one would arrive as its low half, so that a part of the work was done. Tensors of such sizes are
stood in for by their shapes (an expanded dimension costs no memory). No GPU needed."""
import pytest
import torch

import linear_attention_ssm_gdp_gb300 as gdp

BIG = (1 << 32) + 3


class Shaped:
    """What the checks of sizes look at."""
    is_cuda, dtype = True, torch.bfloat16

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def stride(self):
        return (0,) * (len(self.shape) - 1) + (1,)


@pytest.mark.parametrize("shape", [(BIG, 2, 64), (2, BIG, 64), (1, BIG, 2, 64), (BIG, 1, 2, 64), (1, 1, BIG, 64),
                                   (1, 1, 1, BIG)])
def test_rows(shape):
    with pytest.raises(ValueError, match="31 bits"):
        gdp._heads("x", Shaped(*shape), torch.bfloat16)


@pytest.mark.parametrize("shape", [(BIG, 16, 2, 64), (4, BIG, 2, 64), (4, 16, BIG, 64), (4, 16, 2, BIG)])
def test_caches(shape):
    with pytest.raises(ValueError, match="31 bits"):
        gdp._cache_ok(Shaped(*shape), Shaped(*shape), torch.bfloat16)


def test_values_and_tables():
    with pytest.raises(ValueError, match="31 bits"):
        gdp._cache_ok(Shaped(4, 16, 2, 64), Shaped(4, 16, 2, BIG), torch.bfloat16)
    q, cache = Shaped(2, 1, 4, 64), Shaped(4, 16, 2, 64)
    q.dim = lambda: 4
    tables, lens = Shaped(2, BIG), Shaped(2)
    tables.dim, tables.dtype, lens.dtype = lambda: 2, torch.int32, torch.int32
    tables.is_contiguous = lens.is_contiguous = lambda: True
    with pytest.raises(ValueError, match="31 bits"):
        gdp.gdp_attention_paged(q, cache, cache, tables, lens)


def test_sizes_that_fit():
    assert gdp._heads("x", Shaped((1 << 31) - 1, 2, 64), torch.bfloat16)[2] == (1 << 31) - 1
    assert gdp._cache_ok(Shaped(1 << 30, 16, 2, 64), Shaped(1 << 30, 16, 2, 64), torch.bfloat16)[0] == 1 << 30
