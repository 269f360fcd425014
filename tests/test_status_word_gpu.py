"""The status word of the append and of paged attention keeps the worse of what calls report: a word that several calls
share holds 2 (a wait ran out, the output is not whole) whatever a later call finds, and 2 after 1."""
import pytest
import torch

from test_attention_gpu import BF, DEV, FP, problem

pytestmark = pytest.mark.gpu


def word(x):
    return torch.full((1,), x, dtype=torch.int32, device=DEV)


# heads of 64 in bf16 with pages of 16 and of 12: the tensor cores' two ways to load; fp32: the kernel for any size
@pytest.mark.parametrize("dtype,block", [(BF, 16), (BF, 12), (FP, 16)])
@pytest.mark.parametrize("before,after", [(0, 1), (1, 1), (2, 2)])
def test_attention(gdp, dtype, block, before, after):
    d = problem([2, 1, 3], [40, 30, 20], 4, 2, 64, 64, block, dtype)
    pages = d["block_tables"].clone()
    pages[1, 0] = d["k_cache"].shape[0]
    lens = torch.tensor([40, -1, 20], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 2, 1, 6], dtype=torch.int32, device=DEV)
    for bad in (dict(block_tables=pages), dict(context_lens=lens), dict(cu_seqlens=offsets)):
        st = word(before)
        gdp.gdp_attention_paged(**dict(d, **bad), status=st)
        assert int(st) == after
    st = word(before)
    gdp.gdp_attention_paged(**d, status=st)        # nothing to report: left as it was
    assert int(st) == before


@pytest.mark.parametrize("before", [0, 1, 2])
def test_wait_runs_out(gdp, before):
    d = problem([1, 1], [500, 40], 8, 2, 128, 128, 16, BF)
    st = word(before)
    gdp.gdp_debug_wait_fault(3, 0.02)
    try:
        gdp.gdp_attention_paged(**d, status=st)
        torch.cuda.synchronize()
    finally:
        gdp.gdp_debug_wait_fault(0)
    assert int(st) == 2


@pytest.mark.parametrize("before,after", [(0, 1), (1, 1), (2, 2)])
def test_append(gdp, before, after):
    kc, vc = torch.zeros(3, 4, 2, 8, device=DEV), torch.zeros(3, 4, 2, 8, device=DEV)
    k, st = torch.ones(2, 2, 8, device=DEV), word(before)
    gdp.gdp_cache_append(k, k, kc, vc, torch.tensor([12, 3], device=DEV), status=st)
    assert int(st) == after and float(kc.sum()) == 16
