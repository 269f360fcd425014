"""A wait on the device that runs out in the tensor-core kernel of paged attention ends the call with
status 2, and later calls are right."""
import pytest
import torch

from test_attention_gpu import BF, DEV, check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,ctx,D,block", [([1, 1], [500, 40], 128, 16), ([64, 3], [700, 10], 128, 16),
                                              ([64, 3], [700, 10], 128, 5), ([64, 3], [700, 10], 256, 16)])
def test_wait_runs_out(gdp, lens, ctx, D, block):
    d = problem(lens, ctx, 8, 2, D, D, block, BF)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdp.gdp_debug_wait_fault(3, 0.02)
    try:
        gdp.gdp_attention_paged(**d, status=st)
        torch.cuda.synchronize()
    finally:
        gdp.gdp_debug_wait_fault(0)
    assert int(st) == 2
    check(gdp, d)
