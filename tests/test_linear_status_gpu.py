"""What the chunked linear-attention calls report on the device, without a workspace of the caller's."""
import pytest
import torch

from test_linear_gpu import BF, DEV, F32, inputs

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("K,V,dtype", [(128, 128, BF), (32, 48, F32)])
def test_offsets(gdp, K, V, dtype):
    q, k, v, g, _ = inputs(1, 100, 1, 2, K, V, dtype, "token")
    status = torch.full((1,), 77, **I32)
    for cu, want in (([0, 50, 40, 100], 1), ([0, 50, 60, 100], 0), ([0, 10, 20, 101], 1), ([0, 0, 0, 0], 0)):
        o = torch.full((1, 100, 2, V), 7.0, dtype=dtype, device=DEV)
        fs = torch.empty(3, 2, K, V, device=DEV)
        gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=torch.tensor(cu, **I32), out=(o, fs), status=status)
        assert int(status) == want
        assert want == 0 or (bool((o == 7.0).all()) and bool((fs == 0).all()))
    status.fill_(77)
    gdp.gdp_linear_chunk_fwd(q, k, v, g, status=status)  # dense
    assert int(status) == 0


def test_tables(gdp):
    q, k, v, g, _ = inputs(1, 100, 1, 2, 128, 128, BF, "token")
    pool, cu = torch.zeros(4, 2, 128, 128, device=DEV), torch.tensor([0, 50, 100], **I32)
    status = torch.full((1,), 77, **I32)
    for tables, ctx, want in (([[0], [1]], [0, 3], 0), ([[0], [4]], [0, 3], 1), ([[0], [1]], [0, -1], 1)):
        gdp.gdp_linear_chunk_fwd_paged(q, k, v, g, cu, pool, torch.tensor(tables, **I32), torch.tensor(ctx, **I32), 64,
                                       status=status)
        assert int(status) == want


def test_wait_and_refusals(gdp):
    q, k, v, g, _ = inputs(1, 60, 1, 2, 128, 128, BF, "token")
    status = torch.zeros(1, **I32)
    try:
        gdp.gdp_debug_wait_fault(2, 0.05)
        gdp.gdp_linear_chunk_fwd(q, k, v, g, status=status)
        assert int(status) == 2
    finally:
        gdp.gdp_debug_wait_fault(False, 0.0)
    gdp.gdp_linear_chunk_fwd(q, k, v, g, status=status)
    assert int(status) == 0
    for bad in (status.cpu(), status.long(), status[:0]):
        with pytest.raises(ValueError):
            gdp.gdp_linear_chunk_fwd(q, k, v, g, status=bad)
