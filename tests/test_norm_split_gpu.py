"""Group norm of few groups with many elements, whose slices meet in a workspace: against the 64-bit
form with the tolerance of the other norm tests (the output's own rounding and 1e-5 RMS), at the
sizes around the choice of that path, and its refusals."""
import ctypes

import pytest
import torch

from test_plan_norm_gpu import BF, DEV, F32, FP16, check_norm, norm_reference


@pytest.mark.gpu
@pytest.mark.parametrize("N,L,C,G,dt,out", [
    (1, 16384, 128, 1, FP16, FP16), (1, 9001, 80, 1, BF, BF), (2, 7001, 21, 1, F32, F32),
    (1, 16383, 30, 1, BF, BF), (3, 5000, 256, 2, F32, BF), (1, 16384, 96, 32, BF, BF),
    (1, 60000, 24, 8, F32, F32), (2, 9000, 512, 4, F32, F32), (1, 1 << 20, 10, 2, BF, BF),
])
@pytest.mark.parametrize("gate", [False, True])
def test_split(gdp, N, L, C, G, dt, out, gate):
    check_norm(gdp, N, L, C, G, dt, out, gate)


@pytest.mark.gpu
def test_split_strided_and_without_workspace(gdp):
    check_norm(gdp, 2, 9000, 64, 1, BF, BF, True, strided=True)
    x = torch.randn(1, 9000, 64, generator=torch.Generator().manual_seed(0)).to(DEV)
    y, z = gdp.gdp_group_norm(x, 1), torch.empty_like(x)
    st = gdp.load().gdp_group_norm(x.data_ptr(), x.stride(0), x.stride(1), None, 0, 0, None, None, 1, 9000, 64, 1,
                                   1e-5, 1, 2, 2, z.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    ref = norm_reference(x, 1, None, None, None, 1e-5, "silu")
    for got in (y, z):
        assert (got.double().cpu() - ref).abs().max() <= 1e-5 * ref.abs().max()
    with pytest.raises(gdp.GDPError):
        gdp.gdp_group_norm(x, 1, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


@pytest.mark.gpu
def test_split_large_offset(gdp):
    """A mean 1000 times the spread, as in the whole form: half an ulp of the mean, 3e-5, over a
    spread of 2, and as much again for the merged mean: 1e-4."""
    x = (torch.randn(1, 20000, 32, generator=torch.Generator().manual_seed(3)) * 2 + 1000.0).to(DEV)
    y = gdp.gdp_group_norm(x, 1, activation="none")
    ref = norm_reference(x, 1, None, None, None, 1e-5, "none")
    assert (y.double().cpu() - ref).abs().max().item() <= 1e-4


def test_workspace_size_and_refusals():
    import linear_attention_ssm_gdp_gb300 as lib
    size, ws = lib.gdp_group_norm_workspace_size, lib.load().gdp_group_norm_ws
    P = ctypes.c_void_p
    assert size(1, 16384, 128, 1, FP16) > 0
    assert size(8192, 1, 4096, 32, BF) == size(0, 9, 8, 1, BF) == size(4, 9, 8, 3, BF) == 0

    def call(work, nbytes, C=128, G=1):
        return ws(P(1 << 20), 1 << 24, 128, None, 0, 0, None, None, 1, 16384, C, G, 1e-5, 1, 1, 1, P(1 << 20), P(work), nbytes,
                  None)
    no = call(None, 1 << 30)
    assert no == call((1 << 20) + 16, 1 << 30) == call(1 << 20, 8) != 0
    assert b"workspace" in lib.load().gdp_status_string(no).lower()
    assert call(1 << 20, 1 << 30, G=5) == 1
