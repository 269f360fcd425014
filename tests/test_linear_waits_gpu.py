"""Bounded waits of the linear-attention kernel: the test hook makes one run out;
the call returns, its status word says so whichever of the call's launches it was in, and the
next call is right."""
import time

import pytest
import torch

from test_linear_gpu import BF, DEV, TOL_S, err, inputs, o_ok, walk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,cut", [(60, False), (1500, True)])
@pytest.mark.parametrize("packed", [False, True])
def test_wait_runs_out(gdp, T, cut, packed):
    """T = 1500 is cut into segments: the wait is in the state pass, and the output pass that follows
    must not clear the word."""
    H, HV, K, V = 1, 2, 128, 128
    q, k, v, g, s0 = inputs(1, T, H, HV, K, V, BF, "token")
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV) if packed else None
    need = gdp.gdp_linear_chunk_fwd_workspace_size(1, T, 1, H, HV, K, V, BF)
    assert (need > 2 * HV * K * V * 4) == cut  # a state for each of two segments
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    try:
        gdp.gdp_debug_wait_fault(2, 0.05)
        start = time.time()
        gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu, initial_state=s0, workspace=ws)
        status = gdp.gdp_read_status(ws)  # synchronises
        elapsed = time.time() - start
    finally:
        gdp.gdp_debug_wait_fault(False, 0.0)
    assert status == 4 and elapsed < 5.0, (status, elapsed)  # GDP_ERR_DEVICE_TIMEOUT
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu, initial_state=s0, workspace=ws)
    assert gdp.gdp_read_status(ws) == 0
    ro, after = walk(q, k, v, g, s0, K ** -0.5)
    assert o_ok(o, ro) and err(fs, after[-1]) <= TOL_S
