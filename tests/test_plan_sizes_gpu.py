"""The block plan at the sizes where its shared memory passes what a launch may have unasked."""
import os
import subprocess
import sys

import pytest
import torch

from test_plan_norm_gpu import DEV, check_plan

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def requests(n):
    gen = torch.Generator().manual_seed(n)
    ctx = torch.randint(0, 60, (n,), generator=gen).tolist()
    qry = torch.randint(0, 3, (n,), generator=gen).tolist()
    tables = torch.randint(0, 1 << 20, (n, 4), generator=gen, dtype=torch.int32)
    return ctx, qry, tables, torch.randperm(n, generator=gen).tolist(), 2, 16, 2 * n


@pytest.mark.parametrize("n", [6110, 6143])
def test_first_call_of_a_process(n):
    """A larger call before it would have raised the limit already."""
    code = (f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]\n"
            "import linear_attention_ssm_gdp_gb300 as gdp\n"
            "from test_plan_sizes_gpu import check_plan, requests\n"
            f"check_plan(gdp, *requests({n}))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("n", [6109, 6110, 6126, 6143, 6144, 16383, 16384])
def test_many_requests(gdp, n):
    check_plan(gdp, *requests(n))
