"""The block plan at the sizes where its shared memory passes what a launch may have unasked, and with
as many tokens as an int holds."""
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


def test_most_tokens(gdp):
    """max_tokens = 2^31 - 1, 34 GB of outputs of which three requests fill the head."""
    N = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    i32 = dict(dtype=torch.int32, device=DEV)
    tables = torch.full((3, 4), -1, **i32)
    out = gdp.gdp_block_plan(torch.zeros(3, **i32), torch.tensor([5, 0, 20], **i32), tables,
                             torch.tensor([7, 6, 5], **i32), torch.zeros(1, **i32), 16, N)
    cu, req, pos, slot, used = out
    assert cu.tolist() == [0, 5, 5, 25] and int(used) == 3
    assert tables.tolist() == [[7, -1, -1, -1], [-1] * 4, [6, 5, -1, -1]]
    assert req[:25].tolist() == [0] * 5 + [2] * 20 and pos[:25].tolist() == [*range(5), *range(20)]
    assert slot[:25].tolist() == [*range(112, 117), *range(96, 112), *range(80, 84)]
    for t in (req, pos, slot):
        for a in range(25, N, 1 << 28):
            assert int(t[a:a + (1 << 28)].max()) == int(t[a:a + (1 << 28)].min()) == -1
