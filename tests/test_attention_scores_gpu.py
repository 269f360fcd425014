"""Paged attention where scores are far from 0.

The tensor-core kernel takes weights relative to a base that lags behind the row's maximum. Scores of 2^22 and more (in
powers of two) have steps of a half and more, and a score that is not rounded as its base was would make weights of 2^16
and more, or none.
"""
import pytest
import torch

from test_attention_gpu import BF, DEV, FP, HF, UNIT, problem

pytestmark = pytest.mark.gpu


def same_pages(d, n, tokens):
    """d's one request n times, on the same pages: enough items that CTAs hold whole ones."""
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(d, block_tables=d["block_tables"].expand(n, -1).contiguous(),
                context_lens=d["context_lens"].expand(n).contiguous(),
                cu_seqlens=torch.arange(0, n * tokens + 1, tokens, **i32))


def place(d, p):
    """(page, slot) of the positions p of the first request."""
    block = d["k_cache"].shape[1]
    return d["block_tables"][0, p // block].long(), p % block


def bound(o, A, n, dtype):
    """Of o where a score's own error moves no weight: the terms of reference() without e_j."""
    u = UNIT[dtype]
    return u * o.abs() + A * ((u if dtype != FP else 0.0) + 2.0 ** -20 + (80 + n / 16) * 2.0 ** -23)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("rows", [1, 3, 200])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_large_scores_that_are_equal(gdp, dtype, D, rows, sign):
    """Every key has the same score, of up to 2^29 (fp16) or 2^70: o is the values' mean. Products of one
    column are exact, and equal scores are off by the same."""
    n_keys, n = 200, 40
    d = problem([rows], [n_keys - rows], 1, 1, D, D, 16, dtype)
    gen = torch.Generator(device=DEV).manual_seed(D + rows)
    d["k_cache"].zero_()
    d["k_cache"][..., 0] = 2.0 ** (13 if dtype == HF else 30)
    d = same_pages(d, n, rows)
    d["q"] = torch.zeros(1, n * rows, 1, D, device=DEV, dtype=dtype)
    e = torch.rand(n * rows, generator=gen, device=DEV) * (16 if dtype == HF else 40)
    d["q"][0, :, 0, 0] = sign * torch.exp2(e).clamp(max=60000.0 if dtype == HF else 2.0 ** 40).to(dtype)
    got = gdp.gdp_attention_paged(**d, scale=1.0)
    page, at = place(d, torch.arange(n_keys, device=DEV))
    v = d["v_cache"][page, at, 0].double()
    i = torch.arange(n * rows, device=DEV) % rows + n_keys - rows
    o, A = v.cumsum(0)[i] / (i[:, None] + 1), v.abs().cumsum(0)[i] / (i[:, None] + 1)
    bad = (got[0, :, 0].double() - o).abs() - bound(o, A, n_keys, dtype)
    assert bool((bad <= 0).all()), (float(bad.max()), int((bad > 0).sum()), bad.numel())


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_large_scores_far_apart(gdp, dtype, D, up):
    """Scores 2^16 and more apart: the largest one's value alone, first or last in the context."""
    n_keys, n = 300, 40
    d = problem([1], [n_keys - 1], 1, 1, D, D, 16, dtype)
    p = torch.arange(n_keys, device=DEV)
    page, at = place(d, p)
    d["k_cache"].zero_()
    # five steps of sixty keys, which every type holds
    d["k_cache"][page, at, 0, 0] = ((128 + 31 * (p // 60 if up else (n_keys - 1 - p) // 60)) * 2.0 ** 5).to(dtype)
    d = same_pages(d, n, 1)
    d["q"] = torch.zeros(1, n, 1, D, device=DEV, dtype=dtype)
    d["q"][0, :, 0, 0] = torch.exp2(torch.linspace(7, 15.9, n, device=DEV)).to(dtype)
    got = gdp.gdp_attention_paged(**d, scale=1.0)
    last = p >= 240 if up else p < 60              # sixty keys share the largest score
    v = d["v_cache"][page, at, 0].double()[last]
    o, A = v.mean(0), v.abs().mean(0)
    bad = (got[0, :, 0].double() - o).abs() - bound(o, A, n_keys, dtype)
    assert bool((bad <= 0).all()), (float(bad.max()), int((bad > 0).sum()), bad.numel())
