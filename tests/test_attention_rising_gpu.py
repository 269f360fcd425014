"""Paged attention where scores rise along the context: the tensor-core kernel takes weights relative to a base that lags
behind the row's maximum, and scales the outputs and sums that it has when the base moves. Here it moves in nearly every
tile, by another factor in every row.
"""
import pytest
import torch

from test_attention_gpu import BF, DEV, FP, HF, problem, reference
from test_attention_scores_gpu import place, same_pages

pytestmark = pytest.mark.gpu


# tokens and query heads a key head: few rows, 128, and 256 (both slots have rows of their own)
@pytest.mark.parametrize("tokens,G", [(1, 4), (16, 8), (64, 4)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_scores_that_rise(gdp, dtype, D, tokens, G):
    """Up to 24 powers of two from one tile of 64 keys to the next, down to none, by row; few requests, cut into pieces,
    and many, in whole items."""
    ctx, HKV = 703, 1
    one = problem([tokens], [ctx], HKV * G, HKV, D, D, 64, dtype, loud=0.3)
    p = torch.arange(ctx + tokens, device=DEV)
    page, at = place(one, p)
    one["k_cache"][page, at, :, 0] = (p.float() / 64).to(dtype)[:, None]
    one["v_cache"][page, at] += 1.0                # (values of one sign: weights that are off do not average out)
    for n in (2, 200):
        d = same_pages(one, n, tokens)
        d["q"] = one["q"].repeat(1, n, 1, 1)
        slope = torch.arange(n * tokens * HKV * G, device=DEV).view(1, n * tokens, HKV * G) * 0.618034 % 1 * 24
        slope[0, ::5] = -slope[0, ::5]             # and some that fall
        d["q"][..., 0] = (slope * 0.6931471806 * D ** 0.5).to(dtype)
        got = gdp.gdp_attention_paged(**d)
        o, tol = reference(**d)
        bad = (got.flatten(0, 1).double() - o).abs() - tol
        assert bool((bad <= 0).all()), (n, float(bad.max()), int((bad > 0).sum()), bad.numel())
        # the tolerance holds no tile whose weights were left at the base of its own time
        rows = slice(0, 2 * tokens)
        k, v = one["k_cache"][page, at, 0].double(), one["v_cache"][page, at, 0].double()
        x = d["q"][0, rows].double() @ k.T * (D ** -0.5 / 0.6931471805599453)
        i = torch.arange(2 * tokens, device=DEV) % tokens
        x = x.masked_fill((p[None] - ctx > i[:, None])[:, None], -torch.inf)
        w, base = torch.zeros_like(x), torch.full_like(x[..., :1], -torch.inf)
        for j in range(0, x.shape[-1], 64):
            top = x[..., j:j + 64].amax(-1, keepdim=True)
            base = torch.where(top > base + 8, top, base)
            w[..., j:j + 64] = torch.exp2(x[..., j:j + 64] - base)
        wrong = (w / w.sum(-1, keepdim=True)) @ v
        assert bool(((wrong - o[rows]).abs() > tol[rows]).any())
