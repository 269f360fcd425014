"""Linear attention as a server meets it: neighbours in a packed batch, views off the 16-byte grid,
many short sequences, captured graphs, and the operators together in the serving example."""
import importlib.util
import os

import pytest
import torch

from test_linear_gpu import BF, DEV, F32, FP16, TOL_S, err, inputs, o_ok, walk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,V,dtype", [(128, 128, BF), (64, 64, FP16), (48, 40, F32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_neighbours_stay_apart(gdp, K, V, dtype, bad):
    """What is not finite in one sequence of a packed batch, or between them, leaves the others
    bit for bit as they are."""
    q, k, v, g, _ = inputs(1, 700, 1, 2, K, V, dtype, "token")
    cu = torch.tensor([0, 70, 70, 150, 640], dtype=torch.int32, device=DEV)
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu)
    q2, k2, v2, g2 = (x.clone() for x in (q, k, v, g))
    for x in (q2, k2, v2, g2):
        x[:, 70:150] = bad
        x[:, 640:] = bad
    o2, fs2 = gdp.gdp_linear_chunk_fwd(q2, k2, v2, g2, cu_seqlens=cu)
    for a, b in ((0, 70), (150, 640)):
        assert torch.equal(o[:, a:b], o2[:, a:b])
    for s in (0, 1, 3):
        assert torch.equal(fs[s], fs2[s])
    assert not torch.isfinite(o2[:, 70:150].float()).all()


@pytest.mark.parametrize("dtype", [BF, FP16, F32])
@pytest.mark.parametrize("shift", [1, 3])
def test_views_off_the_grid(gdp, dtype, shift):
    """Bases and rows on no 16-byte step: the same numbers as from copies, to rounding."""
    B, T, H, HV, K, V = 2, 200, 2, 4, 64, 64
    q, k, v, g, s0 = inputs(B, T, H, HV, K, V, dtype, "token")
    wide = torch.randn(B, T, 2 * H * K + HV * V + 2 * shift, device=DEV).to(dtype)
    flat = wide[..., shift:-shift]
    flat.copy_(torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], -1))
    q, k, v = flat.split([H * K, H * K, HV * V], -1)
    q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (HV, V))
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, initial_state=s0)
    ro, after = walk(q, k, v, g, s0, K ** -0.5)
    assert o_ok(o, ro) and err(fs, after[-1]) <= TOL_S
    st = s0.clone()
    o = gdp.gdp_linear_recurrent_update(q[:, :3], k[:, :3], v[:, :3], g[:, :3].contiguous(), st)
    assert o_ok(o, ro[:, :3]) and err(st, after[2]) <= TOL_S


@pytest.mark.parametrize("dtype,K,V", [(BF, 8, 8), (F32, 6, 5)])
def test_many_short_sequences(gdp, dtype, K, V):
    """70,000 sequences of one token or none, and a long one among them."""
    n = 70000
    lens = torch.ones(n, dtype=torch.int64)
    lens[::7], lens[n // 2] = 0, 3000
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T = int(cu[-1])
    q, k, v, g, _ = inputs(1, T, 1, 1, K, V, dtype, "token")
    s0 = torch.randn(n, 1, K, V, device=DEV)
    o, fs = gdp.gdp_linear_chunk_fwd(q, k, v, g, cu_seqlens=cu.int().to(DEV), initial_state=s0)
    one = torch.nonzero(lens == 1)[:, 0]
    t = cu[one]
    qq, kk, vv = (x[0, t, 0].double().cpu() for x in (q, k, v))
    want = torch.exp(g[0, t, 0].double().cpu())[:, None, None] * s0[one, 0].double().cpu() + kk[:, :, None] * vv[:, None]
    assert err(fs[one, 0], want) <= TOL_S
    assert o_ok(o[0, t, 0], K ** -0.5 * torch.einsum("nk,nkv->nv", qq, want))
    empty = (lens == 0).to(DEV)
    assert torch.equal(fs[empty], s0[empty])
    a = int(cu[n // 2])
    ro, after = walk(*(x[:, a:a + 3000] for x in (q, k, v, g)), s0[n // 2:n // 2 + 1], K ** -0.5)
    assert o_ok(o[:, a:a + 3000], ro) and err(fs[n // 2], after[-1][0]) <= TOL_S


def test_captured_step(gdp):
    """Plan, paged decode and norm in one captured graph: replays follow the lengths in memory."""
    n, HV, K, V, bs, new = 6, 4, 64, 64, 16, 20
    q, k, v, g, _ = inputs(n, new, 2, HV, K, V, BF, "token")
    i32 = dict(dtype=torch.int32, device=DEV)
    free = torch.randperm(32, generator=torch.Generator().manual_seed(0)).int().to(DEV)
    pool = torch.zeros(32, HV, K, V, device=DEV)
    tables, ctx, used = torch.full((n, 4), -1, **i32), torch.zeros(n, **i32), torch.zeros(1, **i32)
    ones, status = torch.ones(n, **i32), torch.zeros(1, **i32)
    x = [torch.empty_like(t[:, :1]) for t in (q, k, v, g)]
    w = torch.ones(HV * V, device=DEV)
    o = torch.empty(n, 1, HV, V, dtype=BF, device=DEV)

    def step():
        out = gdp.gdp_block_plan(ctx, ones, tables, free, used, bs, n, status=status)
        gdp.gdp_linear_recurrent_update_paged(*x, pool, tables, ctx, bs, out=o)
        y = gdp.gdp_group_norm(o.view(n, HV * V), HV, w)
        used.copy_(out[4])
        ctx.add_(1)
        return y

    for t, a in zip(x, (q, k, v, g)):
        t.copy_(a[:, :1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ro, after = walk(q, k, v, g, None, K ** -0.5)
    for s in range(1, new):
        for t, a in zip(x, (q, k, v, g)):
            t.copy_(a[:, s:s + 1])
        graph.replay()
        assert o_ok(o, ro[:, s:s + 1])
    assert int(status) == 0 and int(used) == 2 * n and ctx.tolist() == [new] * n
    assert err(pool[tables[:, 1].long()], after[-1]) <= TOL_S


def test_serving_example(gdp):
    """Paged prompts, a shared prefix and paged decoding end in the dense form's states. Both see
    the same bf16 activations up to their own roundings of a layer's output, u = 2^-8 each: a few
    of them over two layers, 0.05 of a state's norm at the most."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_linear_attention.py")
    spec = importlib.util.spec_from_file_location("serve_linear_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    streams, off, _ = m.serve(requests=3, prompt=300, new=140)
    assert [len(s) for s in streams] == [440, 403, 366, 256 + 5 + 140, 256 + 65 + 140]
    assert max(off) <= 0.05
