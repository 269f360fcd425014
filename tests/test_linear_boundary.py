"""Refusals of the linear-attention, block-plan and group-norm entry points: every invalid
argument gives its status before anything is launched, so no GPU is needed."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
A = 1 << 20  # an address that is never followed


@pytest.fixture(scope="module")
def so():
    import linear_attention_ssm_gdp_gb300 as gdp
    if not os.path.exists(gdp.LIB_PATH):
        from linear_attention_ssm_gdp_gb300 import _build
        _build.build()
    return gdp.load()


def strides(**kw):
    a = [0, 64, 32] * 3
    for i, x in kw.items():
        a[int(i[1:])] = x
    return (ctypes.c_int64 * 9)(*a)


CHUNK = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(st=None), 1),
    (dict(st=strides(_4=-1)), 1),             # a negative stride
    (dict(H=3, HV=4), 1), (dict(H=0), 1), (dict(T=-1), 1),
    (dict(N=3), 1),                           # a dense batch has a state per batch entry
    (dict(cu=A, B=2), 1),                     # a packed one has B = 1
    (dict(s0=A + 4), 1), (dict(fs=A + 8), 1),  # states off the 16-byte grid
    (dict(K=257), 2), (dict(V=1025), 2), (dict(dt=9), 2), (dict(B=1 << 16, N=1 << 16, T=1 << 16), 2),
    (dict(ws=None), 3), (dict(ws=A + 16), 3), (dict(bytes=0), 3),
]


@pytest.mark.parametrize("kw,status", CHUNK)
def test_chunk_rejects(so, kw, status):
    a = dict(q=A, k=A, v=A, st=strides(), g=None, s0=None, cu=None, N=2, B=2, T=64, H=2, HV=2, K=32, V=32, dt=0,
             o=A, fs=None, ws=A, bytes=1 << 40)
    a.update(kw)
    want = {1: 1, 2: 2, 3: so_workspace_status(so)}[status]
    assert so.gdp_linear_chunk_fwd(P(a["q"]), P(a["k"]), P(a["v"]), a["st"], P(a["g"]), 1, P(a["s0"]), P(a["cu"]),
                                   a["N"], a["B"], a["T"], a["H"], a["HV"], a["K"], a["V"], 1.0, a["dt"],
                                   P(a["o"]), P(a["fs"]), P(a["ws"]), a["bytes"], None) == want


def so_workspace_status(so):
    """The status that names a workspace in its text."""
    return next(s for s in range(6) if b"workspace" in so.gdp_status_string(s).lower())


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), 1), (dict(pool=None), 1), (dict(pool=A + 4), 1), (dict(tables=None), 1), (dict(ctx=None), 1),
    (dict(pages=0), 1), (dict(width=0), 1), (dict(block=0), 1), (dict(block=48), 2), (dict(K=300), 2),
])
def test_paged_chunk_rejects(so, kw, status):
    a = dict(cu=A, N=2, T=64, K=32, V=32, pool=A, pages=4, tables=A, width=2, ctx=A, block=64)
    a.update(kw)
    assert so.gdp_linear_chunk_fwd_paged(P(A), P(A), P(A), strides(), None, 0, P(a["cu"]), a["N"], a["T"], 2, 2,
                                         a["K"], a["V"], 1.0, 0, P(a["pool"]), a["pages"], P(a["tables"]),
                                         a["width"], P(a["ctx"]), a["block"], P(A), P(A), 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), 1), (dict(S=17), 1), (dict(state=None), 1), (dict(state=A + 4), 1), (dict(H=3, HV=4), 1),
    (dict(q=None), 1), (dict(K=257), 2), (dict(V=1025), 2), (dict(dt=9), 2), (dict(n=-1), 1),
])
def test_recurrent_rejects(so, kw, status):
    a = dict(q=A, state=A, n=2, S=1, H=2, HV=2, K=32, V=32, dt=0)
    a.update(kw)
    assert so.gdp_linear_recurrent_update(P(a["q"]), P(A), P(A), strides(), None, 0, P(a["state"]), a["n"], a["S"],
                                          a["H"], a["HV"], a["K"], a["V"], 1.0, a["dt"], P(A), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), 1), (dict(S=17), 1), (dict(pool=None), 1), (dict(pool=A + 4), 1), (dict(pages=0), 1),
    (dict(width=0), 1), (dict(tables=None), 1), (dict(ctx=None), 1), (dict(block=0), 1), (dict(V=2000), 2),
])
def test_paged_recurrent_rejects(so, kw, status):
    a = dict(pool=A, pages=4, tables=A, width=2, ctx=A, block=16, S=1, V=32)
    a.update(kw)
    assert so.gdp_linear_recurrent_update_paged(P(A), P(A), P(A), strides(), None, 0, P(a["pool"]), a["pages"],
                                                P(a["tables"]), a["width"], P(a["ctx"]), a["block"], 2, a["S"], 2,
                                                2, 32, a["V"], 1.0, 0, P(A), None, None) == status


def test_empty_decode_is_a_no_op(so):
    assert so.gdp_linear_recurrent_update(None, None, None, None, None, 0, None, 0, 1, 2, 2, 32, 32, 1.0, 0, None,
                                          None) == 0


def test_workspace_size(so):
    size = so.gdp_linear_chunk_fwd_workspace_size
    assert size(2, 64, 2, 2, 2, 32, 32, 0) > 0
    assert size(2, 64, 2, 3, 4, 32, 32, 0) == size(2, 64, 2, 2, 2, 257, 32, 0) == size(2, 64, 2, 2, 2, 32, 32, 9) == 0
    # segments cost a state each: a long sequence with few heads needs them
    assert size(1, 65536, 1, 1, 1, 128, 128, 0) >= 2 * 128 * 128 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(block=0), 1), (dict(tokens=-1), 1), (dict(n_free=-1), 1), (dict(width=-1), 1),
    (dict(cu=None), 1), (dict(used=None), 1), (dict(used_out=None), 1), (dict(used_out=A), 1), (dict(ctx=None), 1),
    (dict(query=None), 1), (dict(tables=None), 1), (dict(free=None), 1), (dict(slot=None), 1), (dict(req=None), 1),
    (dict(pos=None), 1), (dict(n=16385), 2), (dict(width=1 << 20, block=1 << 11), 2),
])
def test_block_plan_rejects(so, kw, status):
    a = dict(ctx=A, query=A, n=4, tables=A, width=8, free=A, n_free=9, used=A, block=16, tokens=32, cu=A, req=A,
             pos=A, slot=A, used_out=A + 64)
    a.update(kw)
    assert so.gdp_block_plan(P(a["ctx"]), P(a["query"]), a["n"], P(a["tables"]), a["width"], P(a["free"]),
                             a["n_free"], P(a["used"]), a["block"], a["tokens"], P(a["cu"]), P(a["req"]),
                             P(a["pos"]), P(a["slot"]), P(a["used_out"]), None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(L=-1), 1), (dict(C=0), 1), (dict(G=0), 1), (dict(G=5), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(x_sl=63), 1), (dict(x_sn=63), 1),
    (dict(gate=A, g_sl=8), 1), (dict(act=2), 2), (dict(dt=9), 2), (dict(dt=0, out=2), 2), (dict(L=1 << 31), 2),
])
def test_group_norm_rejects(so, kw, status):
    a = dict(x=A, x_sn=640, x_sl=64, gate=None, g_sn=640, g_sl=64, N=2, L=10, C=64, G=4, eps=1e-5, act=1, dt=2, out=2,
             y=A)
    a.update(kw)
    assert so.gdp_group_norm(P(a["x"]), a["x_sn"], a["x_sl"], P(a["gate"]), a["g_sn"], a["g_sl"], None, None, a["N"],
                             a["L"], a["C"], a["G"], a["eps"], a["act"], a["dt"], a["out"], P(a["y"]), None) == status


def test_empty_norm_is_a_no_op(so):
    assert so.gdp_group_norm(None, 64, 64, None, 0, 0, None, None, 0, 1, 64, 4, 1e-5, 0, 0, 0, None, None) == 0
