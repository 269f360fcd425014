"""Refusals of the rotation, append and paged-attention entry points, and the rotation's
frequencies: every invalid argument gives its status before anything is launched, so no GPU is
needed."""
import ctypes
import math
import os

import pytest
import torch

P = ctypes.c_void_p
A = 1 << 20  # an address that is never followed


@pytest.fixture(scope="module")
def lib():
    import linear_attention_ssm_gdp_gb300 as gdp
    if not os.path.exists(gdp.LIB_PATH):
        from linear_attention_ssm_gdp_gb300 import _build
        _build.build()
    gdp.load()
    return gdp


@pytest.fixture(scope="module")
def so(lib):
    return lib.load()


def st(*s):
    return (ctypes.c_int64 * len(s))(*s)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(xs=None), 1), (dict(ys=None), 1), (dict(xs=st(0, -1, 8)), 1),
    (dict(pos=None), 1), (dict(f=None), 1), (dict(R=7), 1), (dict(R=-2), 1), (dict(R=34), 1), (dict(offset=-1), 1),
    (dict(R=16, offset=17), 1), (dict(a=NAN), 1), (dict(a=INF), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=-1), 1),
    (dict(D=0, R=0), 1), (dict(D=1025), 2), (dict(dt=3), 2), (dict(B=1 << 16, T=1 << 15), 2), (dict(H=1 << 26), 2),
    (dict(y=A, ys=st(0, 128, 32)), 1),        # in place with other strides
    (dict(ys=st(0, 64, 0)), 1), (dict(ys=st(0, 0, 32)), 1), (dict(B=2, ys=st(0, 64, 32)), 1),  # elements in one place
])
def test_rotary_rejects(so, kw, status):
    a = dict(x=A, xs=st(0, 64, 32), pos=A, f=A, R=32, offset=0, a=1.0, B=1, T=4, H=2, D=32, dt=0, y=2 * A,
             ys=st(0, 64, 32))
    a.update(kw)
    assert so.gdp_rotary(P(a["x"]), a["xs"], P(a["pos"]), P(a["f"]), a["R"], a["offset"], 0, a["a"], 0, a["B"], a["T"],
                         a["H"], a["D"], a["dt"], P(a["y"]), a["ys"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(st=None), 1), (dict(st=st(*[0, 64, 32] * 2, 0, 64, -1)), 1),
    (dict(q=A, q_out=None), 1), (dict(q=A, q_out=A, H=4), 1), (dict(slot=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=st(64, -32, 32)), 1), (dict(pos=None), 1), (dict(f=None), 1),
    (dict(R=40), 1), (dict(offset=1), 1), (dict(a=NAN), 1), (dict(pages=-1), 1), (dict(block=0), 1), (dict(HKV=0), 1),
    (dict(DV=0), 1), (dict(H=-1), 1), (dict(T=-1), 1), (dict(dt=7), 2), (dict(D=2000), 2), (dict(DV=1025), 2),
    (dict(HKV=1 << 25), 2), (dict(ks=st(256, 64, 0)), 1), (dict(vs=st(0, 64, 32)), 1),  # slots in one place
])
def test_append_rejects(so, kw, status):
    a = dict(q=None, k=A, v=A, st=st(*[0, 64, 32] * 3), pos=A, f=A, R=32, offset=0, a=1.0, B=1, T=4, H=2, HKV=2, D=32,
             DV=32, dt=0, slot=A, kc=A, ks=st(256, 64, 32), vc=A, vs=st(256, 64, 32), pages=3, block=4, q_out=2 * A)
    a.update(kw)
    assert so.gdp_cache_append(P(a["q"]), P(a["k"]), P(a["v"]), a["st"], P(a["pos"]), P(a["f"]), a["R"], a["offset"], 0,
                               a["a"], a["B"], a["T"], a["H"], a["HKV"], a["D"], a["DV"], a["dt"], P(a["slot"]),
                               P(a["kc"]), a["ks"], P(a["vc"]), a["vs"], a["pages"], a["block"], P(a["q_out"]), None,
                               None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(qs=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(qs=st(0, -1, 8)), 1), (dict(ks=st(-1, 8, 8)), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(pages=-1), 1),
    (dict(block=0), 1), (dict(tables=None), 1), (dict(width=-1), 1), (dict(ctx=None), 1), (dict(cu=A, B=2), 1),
    (dict(N=3), 1), (dict(N=-1), 1), (dict(H=5), 1), (dict(H=0), 1), (dict(HKV=0), 1), (dict(D=0), 1), (dict(DV=0), 1),
    (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(D=257), 2), (dict(DV=257), 2), (dict(dt=5), 2),
    (dict(width=1 << 20, block=1 << 11), 2), (dict(B=1 << 17, N=1 << 17, T=1 << 17), 2),
    (dict(T=1 << 30, B=1, N=1), 2),           # rows of a request past 32 bits
    (dict(ws=None), 5), (dict(ws=A + 16), 5), (dict(bytes=100), 5),
])
def test_attention_rejects(so, kw, status):
    a = dict(q=A, qs=st(64, 64, 16), kc=A, ks=st(256, 64, 32), vc=A, vs=st(256, 64, 32), pages=3, block=4, tables=A,
             width=4, ctx=A, cu=None, N=2, B=2, T=1, H=4, HKV=2, D=32, DV=32, scale=1.0, dt=0, o=A, ws=A,
             bytes=1 << 40)
    a.update(kw)
    assert so.gdp_attention_paged(P(a["q"]), a["qs"], P(a["kc"]), a["ks"], P(a["vc"]), a["vs"], a["pages"], a["block"],
                                  P(a["tables"]), a["width"], P(a["ctx"]), P(a["cu"]), a["N"], None, a["B"], a["T"],
                                  a["H"], a["HKV"], a["D"], a["DV"], a["scale"], a["dt"], P(a["o"]), None, P(a["ws"]),
                                  a["bytes"], None) == status


def test_empty_calls_launch_nothing(so):
    s3, s9 = st(0, 0, 0), st(*[0] * 9)
    assert so.gdp_rotary(None, None, None, None, 32, 0, 0, 1.0, 0, 1, 0, 2, 32, 0, None, None, None) == 0
    assert so.gdp_cache_append(None, None, None, s9, None, None, 0, 0, 0, 1.0, 1, 0, 2, 2, 32, 32, 0, None, None, s3,
                               None, s3, 0, 4, None, None, None) == 0
    assert so.gdp_attention_paged(None, s3, None, s3, None, s3, 0, 4, None, 0, None, None, 0, None, 0, 1, 4, 2, 32, 32,
                                  1.0, 0, None, None, None, 0, None) == 0


def test_workspace_size(so):
    size = so.gdp_attention_paged_workspace_size
    assert size(2, 1, 2, 4, 2, 32, 32, 0) > 0
    assert size(2, 1, 2, 5, 2, 32, 32, 0) == size(2, 1, 2, 4, 2, 257, 32, 0) == size(2, 1, 2, 4, 2, 32, 32, 9) == 0
    assert size(2, 64, 2, 64, 2, 128, 128, 0) >= size(2, 1, 2, 64, 2, 128, 128, 0)


def test_python_checks(lib):
    """What the binding refuses by itself, on CPU tensors."""
    x, pos = torch.zeros(4, 2, 8), torch.zeros(4, dtype=torch.int32)
    f, _ = lib.gdp_rotary_frequencies(8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lib.gdp_rotary(x, pos, f)
    with pytest.raises(ValueError):
        lib.gdp_rotary(x.double(), pos, f)
    with pytest.raises(ValueError, match="CUDA"):
        lib.gdp_cache_append(x, x, x[None], x[None], pos.long())
    with pytest.raises(ValueError):
        lib.gdp_attention_paged(x, x[None], x[None], pos[None], pos)
    with pytest.raises(ValueError, match="scaling"):
        lib.gdp_rotary_frequencies(8, scaling="other")
    with pytest.raises(lib.GDPError):
        lib.gdp_rotary_frequencies(7)


@pytest.mark.parametrize("kw,status", [
    (dict(R=5), 1), (dict(R=-2), 1), (dict(base=0.0), 1), (dict(base=NAN), 1), (dict(out=None), 1), (dict(kind=4), 2),
    (dict(kind=1, factor=0.0), 1), (dict(kind=2, length=0.0), 1), (dict(kind=2, low=2.0, high=2.0), 1),
    (dict(kind=3, low=0.0), 1), (dict(kind=3, high=INF), 1), (dict(kind=2, base=1.0), 1),
])
def test_frequencies_reject(so, kw, status):
    a = dict(R=8, base=1e4, kind=0, factor=2.0, length=100.0, low=1.0, high=4.0, out=(ctypes.c_double * 8)())
    a.update(kw)
    assert so.gdp_rotary_frequencies(a["R"], a["base"], a["kind"], a["factor"], a["length"], a["low"], a["high"],
                                     a["out"], None) == status


def test_frequencies(lib):
    """Against the formulas; 1e-14 holds the roundings of pow and a few products."""
    def close(a, b):
        return all(abs(x - y) <= 1e-14 * abs(y) for x, y in zip(a.tolist(), b)) and len(a) == len(b)

    R, base, L = 64, 50000.0, 4096.0
    plain = [base ** (-2 * i / R) for i in range(R // 2)]
    f, a = lib.gdp_rotary_frequencies(R, base, device="cpu")
    assert close(f, plain) and a == 1.0
    f, a = lib.gdp_rotary_frequencies(R, base, "linear", 8.0, device="cpu")
    assert close(f, [x / 8 for x in plain]) and a == 1.0
    f, a = lib.gdp_rotary_frequencies(R, base, "ramp", 8.0, L, 1.0, 32.0, device="cpu")
    lo = math.floor(R * math.log(L / (32 * 2 * math.pi)) / (2 * math.log(base)))
    hi = math.ceil(R * math.log(L / (2 * math.pi)) / (2 * math.log(base)))
    t = [min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(R // 2)]
    assert close(f, [x * (1 - s) + x / 8 * s for x, s in zip(plain, t)]) and abs(a - 0.1 * math.log(8) - 1) < 1e-14
    assert f[0] == plain[0] and 0 < lo < hi < R // 2
    f, a = lib.gdp_rotary_frequencies(R, base, "wavelength", 8.0, L, 1.0, 4.0, device="cpu")
    s = [min(max((L * x / (2 * math.pi) - 1) / 3, 0.0), 1.0) for x in plain]
    assert close(f, [x * k + x / 8 * (1 - k) for x, k in zip(plain, s)]) and a == 1.0
    assert 0.0 in s and 1.0 in s and any(0 < k < 1 for k in s)
    assert lib.gdp_rotary_frequencies(0, device="cpu")[0].numel() == 0
    # base 1, one pair: no angle formula divides by ln(base) there
    assert lib.gdp_rotary_frequencies(2, 1.0, device="cpu")[0].tolist() == [1.0]


class _On:
    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("current,devices,ok", [(0, (0, None, 0), True), (1, (1, 1), True), (0, (1, 1), False),
                                                (0, (0, 1), False), (1, (1, None, 0), False)])
def test_tensors_elsewhere_are_refused(lib, monkeypatch, current, devices, ok):
    monkeypatch.setattr(lib, "_current_device", lambda: current)
    ts = [None if d is None else _On(d) for d in devices]
    if ok:
        lib._one_device(*ts)
    else:
        with pytest.raises(ValueError, match="current CUDA device"):
            lib._one_device(*ts)
