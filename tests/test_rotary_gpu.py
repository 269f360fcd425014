"""Position rotation and appending to a paged cache, against their formulas in 64 bits.

Tolerances. A turned value is a c - b s with c, s from a phase known to 2^-63 of a turn: its rest in
[-1/8, 1/8] turns as a float is off by 2^-24 of at most pi / 4, sincospif by 2 ulp, the amplitude's
product, the two products and the sum by 2^-24 each: 8 x 2^-24 A (|a| + |b|) holds them all. A 16-bit
output adds half a step, u |y| with u = 2^-8 (bf16) or 2^-11 (fp16). Angles in the reference are
position times frequency in fp64, off by 2^-53 of at most 2^20 radians. Copies are exact.
"""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0, torch.float64: 0.0}
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def turned(x, pos, f, amplitude, offset, inter, sign=1.0):
    """Reference in fp64 and the tolerance, both shaped as x [..., H, D]."""
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    m = f.numel()
    i = offset + torch.arange(m, device=x.device) * (2 if inter else 1)
    j = i + (1 if inter else m)
    a, b = x.double()[..., i], x.double()[..., j]
    t = sign * pos.double()[..., None, None] * f
    y[..., i] = amplitude * (a * torch.cos(t) - b * torch.sin(t))
    y[..., j] = amplitude * (a * torch.sin(t) + b * torch.cos(t))
    size = 8 * 2.0 ** -24 * abs(amplitude) * (a.abs() + b.abs())
    tol[..., i] = size + UNIT[x.dtype] * y[..., i].abs()
    tol[..., j] = size + UNIT[x.dtype] * y[..., j].abs()
    return y, tol


def check(got, ref):
    y, tol = ref
    assert got.shape == y.shape
    assert bool(((got.double() - y).abs() <= tol).all()), float(((got.double() - y).abs() - tol).max())


def rows(gen, lead, sizes, dtype, fused):
    if not fused:
        return [torch.randn(*lead, H, D, generator=gen, device=DEV).to(dtype) for H, D in sizes]
    x = torch.randn(*lead, sum(H * D for H, D in sizes), generator=gen, device=DEV).to(dtype)
    return [p.unflatten(-1, s) for p, s in zip(x.split([H * D for H, D in sizes], -1), sizes)]


ROTARY = [
    # lead, H, D, R, offset, inter, dtype, fused
    ((1,), 1, 2, 2, 0, False, FP, False),
    ((1,), 16, 128, 128, 0, False, BF, False),
    ((37,), 5, 128, 128, 0, True, HF, True),
    ((300,), 3, 80, 48, 16, True, FP, True),
    ((2, 33), 4, 64, 32, 32, False, BF, True),     # whole vectors, the last half of the head
    ((129,), 2, 72, 36, 0, False, BF, False),      # half of the pairs is no whole vector
    ((129,), 2, 72, 36, 3, True, HF, False),       # pairs straddle vectors
    ((7,), 3, 33, 10, 21, True, BF, False),        # an odd head
    ((5,), 2, 1024, 1024, 0, False, BF, False),
    ((1000,), 1, 8, 2, 0, False, FP, False),
    ((50,), 70, 256, 0, 0, False, BF, False),      # nothing to turn: a copy
]


@pytest.mark.parametrize("lead,H,D,R,offset,inter,dtype,fused", ROTARY)
@pytest.mark.parametrize("backward", [False, True])
def test_rotary(gdp, lead, H, D, R, offset, inter, dtype, fused, backward):
    gen = torch.Generator(device=DEV).manual_seed(D + R)
    x = rows(gen, lead, [(H, D)] * 3, dtype, fused)[1]
    pos = torch.randint(0, 1 << 20, lead, generator=gen, device=DEV, dtype=torch.int32)
    f, _ = gdp.gdp_rotary_frequencies(R)
    a = 1.0 if D % 2 else 1.25
    want = turned(x, pos, f, a, offset, inter, -1.0 if backward else 1.0)
    y = gdp.gdp_rotary(x, pos, f, offset=offset, interleaved=inter, amplitude=a, backward=backward)
    check(y, want)
    assert y.is_contiguous()
    gdp.gdp_rotary(x, pos, f, offset=offset, interleaved=inter, amplitude=a, backward=backward, out=x)  # in place
    assert torch.equal(x, y)


def test_rotary_leaves_the_rest_of_a_projection(gdp):
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(9, 3 * 4 * 64, generator=gen, device=DEV).bfloat16()
    keep = x.clone()
    q = x[:, 256:512].unflatten(-1, (4, 64))
    f, _ = gdp.gdp_rotary_frequencies(64)
    gdp.gdp_rotary(q, torch.arange(9, dtype=torch.int32, device=DEV), f, out=q)
    assert torch.equal(x[:, :256], keep[:, :256]) and torch.equal(x[:, 512:], keep[:, 512:])
    assert not torch.equal(x[:, 256:512], keep[:, 256:512])


def test_rotary_gradient(gdp):
    """backward is the transpose: <g, R x> = <R^T g, x>, and the derivative along a direction."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    x, g, d = (torch.randn(40, 3, 48, generator=gen, device=DEV) for _ in range(3))
    pos = torch.randint(-5, 100000, (40,), generator=gen, device=DEV, dtype=torch.int32)
    f, a = gdp.gdp_rotary_frequencies(32, scaling="ramp", factor=8.0, original_length=4096)
    kw = dict(offset=8, interleaved=True, amplitude=a)
    gx = gdp.gdp_rotary(g, pos, f, backward=True, **kw).double()
    # linear, so the difference of two steps is exact up to the outputs' rounding
    hi = gdp.gdp_rotary(x + d, pos, f, **kw).double()
    lo = gdp.gdp_rotary(x - d, pos, f, **kw).double()
    along = ((hi - lo) / 2 * g.double()).sum()
    want = (gx * ((x + d).double() - (x - d).double()) / 2).sum()
    # each output is off by 8 x 2^-24 of its pair's sizes at most
    tol = 8 * 2.0 ** -24 * a * 4 * float((g.abs().double() * (x.abs() + d.abs()).double()).sum() * 2)
    assert abs(float(along - want)) <= tol
    x2 = x.double().requires_grad_()
    turned(x2, pos, f, a, 8, True)[0].backward(g.double())
    check(gx.float(), (x2.grad, turned(g, pos, f, a, 8, True, -1.0)[1]))


def test_rotary_far_positions(gdp):
    """Any int32 position, against angles in exact fractions."""
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567891, -77]
    f, _ = gdp.gdp_rotary_frequencies(16, base=500000.0)
    x = torch.zeros(len(pos), 1, 16, device=DEV)
    x[..., :8] = 1.0
    y = gdp.gdp_rotary(x, torch.tensor(pos, dtype=torch.int32, device=DEV), f).double().cpu()
    for n, p in enumerate(pos):
        for i, fi in enumerate(f.tolist()):
            rest = Fraction(fi) * p / (2 * pi) % 1
            angle = 2 * math.pi * float(rest)
            # 1 / 2 pi, its product and the phase in fp64: 3 x 2^-53 of the turns
            tol = 8 * 2.0 ** -24 + 2 * math.pi * 3 * 2.0 ** -53 * abs(p) * fi / (2 * math.pi) + 1e-15
            assert abs(float(y[n, 0, i]) - math.cos(angle)) <= tol
            assert abs(float(y[n, 0, i + 8]) - math.sin(angle)) <= tol


def cache(gen, pages, block, H, D, dtype, kind):
    if kind == "heads":                            # head-major pages
        return torch.randn(pages, H, block, D, generator=gen, device=DEV).to(dtype).transpose(1, 2)
    if kind == "pair":                             # one half of a buffer of both
        return torch.randn(pages, 2, block, H, D, generator=gen, device=DEV).to(dtype)[:, 1]
    return torch.randn(pages, block, H, D, generator=gen, device=DEV).to(dtype)


APPEND = [
    # T, H, HKV, D, DV, R, block, inter, dtype, fused, layout
    (1, 4, 1, 128, 128, 128, 64, False, BF, True, "plain"),
    (200, 8, 2, 128, 128, 128, 16, False, BF, True, "heads"),
    (77, 6, 3, 72, 40, 36, 24, True, FP, False, "pair"),
    (77, 6, 3, 72, 40, 36, 24, False, HF, False, "heads"),
    (65, 0, 2, 64, 64, 0, 1, False, HF, True, "plain"),
    (300, 3, 3, 33, 17, 12, 7, True, BF, False, "plain"),
    (5000, 2, 1, 64, 64, 64, 128, False, BF, True, "pair"),
]


@pytest.mark.parametrize("T,H,HKV,D,DV,R,block,inter,dtype,fused,layout", APPEND)
def test_append(gdp, T, H, HKV, D, DV, R, block, inter, dtype, fused, layout):
    gen = torch.Generator(device=DEV).manual_seed(T)
    q, k, v = rows(gen, (T,), [(H, D), (HKV, D), (HKV, DV)], dtype, fused)
    pages = -(-T // block) + 3
    kc, vc = cache(gen, pages, block, HKV, D, dtype, layout), cache(gen, pages, block, HKV, DV, dtype, layout)
    slot = torch.randperm(pages * block, generator=gen, device=DEV)[:T]
    slot[torch.rand(T, generator=gen, device=DEV) < 0.2] = -1
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, device=DEV, dtype=torch.int32)
    f = gdp.gdp_rotary_frequencies(R)[0] if R else None
    keep = slot >= 0
    at = slot[keep]
    want_k, tol_k = kc.double().clone(), torch.zeros(kc.shape, dtype=torch.float64, device=DEV)
    want_v = vc.clone()
    if R:
        y, t = turned(k, pos, f, 1.0, 0, inter)
    else:
        y, t = k.double(), torch.zeros(k.shape, dtype=torch.float64, device=DEV)
    want_k[at // block, at % block], tol_k[at // block, at % block] = y[keep], t[keep]
    want_v[at // block, at % block] = v[keep]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo = gdp.gdp_cache_append(k, v, kc, vc, slot, positions=pos if R else None, frequencies=f, interleaved=inter,
                              q=q if H else None, status=status)
    assert int(status) == 0
    check(kc, (want_k, tol_k))
    assert torch.equal(vc, want_v)
    if H:
        check(qo, turned(q, pos, f, 1.0, 0, inter))
    else:
        assert qo is None


def test_append_refuses_slots_on_the_device(gdp):
    kc = torch.zeros(3, 4, 2, 8, device=DEV)
    vc = torch.zeros(3, 4, 2, 8, device=DEV)
    k = torch.ones(5, 2, 8, device=DEV)
    slot = torch.tensor([12, -1, 11, -2, 1 << 40], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdp.gdp_cache_append(k, 2 * k, kc, vc, slot, status=status)
    assert int(status) == 1
    assert float(kc.sum()) == 16 and float(vc.sum()) == 32 and bool((kc[2, 3] == 1).all())


def test_append_like_rotary_then_copy(gdp):
    """The same numbers as gdp_rotary gives, bit for bit, and in a captured graph with new slots."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    q, k, v = rows(gen, (64,), [(8, 128), (2, 128), (2, 128)], BF, True)
    pos = torch.randint(0, 9000, (64,), generator=gen, device=DEV, dtype=torch.int32)
    f, a = gdp.gdp_rotary_frequencies(128, scaling="wavelength", factor=8.0, original_length=4096, high=4.0)
    kc, vc = torch.zeros(6, 16, 2, 128, device=DEV, dtype=BF), torch.zeros(6, 16, 2, 128, device=DEV, dtype=BF)
    slot = torch.arange(64, device=DEV)
    qo = torch.empty(64, 8, 128, device=DEV, dtype=BF)
    call = lambda: gdp.gdp_cache_append(k, v, kc, vc, slot, positions=pos, frequencies=f, amplitude=a, q=q,  # noqa: E731
                                        q_out=qo)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(qo, gdp.gdp_rotary(q, pos, f, amplitude=a))
    assert torch.equal(kc.flatten(0, 1)[:64], gdp.gdp_rotary(k, pos, f, amplitude=a))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    kc.zero_(), vc.zero_(), qo.zero_()
    slot.add_(32)
    pos.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kc.flatten(0, 1)[32:], gdp.gdp_rotary(k, pos, f, amplitude=a))
    assert torch.equal(vc.flatten(0, 1)[32:], v) and float(kc.flatten(0, 1)[:32].abs().sum()) == 0
    assert torch.equal(qo, gdp.gdp_rotary(q, pos, f, amplitude=a))


def test_empty_calls(gdp):
    f, _ = gdp.gdp_rotary_frequencies(8)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert gdp.gdp_rotary(torch.zeros(0, 2, 8, device=DEV), none, f).shape == (0, 2, 8)
    c = torch.zeros(0, 4, 2, 8, device=DEV)
    assert gdp.gdp_cache_append(torch.zeros(0, 2, 8, device=DEV), torch.zeros(0, 2, 8, device=DEV), c, c, none.long()) is None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)  # a cache without pages keeps nothing
    k = torch.zeros(1, 2, 8, device=DEV)
    gdp.gdp_cache_append(k, k, c, c, torch.zeros(1, dtype=torch.int64, device=DEV), status=status)
    assert int(status) == 1
