"""Segments of the chunked linear-attention forms, both sides' arithmetic without a GPU: whatever
the device may cut has its place in the scratch that the host planned."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHUNK = 64
SOURCE = r"""
#include "linear_plan.h"
using namespace gdp::linear;
extern "C" {
void plan(int N, int B, int T, int HV, int K, int V, int packed, int vt, int G, long long* out) {
  const Plan x = plan_of(N, B, T, HV, K, V, packed, vt, Cost{1.85, 1.2, 3.0, 6.0}, G);
  out[0] = x.nseg, out[1] = x.Lseg, out[2] = x.bound, out[3] = x.segS, out[4] = x.total, out[5] = x.slots;
}
int segments(int off, int n, int Lseg) { return segment_count(off, n, Lseg); }
void span(int off, int n, int Lseg, int j, int* out) { segment_span(off, n, Lseg, j, &out[0], &out[1]); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    so = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "linear_attention_ssm_gdp_gb300", "csrc"), str(d / "plan.cpp"), "-o", so],
                   check=True)
    return ctypes.CDLL(so)


def plan(lib, N, B, T, HV, K=128, V=128, packed=1, vt=128, G=152):
    out = (ctypes.c_longlong * 6)()
    lib.plan(N, B, T, HV, K, V, packed, vt, G, out)
    return dict(zip(("nseg", "Lseg", "bound", "segS", "total", "slots"), out))


@pytest.mark.parametrize("G", [148, 152])
@pytest.mark.parametrize("V,vt", [(128, 128), (128, 64), (80, 32)])
def test_no_cut_without_scratch(lib, G, V, vt):
    """A sequence that starts inside a chunk (a paged one with a context) spans up to 63 positions
    more than it has tokens; where the plan has no scratch, no offset may cut it."""
    lengths = [1, 63, 64, 65, 448, 449, 450, 500, 511, 512, 513, 575, 576, 577, 640, 1000, 4095, 4096, 16384, 100000]
    for HV in (1, 2, 16, 32, 74, 75, 76, 148, 150, 152, 160, 304):
        for T in lengths + [random.Random(HV).randint(1, 20000) for _ in range(40)]:
            x = plan(lib, 1, 1, T, HV, V=V, vt=vt, G=G)
            cut = max(lib.segments(off, T, x["Lseg"]) for off in range(CHUNK))
            assert cut == 1 or x["segS"], (T, HV, x, cut)


def test_counts_stay_in_bounds(lib):
    """Records of every sequence, however lengths and offsets fall."""
    rng = random.Random(0)
    for _ in range(3000):
        N, HV = rng.randint(1, 40), rng.choice([1, 4, 32, 76, 152])
        lens = [rng.choice([0, 1, rng.randint(1, 700), rng.randint(1, 5000)]) for _ in range(N)]
        T = max(1, sum(lens))
        x = plan(lib, N, 1, T, HV)
        n = sum(lib.segments(rng.choice([0, 63, rng.randint(0, 63)]), n, x["Lseg"]) for n in lens)
        assert n <= x["bound"]


def test_dense_segments_cover_the_sequence(lib):
    for T in list(range(1, 300)) + [4096, 8191, 16384, 100001]:
        for B, HV in ((1, 1), (2, 16), (4, 32)):
            x = plan(lib, B, B, T, HV, packed=0)
            assert (x["nseg"] - 1) * x["Lseg"] < T <= x["nseg"] * x["Lseg"] and x["bound"] == B * x["nseg"]
            assert (x["nseg"] > 1) == bool(x["segS"])


def test_scratch_is_for_cut_sequences(lib):
    """A state of scratch for each segment of a cut sequence, none for whole ones, and enough for
    however the lengths fall."""
    rng = random.Random(1)
    for _ in range(4000):
        N, HV = rng.randint(1, 40), rng.choice([1, 4, 32, 76, 152])
        lens = [rng.choice([0, 1, 450, 451, 512, 513, 1024, 1025, rng.randint(1, 5000)]) for _ in range(N)]
        T = max(1, sum(lens))
        x = plan(lib, N, 1, T, HV)
        counts = [lib.segments(rng.choice([0, 63, rng.randint(0, 63)]), n, x["Lseg"]) for n in lens]
        assert sum(c for c in counts if c > 1) <= x["slots"]
        assert x["slots"] <= 2 * T / (x["Lseg"] - 62) + 1


@pytest.mark.parametrize("N,T", [(256, 8192), (600, 600), (1000, 1000), (1024, 4096)])
def test_many_short_requests_need_little(N, T):
    """Through the library's own query: 32 heads of 128 x 128, a request's state is 2 MB."""
    import linear_attention_ssm_gdp_gb300 as gdp
    if not os.path.exists(gdp.LIB_PATH):
        from linear_attention_ssm_gdp_gb300 import _build
        _build.build()
    size = gdp.load().gdp_linear_chunk_fwd_workspace_size
    for dtype in (0, 1, 2):
        assert size(1, T, N, 32, 32, 128, 128, dtype) <= max(50 << 20, T // 256 * (3 << 20))


MOST = 2 ** 31 - 4096  # tokens of a chunked call


@pytest.mark.parametrize("T", [MOST, MOST - 63, 1_900_000_000, 2 ** 30 + 1])
@pytest.mark.parametrize("HV,G", [(1, 152), (100, 152), (151, 152), (152, 152), (400, 152)])
def test_longest_sequences(lib, T, HV, G):
    """Lengths that fill an int: segments follow one another and end with the sequence."""
    for packed, off in ((1, 0), (1, 63), (0, 0)):
        x = plan(lib, 1, 1, T, HV, packed=packed)
        assert 0 < x["Lseg"] and (x["bound"] - 1) * x["Lseg"] < T + 2 * x["Lseg"]
        if not packed:
            assert (x["nseg"] - 1) * x["Lseg"] < T <= x["nseg"] * x["Lseg"]
            continue
        n, at = lib.segments(off, T, x["Lseg"]), 0
        assert n == -(-(off + T) // x["Lseg"]) <= x["bound"] and (n == 1 or n <= x["slots"])
        for j in range(n):
            ends = (ctypes.c_int * 2)()
            lib.span(off, T, x["Lseg"], j, ends)
            lo, hi = ends
            assert lo == at and lo < hi <= T
            at = hi
        assert at == T


def test_many_sequences(lib):
    """Records are counted in 64 bits."""
    x = plan(lib, 2 ** 31 - 2, 1, 64, 1)
    assert x["bound"] > 2 ** 31 and x["total"] > 32 * 2 ** 31


@pytest.mark.parametrize("B,T,N,status", [(1, MOST + 1, 1, 2), (1, 2 ** 31 - 1, 1, 2), (1, 64, 2 ** 31 - 2, 2)])
def test_refused_lengths(B, T, N, status):
    import linear_attention_ssm_gdp_gb300 as gdp
    A = ctypes.c_void_p(1 << 20)
    st = (ctypes.c_int64 * 9)(*[64] * 9)
    assert gdp.load().gdp_linear_chunk_fwd(A, A, A, st, None, 0, None, A, N, B, T, 1, 1, 32, 32, 1.0, 0, A, None, A,
                                           1 << 62, None) == status
    assert gdp.load().gdp_linear_chunk_fwd_workspace_size(B, T, N, 1, 1, 32, 32, 0) == 0
