"""A scale that is finite, but not once it is in powers of two (times log2 e, 1.44), is refused before anything is
launched: every score would be infinite, or NaN where it is 0. No GPU needed."""
import ctypes
import os

import pytest

import linear_attention_ssm_gdp_gb300 as gdp

P = ctypes.c_void_p
A = 1 << 20  # an address that is never followed


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(gdp.LIB_PATH):
        from linear_attention_ssm_gdp_gb300 import _build
        _build.build()


def call(scale):
    st = (ctypes.c_int64 * 3)(64, 64, 16)
    # a workspace of no bytes: what is not refused for its scale is refused for that (5)
    return gdp.load().gdp_attention_paged(P(A), st, P(A), st, P(A), st, 3, 4, P(A), 4, P(A), None, 2, None, 2, 1, 4, 2,
                                          16, 16, scale, 0, P(A), None, P(A), 0, None)


@pytest.mark.parametrize("scale,status", [(1.0, 5), (0.0, 5), (-1e38, 5), (2.3e38, 5), (2.4e38, 1), (-3.4e38, 1),
                                          (float("inf"), 1), (float("nan"), 1)])
def test_scale(scale, status):
    assert call(scale) == status
