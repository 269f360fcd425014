"""Group norm of single positions whose groups or rows are not whole vectors, many samples: the
64-bit form, with the tolerance of the other norm tests."""
import pytest

from test_plan_norm_gpu import BF, F32, FP16, check_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,C,G,dt,out", [
    (20011, 12, 4, F32, F32), (30001, 6, 2, FP16, FP16), (3, 3, 3, BF, BF), (1001, 130, 10, BF, BF),
    (513, 1023, 1, F32, BF), (77, 2050, 2, FP16, FP16), (9, 63, 7, F32, FP16), (5, 9, 1, BF, BF),
])
@pytest.mark.parametrize("gate", [False, True])
def test_elements(gdp, N, C, G, dt, out, gate):
    check_norm(gdp, N, 1, C, G, dt, out, gate)
    check_norm(gdp, N, 1, C, G, dt, out, gate, strided=True, affine=False)
