"""Which kernel a norm of single positions runs, by the names in a captured graph, and its results around
those choices: fp32 groups of 516 to 1024 channels in whole vectors are not read element by element
where latency counts or their vectors fill the lanes."""
import ctypes

import pytest
import torch

from test_plan_norm_gpu import BF, DEV, F32, FP16, check_norm

pytestmark = pytest.mark.gpu


def kernel_names(graph):
    """Names of a captured graph's kernels, from the driver."""
    cu, P = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p
    raw, n = P(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes, names = (P * n.value)(), []
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        params = (P * 16)()  # func, grid, block and shared memory (32 bytes), params, extra, kernel, context
        assert cu.cuGraphKernelNodeGetParams_v2(P(node), ctypes.byref(params)) == 0
        name = ctypes.c_char_p()
        get, handle = (cu.cuFuncGetName, params[0]) if params[0] else (cu.cuKernelGetName, params[7])
        assert get(ctypes.byref(name), P(handle)) == 0
        names.append(name.value.decode())
    return names


def kernel_of(gdp, N, C, G, dtype):
    x, out = torch.zeros(N, 1, C, dtype=dtype, device=DEV), torch.empty(N, 1, C, dtype=dtype, device=DEV)
    gdp.gdp_group_norm(x, G, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        gdp.gdp_group_norm(x, G, out=out)
    (name,) = kernel_names(graph)
    return next(k for k in ("norm_rows_kernel", "norm_elements_kernel", "norm_map_kernel") if k in name)


@pytest.mark.parametrize("N,C,G,dtype,want", [
    (200, 2560, 4, F32, "norm_rows_kernel"), (1, 640, 1, F32, "norm_rows_kernel"), (3000, 1024, 1, F32, "norm_rows_kernel"),
    (9000, 1800, 2, F32, "norm_rows_kernel"), (2, 516, 1, F32, "norm_rows_kernel"), (64, 512, 1, F32, "norm_rows_kernel"),
    (300, 4096, 4, BF, "norm_rows_kernel"), (20000, 640, 1, F32, "norm_elements_kernel"),
    (300, 2044, 4, F32, "norm_elements_kernel"), (300, 60, 6, BF, "norm_elements_kernel"),
    (9, 2100, 2, FP16, "norm_map_kernel"), (9, 4096, 2, BF, "norm_map_kernel"), (9, 1028, 1, F32, "norm_map_kernel"),
])
def test_choice(gdp, N, C, G, dtype, want):
    assert kernel_of(gdp, N, C, G, dtype) == want


@pytest.mark.parametrize("N,C,G,dt,out", [
    (200, 2560, 4, F32, F32), (3, 516, 1, F32, BF), (77, 1800, 2, F32, FP16), (40, 1024, 1, F32, F32),
    (20000, 640, 1, F32, BF), (9, 2056, 2, F32, F32), (3000, 772, 1, F32, F32),
])
@pytest.mark.parametrize("gate", [False, True])
def test_around_the_choice(gdp, N, C, G, dt, out, gate):
    check_norm(gdp, N, 1, C, G, dt, out, gate)
    check_norm(gdp, N, 1, C, G, dt, out, gate, strided=True, affine=False)
