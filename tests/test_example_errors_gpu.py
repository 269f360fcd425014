"""The serving example keeps what any of its steps reported, not the last one's word alone."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_errors_of_earlier_steps_stay():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_linear_attention.py")
    spec = importlib.util.spec_from_file_location("serve_linear_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    rng = torch.Generator(device=DEV).manual_seed(0)
    layers = [m.Layer(64, 1, 2, 16, 16, rng, DEV)]
    s = m.Server(layers, torch.randn(10, 64, generator=rng, device=DEV).bfloat16(), 4, 2, 2, 64, DEV)
    s.prompts([[1, 2, 3]])
    assert s.errors() == 0
    s.plan(slice(1, 2), torch.tensor([-1], dtype=torch.int32, device=DEV), 4)  # a negative length
    s.decode(torch.tensor([3], device=DEV))
    assert s.errors() == 1
    s.ctx[0] = -5  # the paged prompt form skips it
    q, k, v, _, g = layers[0].project(torch.randn(4, 64, generator=rng, device=DEV).bfloat16())
    s.attend_prompts(q, k, v, g, torch.tensor([0, 4], dtype=torch.int32, device=DEV), s.pools[0], s.tables[:1], s.ctx[:1])
    assert s.errors() & 1
