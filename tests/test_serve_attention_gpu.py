"""The attention serving example runs: prompts, drafted trees, accepted tokens appended again."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_example_runs(gdp):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_attention.py")
    spec = importlib.util.spec_from_file_location("serve_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    streams, lens, off = m.serve(requests=5, prompt=90, steps=6)
    assert all(len(x) >= n + 6 for x, n in zip(streams, lens))
    # the projection of one token and of many may round differently (bf16, half a step 2^-8, of k and of its rotation)
    assert off <= 2.0 ** -7
