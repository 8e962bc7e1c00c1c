"""The example that runs the 8-bit layers and the 8-bit latent cache together, prompts and single tokens: what the layer adds
differs from 32 bits by what E4M3 rounding makes.

A rounding to E4M3 is off by at most 2^-4 of the element, about 2^-4 / sqrt(3) * 2/3 = 0.024 of it in the mean square (uniform
within a step, averaged over a binade). A product's relative error in the mean square is sqrt(2) * 0.024 = 0.034 (rows and
weights, independent terms), and the layer's sum meets at most six such roundings one after another (two products and the cache
on the way to the attention's output, then out; gate or up, the product's rounding, down): below sqrt(6) * 0.034 = 0.083
if all were passed on in full; 2^-3 leaves room for the softmax's share and for few rows."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantised_layer.py")


def test_example_runs():
    from mla_block_diffusion_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("quantised_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert 0 < example.main(tokens=6, seed=3) < 2.0 ** -3
