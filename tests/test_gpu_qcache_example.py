"""The example that runs the 8-bit latent cache's three calls together: pages are neither lost nor shared, and the
outputs differ from the unquantised cache's by what E4M3 rounding makes.

Elements are rounded by at most 2^-4 of themselves (uniformly within: 2^-4 / sqrt(3) rms at the worst, about two thirds
of that over a binade). Attention averages values with independent errors, so an output's relative error is that of a
value, and the scores' errors (relative 2^-4 again, scores of order one) add as much: below 2^-3 together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantised_cache.py")


def test_example_runs():
    from mla_block_diffusion_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("quantised_cache", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, pages = example.main(steps=24, seed=3)
    assert pages == 64 and 0 < worst < 2.0 ** -3
