"""examples/paged_decode.py: planning, append and attention between FP8 projections, one step
captured as a graph and replayed, against float64 at the end."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


@pytest.mark.parametrize("requests,steps", [(1, 3), (16, 8), (70, 66)])
def test_the_example_agrees_with_float64(requests, steps):
    # 66 steps: every request takes a new page inside the replays
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # outputs are rounded to bf16 once (half of 2^-7 of an element at most), weights to 16 bits
    assert example.main(["--requests", str(requests), "--steps", str(steps)]) < 2.0 ** -8
