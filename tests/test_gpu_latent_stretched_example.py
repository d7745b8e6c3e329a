"""examples/latent_decode.py with stretched positions: the frequencies' amplitude is in the scale."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_decode.py")


@pytest.mark.parametrize("factor", [1.0, 8.0])
def test_the_example_with_stretched_positions(factor):
    spec = importlib.util.spec_from_file_location("latent_decode", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(2, 64, factor, torch.device("cuda:0"))
    assert layer.scale == example.SCALE * (1 if factor == 1 else 0.1 * math.log(factor) + 1) ** 2
    # a new token's key is turned, not scaled: its size is the projection's, to bf16's rounding of each
    b = layer.buffers(2, 1)
    for _ in range(3):
        layer.step(torch.randn(2, example.DIM, dtype=torch.bfloat16, device="cuda:0"),
                   torch.ones(2, dtype=torch.int32, device="cuda:0"), b)
    key = b["qkv"][:, example.Q + example.LATENT:example.Q + example.KV].double()
    slots = b["plan"].slot_map.long()
    held = layer.cache[2].flatten(0, 1)[slots].double()
    assert torch.allclose(held.norm(dim=1), key.norm(dim=1), rtol=2.0 ** -8)
    assert torch.allclose(b["q_rope"].double().norm(dim=2),
                          b["qkv"][:, :example.Q].unflatten(1, (example.HEADS, -1))[..., example.NOPE:].double().norm(dim=2),
                          rtol=2.0 ** -8)
    # as the example's own test: outputs are rounded to bf16 once, weights to fp16
    assert example.main(["--requests", "5", "--steps", "4", "--factor", str(factor)]) < 2.0 ** -8
