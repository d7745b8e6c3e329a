"""examples/paged_decode.py's layer: a request that is idle for some steps, or refused for want of
pages, goes on from the tokens it has."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import announce, dev

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


def test_idle_and_refused_requests_keep_their_tokens():
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    torch.manual_seed(3)
    layer = ex.Layer(3, 192, dev())
    pages = 3 * (192 // ex.PAGE)
    # the last step's third request would pass its row of the block table
    steps = [[70, 64, 1], [1, 0, 1], [0, 0, 1], [1, 1, 1], [1, 1, 190]]
    want = torch.zeros(3, dtype=torch.int64)
    for new in steps:
        n = torch.tensor(new)
        kept = n * (want + n <= 192)
        T = int(n.sum())
        b = layer.buffers(T, int(n.max()))
        announce(f"layer step {new}")
        layer.step(torch.randn(T, ex.DIM, dtype=torch.bfloat16, device=dev()), n.to(dev(), torch.int32), b)
        torch.cuda.synchronize()
        want += kept
        assert layer.ctx.cpu().tolist() == want.tolist(), f"lengths after {new}"
        taken = int(layer.free_head[0])
        assert taken == int((-(-want // ex.PAGE)).sum()) <= pages, "a page was taken twice"
        last = torch.cumsum(n, 0) - 1
        for r in range(3):
            if kept[r]:
                exact = layer.exact(b["qkv"][last[r], :ex.HEADS_Q * ex.WIDTH].view(ex.HEADS_Q, ex.WIDTH), r)
                err = (b["out"][last[r]].double() - exact).norm() / exact.norm()
                # the output is rounded to bf16 once: half of 2^-7 of an element at most
                assert err < 2.0 ** -8, f"request {r} after {new}"
