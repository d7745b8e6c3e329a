"""The allocating calls on another stream than the current one, which is kept busy meanwhile: the
same results as on the current stream, at once and after that stream has ended its work."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
from gpu_helpers import announce, dev
from kv_helpers import Cache, bf16, i32, offsets

pytestmark = pytest.mark.gpu


def busy():
    """A few tens of milliseconds of work on the current stream."""
    x = torch.randn(8192, 8192, dtype=torch.bfloat16, device=dev())
    for _ in range(40):
        x = (x @ x).clamp_(-1, 1)
    return x


def on_side_stream(call, raw):
    """call(stream) on a new stream; the results read there, and again when all work has ended."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    out = call(s.cuda_stream if raw else s)
    # memory the call has dropped, if it were the current stream's, would be taken here
    junk = [torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=dev()) for _ in range(4)]
    with torch.cuda.stream(s):
        early = [t.clone() for t in out]
    torch.cuda.synchronize()
    del junk
    return early, out


def check(call, what):
    want = call(None)
    torch.cuda.synchronize()
    for raw in (False, True):
        announce(f"{what} on a side stream, raw handle {raw}")
        early, late = on_side_stream(call, raw)
        for e, l, w in zip(early, late, want):
            assert torch.equal(e.view(torch.uint8), w.view(torch.uint8)), f"{what}: read on its stream"
            assert torch.equal(l.view(torch.uint8), w.view(torch.uint8)), f"{what}: read at the end"
    announce(f"{what} on the default stream's handle")
    got = call(0)
    torch.cuda.synchronize()
    assert all(torch.equal(g.view(torch.uint8), w.view(torch.uint8)) for g, w in zip(got, want))


@pytest.mark.parametrize("new", [1, 40])
def test_attention(new):
    # 1: partial sums of the long requests go through the workspace; 40: parts of blocks do
    rng = np.random.default_rng(new)
    kv = [5000, 40, 777]
    cache = Cache(rng, kv, 2, 64, 128, 128)
    q_off = offsets([new] * 3)
    plan = bfp8.KVPlan(i32(q_off), i32(kv), i32(offsets([-(-n // 128) for n in kv])), None, None, None)
    q = bf16(rng.standard_normal((3 * new + 2, 8, 128)))         # two rows of no request
    gpu, table = cache.gpu(), i32(np.clip(cache.table, 0, None))
    check(lambda s: [bfp8.attn_paged(q, gpu, table, plan, new, stream=s)], f"attention, {new} new")


def test_plan():
    free = i32(np.arange(300, 400))
    ctx, new = i32([0, 31, 64, 100, 7]), i32([70, 1, 0, 1, 3])
    table = i32(np.arange(40).reshape(5, 8))

    def call(s):
        tab = table.clone()
        torch.cuda.synchronize()                             # the input is written
        return [*bfp8.kv_plan(ctx, new, free, tab, 32, 80, stream=s), tab]
    check(call, "plan")


def test_linear():
    from block_scaled_fp8_04_amd import synth

    w, s_w = (t.to(dev()) for t in synth.weight(512, 1024, 1, 2, -10.0, -4.0))
    x = torch.randn(300, 1024, dtype=torch.bfloat16, device=dev())
    check(lambda s: [bfp8.linear_fp8(x, w, s_w, stream=s), *bfp8.act_quant(x, s)], "linear")
