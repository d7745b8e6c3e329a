"""One attention layer serving a batch: FP8 projections around a paged e4m3 cache.

    python examples/paged_decode.py [--requests 16] [--steps 8]

Every step plans its pages on the GPU (bfp8_kv_plan), projects the new tokens' hidden states
(bfp8_linear_fp8), quantizes their keys and values into the cache (bfp8_kv_append) and attends
over it (bfp8_attn_paged).  The first step takes the requests' prompts, the later ones a token
each; these are one captured graph that carries lengths and the free list along by itself.  At
the end the last step's attention is compared with float64 over the widened cache.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_04_amd as bfp8                      # noqa: E402
from block_scaled_fp8_04_amd import synth                   # noqa: E402

DIM, HEADS_Q, HEADS, WIDTH, PAGE = 1024, 16, 4, 128, 64
QKV = (HEADS_Q + 2 * HEADS) * WIDTH


class Layer:
    """The layer's weights, its cache, and the buffers of a step of T tokens (of R requests)."""

    def __init__(self, R, max_len, dev):
        self.w_qkv = [t.to(dev) for t in synth.weight(QKV, DIM, 1, 2, -10.0, -4.0)]
        self.w_out = [t.to(dev) for t in synth.weight(DIM, HEADS_Q * WIDTH, 3, 4, -10.0, -4.0)]
        pages = R * -(-max_len // PAGE)
        self.cache = bfp8.kv_cache_buffers(pages, HEADS, PAGE, WIDTH, WIDTH, dev)
        self.table = torch.zeros(R, -(-max_len // PAGE), dtype=torch.int32, device=dev)
        self.free = torch.randperm(pages, device=dev).to(torch.int32)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(R, dtype=torch.int32, device=dev)
        self.R = R

    def buffers(self, T, max_new):
        dev = self.ctx.device
        return {"plan": bfp8.kv_plan_buffers(self.R, T, dev),
                "qkv": torch.empty(T, QKV, dtype=torch.bfloat16, device=dev),
                "out": torch.zeros(T, HEADS_Q, WIDTH, dtype=torch.bfloat16, device=dev),
                "y": torch.empty(T, DIM, dtype=torch.bfloat16, device=dev),
                "ws_qkv": bfp8.linear_workspace(T, QKV, DIM, dev),
                "ws_out": bfp8.linear_workspace(T, DIM, HEADS_Q * WIDTH, dev),
                "ws": bfp8.attn_paged_workspace(self.R, max_new, HEADS_Q, HEADS, WIDTH, WIDTH, dev),
                "max_new": max_new}

    def step(self, x, new_lens, b):
        """x bf16 [T, DIM], the requests' new tokens one after the other; returns b["y"]."""
        plan = b["plan"]
        bfp8.bfp8_kv_plan(self.ctx, new_lens, self.free, self.table, PAGE, plan, self.free_head)
        bfp8.bfp8_linear_fp8(x, *self.w_qkv, b["qkv"], b["ws_qkv"])
        q, k, v = (t.unflatten(1, (-1, WIDTH)) for t in
                   b["qkv"].split([HEADS_Q * WIDTH, HEADS * WIDTH, HEADS * WIDTH], dim=1))
        bfp8.bfp8_kv_append(k, v, plan.slot_map, *self.cache)
        bfp8.bfp8_attn_paged(q, *self.cache, self.table, plan.q_offsets, plan.kv_lens, plan.tile_offsets,
                             b["max_new"], WIDTH ** -0.5, b["out"], None, b["ws"])
        bfp8.bfp8_linear_fp8(b["out"].flatten(1), *self.w_out, b["y"], b["ws_out"])
        # an idle or refused request has a kv_len of 0 and keeps what it has
        self.ctx.copy_(torch.where(plan.kv_lens > 0, plan.kv_lens, self.ctx))
        self.free_head.copy_(plan.counts[1:2])
        return b["y"]

    def exact(self, q, r):
        """Attention of request r's last query in float64, over its widened cache."""
        n = int(self.ctx[r])
        k, ks, v, vs = self.cache
        pages = self.table[r, :-(-n // PAGE)].long()
        wide = lambda c, s: c.view(torch.float8_e4m3fn).double() * s[..., None, None]       # noqa: E731
        keys = wide(k[pages], ks[pages]).transpose(0, 1).flatten(1, 2)[:, :n]                # [H, n, D]
        vals = wide(v[pages], vs[pages]).permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
        s = (q.double().view(HEADS, -1, WIDTH) * WIDTH ** -0.5) @ keys.transpose(1, 2)
        return (s.softmax(-1) @ vals).flatten(0, 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    torch.manual_seed(0)
    R = args.requests
    prompts = torch.randint(1, 400, (R,))
    T = int(prompts.sum())
    layer = Layer(R, 400 + args.steps + 1, dev)

    layer.step(torch.randn(T, DIM, dtype=torch.bfloat16, device=dev), prompts.to(dev, torch.int32),
               layer.buffers(T, int(prompts.max())))
    ones = torch.ones(R, dtype=torch.int32, device=dev)
    x = torch.randn(R, DIM, dtype=torch.bfloat16, device=dev)
    b = layer.buffers(R, 1)
    layer.step(x, ones, b)                                  # once outside the graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, ones, b)
    def feed_back():
        x.copy_(b["y"] / b["y"].float().pow(2).mean(1, keepdim=True).sqrt())

    feed_back()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.steps):
        graph.replay()
        feed_back()
    torch.cuda.synchronize()
    took = (time.perf_counter() - start) / max(args.steps, 1)
    assert layer.ctx.cpu().tolist() == (prompts + 1 + args.steps).tolist()

    worst = 0.0
    for r in range(R):
        want = layer.exact(b["qkv"][r, :HEADS_Q * WIDTH].view(HEADS_Q, WIDTH), r)
        worst = max(worst, ((b["out"][r].double() - want).norm() / want.norm()).item())
    print(f"{R} requests, prompts of {int(prompts.min())} to {int(prompts.max())} tokens, {args.steps} "
          f"steps at {took * 1e6:.0f} us; attention is off by {worst:.2e} of its norm at most")
    return worst


if __name__ == "__main__":
    # the output is rounded to bf16 once: half of 2^-7 of an element at most
    sys.exit(0 if main() < 2.0 ** -8 else 1)
