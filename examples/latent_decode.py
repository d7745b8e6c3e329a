"""One layer of latent attention serving a batch, in the absorbed form.

    python examples/latent_decode.py [--requests 16] [--steps 8] [--factor 1]

Every step plans its pages (bfp8_kv_plan), projects the new tokens' hidden states to queries and to
the shared latent (bfp8_linear_fp8), rotates the queries (bfp8_rope), brings the latents into the
paged cache, normed, rotated and quantized (bfp8_latent_append), and attends over them
(bfp8_attn_latent) with the key and value projections of the heads absorbed into the queries and the
outputs.  The first step takes the requests' prompts, the later ones a token each; these are one
captured graph that carries lengths and the free list along by itself.  At the end the last step's
attention is compared with float64 over the latents that bfp8_latent_gather reads back.

With --factor, positions are stretched (bfp8.rope_frequencies).  The amplitude that belongs to them
is one of the whole logit: the rotated dims are only a part of it, so they are turned as they are, and
its square goes into the scale.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_04_amd as bfp8                      # noqa: E402
from block_scaled_fp8_04_amd import synth                   # noqa: E402

DIM, HEADS, NOPE, ROPE, VALUE, LATENT, PAGE = 1024, 16, 128, 64, 128, 512, 64
Q, KV = HEADS * (NOPE + ROPE), LATENT + ROPE
KV_ROWS = -(-KV // 128) * 128                                # whole scale blocks: the last rows are not used
SCALE = (NOPE + ROPE) ** -0.5


class Layer:
    """The layer's weights, its cache, and the buffers of a step of T tokens (of R requests)."""

    def __init__(self, R, max_len, factor, dev):
        self.w_in = [t.to(dev) for t in synth.weight(Q + KV_ROWS, DIM, 1, 2, -10.0, -4.0)]
        self.w_out = [t.to(dev) for t in synth.weight(DIM, HEADS * VALUE, 3, 4, -10.0, -4.0)]
        # keys and values of a head from the latent: [H, 128, 512], and [H, 512, 128]
        self.w_k = (torch.randn(HEADS, NOPE, LATENT, device=dev) * LATENT ** -0.5).bfloat16()
        self.w_v = (torch.randn(HEADS, LATENT, VALUE, device=dev) * LATENT ** -0.5).bfloat16()
        self.norm = torch.ones(LATENT, dtype=torch.bfloat16, device=dev)
        self.freq, amplitude = bfp8.rope_frequencies(ROPE, factor=factor, device=dev)
        self.scale = SCALE * amplitude ** 2
        pages = R * -(-max_len // PAGE)
        self.cache = bfp8.latent_cache_buffers(pages, PAGE, dev)
        self.table = torch.zeros(R, -(-max_len // PAGE), dtype=torch.int32, device=dev)
        self.free = torch.randperm(pages, device=dev).to(torch.int32)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(R, dtype=torch.int32, device=dev)
        self.R = R

    def buffers(self, T, max_new):
        dev = self.ctx.device
        empty = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device=dev)        # noqa: E731
        return {"plan": bfp8.kv_plan_buffers(self.R, T, dev), "qkv": empty(T, Q + KV_ROWS),
                "q_rope": empty(T, HEADS, ROPE), "out": torch.zeros_like(empty(T, HEADS, LATENT)), "y": empty(T, DIM),
                "ws_in": bfp8.linear_workspace(T, Q + KV_ROWS, DIM, dev),
                "ws_out": bfp8.linear_workspace(T, DIM, HEADS * VALUE, dev),
                "ws": bfp8.attn_latent_workspace(self.R, max_new, HEADS, dev), "max_new": max_new}

    def step(self, x, new_lens, b):
        """x bf16 [T, DIM], the requests' new tokens one after the other; returns b["y"]."""
        plan = b["plan"]
        bfp8.bfp8_kv_plan(self.ctx, new_lens, self.free, self.table, PAGE, plan, self.free_head)
        bfp8.bfp8_linear_fp8(x, *self.w_in, b["qkv"], b["ws_in"])
        q = b["qkv"][:, :Q].unflatten(1, (HEADS, NOPE + ROPE))
        bfp8.bfp8_rope(q[..., NOPE:], plan.positions, self.freq, b["q_rope"], True)
        bfp8.bfp8_latent_append(b["qkv"][:, Q:Q + KV], plan.slot_map, plan.positions, self.freq, *self.cache,
                                norm_weight=self.norm, interleaved=True)
        b["q_latent"] = (q[..., :NOPE].transpose(0, 1).contiguous() @ self.w_k).transpose(0, 1)     # [T, H, 512]
        bfp8.bfp8_attn_latent(b["q_latent"], b["q_rope"], *self.cache, self.table, plan.q_offsets, plan.kv_lens,
                              b["max_new"], self.scale, b["out"], None, b["ws"])
        values = (b["out"].transpose(0, 1).contiguous() @ self.w_v).transpose(0, 1)                 # [T, H, 128]
        bfp8.bfp8_linear_fp8(values.flatten(1), *self.w_out, b["y"], b["ws_out"])
        # an idle or refused request has a kv_len of 0 and keeps what it has
        self.ctx.copy_(torch.where(plan.kv_lens > 0, plan.kv_lens, self.ctx))
        self.free_head.copy_(plan.counts[1:2])
        return b["y"]

    def exact(self, b):
        """The last queries' attention in float64, [R, H, 512], over the cached tokens read back."""
        ends = torch.nn.functional.pad(self.ctx.cumsum(0), (1, 0)).to(torch.int32)
        latent, rope = (t.double() for t in bfp8.latent_gather(self.cache, self.table, ends, int(ends[-1])))
        out = []
        for r in range(self.R):
            c, k = latent[ends[r]:ends[r + 1]], rope[ends[r]:ends[r + 1]]
            s = (b["q_latent"][r].double() @ c.T + b["q_rope"][r].double() @ k.T) * self.scale
            out.append(s.softmax(-1) @ c)
        return torch.stack(out)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--factor", type=float, default=1.0)
    args = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    torch.manual_seed(0)
    R = args.requests
    prompts = torch.randint(1, 400, (R,))
    T = int(prompts.sum())
    layer = Layer(R, 400 + args.steps + 1, args.factor, dev)

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

    want = layer.exact(b)
    worst = ((b["out"].double() - want).norm(dim=(1, 2)) / want.norm(dim=(1, 2))).max().item()
    print(f"{R} requests, prompts of {int(prompts.min())} to {int(prompts.max())} tokens, {args.steps} "
          f"steps at {took * 1e6:.0f} us; attention is off by {worst:.2e} of its norm at most")
    return worst


if __name__ == "__main__":
    # the output is rounded to bf16 once: half of 2^-7 of an element at most
    sys.exit(0 if main() < 2.0 ** -8 else 1)
