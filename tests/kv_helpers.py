"""Seeded paged caches, the library's calls on them, and the bounds of the attention tests."""
import numpy as np
import torch

import block_scaled_fp8_04_amd as bfp8
import kv_reference as ref
from gpu_helpers import canary_intact, dev, with_canary


def bf16(x):
    """float array -> bf16 tensor on the GPU."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).to(dev())


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev())


def host(t):
    return t.detach().cpu().numpy()


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


class Cache:
    """A pool with random finite codes and scales; pages of the requests are drawn at random, every
    byte behind a request's last token and every unused page is NaN."""

    def __init__(self, rng, kv_lens, H, B, dk, dv, spare=3, spread=3):
        need = [-(-int(n) // B) for n in kv_lens]
        P = sum(need) + spare
        self.k = rng.integers(0, 127, (P, H, B, dk), dtype=np.uint8) | \
            (rng.integers(0, 2, (P, H, B, dk), dtype=np.uint8) << 7)
        self.v = rng.integers(0, 127, (P, H, dv, B), dtype=np.uint8) | \
            (rng.integers(0, 2, (P, H, dv, B), dtype=np.uint8) << 7)
        # codes spread evenly over the binades: typical size 1 at scale 1, so logits stay small
        self.ks = (2.0 ** rng.integers(-6 - spread, -5, (P, H))).astype(np.float32)
        self.vs = (2.0 ** rng.integers(-spread, 1, (P, H))).astype(np.float32)
        order = rng.permutation(P)
        W = max(need, default=0) + 2
        self.table = rng.integers(-5, P + 5, (len(need), W)).astype(np.int32)    # stale entries
        used, at = np.zeros(P, bool), 0
        for r, n in enumerate(need):
            pages = order[at:at + n]
            at += n
            self.table[r, :n] = pages
            used[pages] = True
            tail = int(kv_lens[r]) - (n - 1) * B
            if n:
                self.k[pages[-1], :, tail:] = 0x7F
                self.v[pages[-1], :, :, tail:] = 0xFF
        self.k[~used], self.v[~used] = 0x7F, 0x7F
        self.ks[~used] = np.nan
        self.vs[~used] = np.nan
        self.arrays = (self.k, self.ks, self.v, self.vs)

    def gpu(self):
        return tuple(torch.from_numpy(x).to(dev()) for x in self.arrays)


def attend(q, cache, table, q_off, kv_lens, max_new, scale, workspace=True, lse=True):
    """The library's call with guard bands around its outputs; returns out, lse (tensors)."""
    T, Hq, dk = q.shape
    H, dv = cache[0].shape[1], cache[2].shape[2]
    R = len(kv_lens)
    raw_o, out, pad = with_canary((T, Hq, dv), torch.bfloat16)
    raw_l, ls, _ = with_canary((T, Hq), torch.float32)
    tiles = offsets([-(-max(int(n), 0) // 128) for n in kv_lens])
    ws = None
    if workspace:
        n = bfp8.bfp8_attn_paged_workspace_size(R, max_new, Hq, H, dk, dv)
        raw_w, ws, _ = with_canary((max(n, 16),), torch.uint8)
        ws.fill_(0xFF)                                     # NaN everywhere
    bfp8.bfp8_attn_paged(q, *cache, i32(table), i32(q_off), i32(kv_lens), i32(tiles), max_new, scale,
                         out, ls if lse else None, ws)
    torch.cuda.synchronize()
    assert canary_intact(raw_o, pad) and canary_intact(raw_l, pad), "wrote outside an output"
    assert not workspace or canary_intact(raw_w, pad), "wrote outside the workspace"
    return out, ls


def check_attention(out, lse, q, arrays, table, q_off, kv_lens, scale, what=""):
    """Elementwise and in the mean.  The bounds leave room for weights that are off by 2^-8 (the
    kernels' two terms of a weight stay far below: kv_terms.bound) and for the logits' fp32 error.
    The output's one bf16 rounding is 2^-8 of the result at most: 2^-9 stands here, and the room of
    the weights takes the rest."""
    want, want_lse, weight, slack = ref.attention(q, *arrays, table, q_off, kv_lens, scale)
    got, got_lse = f64(out), f64(lse)
    rows = ~np.isnan(want_lse)
    if not rows.any():
        return
    g, w, a = got[rows], want[rows], weight[rows]
    assert np.isfinite(g).all(), f"{what}: not finite"
    err = np.abs(g - w)
    bound = 2.0 ** -9 * np.abs(w) + (2.0 ** -8 + 2 * slack[rows][..., None]) * a + 1e-30
    assert (err <= bound).all(), f"{what}: worst err/bound {np.max(err / bound):.3f}"
    rms = lambda x: float(np.sqrt(np.mean(x ** 2)))                                  # noqa: E731
    assert rms(err) <= 2.0 ** -9 * (rms(w) + rms(a)) + 1e-30, f"{what}: rms error {rms(err):.3e}"
    wl, gl = want_lse[rows], got_lse[rows]
    dead = np.isinf(wl)
    assert np.array_equal(dead, np.isneginf(gl)), f"{what}: rows that see nothing"
    l_err = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, wl))
    l_bound = 2 * slack[rows] + 2.0 ** -20 * (1 + np.where(dead, 0, np.abs(wl)))
    assert (l_err <= l_bound).all(), f"{what}: lse off by {l_err.max():.3e}"
