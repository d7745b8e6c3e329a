"""Seeded latent caches, the library's attention call on them, and its check."""
import numpy as np
import torch

import block_scaled_fp8_04_amd as bfp8
import latent_reference as ref
from gpu_helpers import canary_intact, dev, with_canary
from kv_helpers import bf16, f64, i32


class LatentCache:
    """A pool with random finite codes and scales; the requests' pages are drawn at random, every byte
    behind a request's last token and every unused page is NaN."""

    def __init__(self, rng, kv_lens, B, spare=3, spread=3):
        need = [-(-int(n) // B) for n in kv_lens]
        P = sum(need) + spare
        # codes spread evenly over the binades: typical size 1 at scale 1, so logits stay small
        self.codes = rng.integers(0, 127, (P, B, ref.LATENT), dtype=np.uint8) | \
            (rng.integers(0, 2, (P, B, ref.LATENT), dtype=np.uint8) << 7)
        self.scales = (2.0 ** rng.integers(-6 - spread, -5, (P, B))).astype(np.float32)
        self.rope = f64(bf16(rng.standard_normal((P, B, ref.ROPE))))
        order = rng.permutation(P)
        W = max(need, default=0) + 2
        self.table = rng.integers(-5, P + 5, (len(need), W)).astype(np.int32)          # stale entries
        used, at = np.zeros(P, bool), 0
        for r, n in enumerate(need):
            pages = order[at:at + n]
            at += n
            self.table[r, :n] = pages
            used[pages] = True
            tail = int(kv_lens[r]) - (n - 1) * B
            if n:
                self.codes[pages[-1], tail:] = 0xFF
                self.scales[pages[-1], tail:] = np.nan
                self.rope[pages[-1], tail:] = np.nan
        self.codes[~used], self.scales[~used], self.rope[~used] = 0x7F, np.nan, np.nan
        self.used = used

    @property
    def arrays(self):
        return self.codes, self.scales, self.rope

    def gpu(self):
        return (torch.from_numpy(self.codes).to(dev()), torch.from_numpy(self.scales).to(dev()),
                torch.from_numpy(self.rope).to(torch.bfloat16).to(dev()))


def queries(rng, T, H, size=0.05):
    return bf16(size * rng.standard_normal((T, H, ref.LATENT))), bf16(rng.standard_normal((T, H, ref.ROPE)))


def attend(ql, qr, cache, table, q_off, kv_lens, max_new, scale, workspace=True, lse=True):
    """The library's call with guard bands around its outputs; returns out, lse (tensors)."""
    T, H, _ = ql.shape
    raw_o, out, pad = with_canary((T, H, ref.LATENT), torch.bfloat16)
    raw_l, ls, _ = with_canary((T, H), torch.float32)
    ws = None
    if workspace:
        n = bfp8.bfp8_attn_latent_workspace_size(len(kv_lens), max_new, H)
        raw_w, ws, _ = with_canary((max(n, 16),), torch.uint8)
        ws.fill_(0xFF)                                     # NaN everywhere
    bfp8.bfp8_attn_latent(ql, qr, *cache, i32(table), i32(q_off), i32(kv_lens), max_new, scale, out,
                          ls if lse else None, ws)
    torch.cuda.synchronize()
    assert canary_intact(raw_o, pad) and canary_intact(raw_l, pad), "wrote outside an output"
    assert not workspace or canary_intact(raw_w, pad), "wrote outside the workspace"
    return out, ls


def check(out, lse, ql, qr, arrays, table, q_off, kv_lens, scale, what="", rows=None):
    """Elementwise: the output's rounding, 2^-8 of it at most, on top of the reference's bounds."""
    want, want_lse, bound, lse_bound = ref.attention(f64(ql), f64(qr), arrays, table, q_off, kv_lens, scale)
    got, got_lse = f64(out), f64(lse)
    live = ~np.isnan(want_lse)
    if rows is not None:
        live &= rows
    if not live.any():
        return 0.0
    g, w, b = got[live], want[live], bound[live]
    assert np.isfinite(g).all(), f"{what}: not finite"
    b = b + 2.0 ** -8 * np.abs(w) + 1e-30
    worst = np.max(np.abs(g - w) / b)
    assert worst <= 1, f"{what}: worst err/bound {worst:.3f}"
    wl, gl = want_lse[live], got_lse[live]
    dead = np.isinf(wl)
    assert np.array_equal(dead, np.isneginf(gl)), f"{what}: rows that see nothing"
    err = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, wl))
    assert (err <= lse_bound[live] + 1e-30).all(), f"{what}: lse off by {err.max():.3e}"
    return worst
