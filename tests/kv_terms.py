"""Attention over the paged cache held to the precision the library states: a 64-bit reference that
takes a request's queries at once, the bound that follows from the stated roundings, and caches whose
weighted values cancel, so that every bit of a weight shows."""
import numpy as np

import kv_reference as ref

# bits of the e4m3 codes of 1.0 and -1.0
ONE, MINUS_ONE = 0x38, 0xB8


def attention(q, k_cache, k_scales, v_cache, v_scales, table, q_off, kv_lens, scale):
    """What kv_reference.attention returns, one product per request and KV head."""
    T, Hq, dk = q.shape
    H, B, dv = k_cache.shape[1], k_cache.shape[2], v_cache.shape[2]
    G = Hq // H
    out, lse = np.full((T, Hq, dv), np.nan), np.full((T, Hq), np.nan)
    weight, slack = np.zeros((T, Hq, dv)), np.zeros((T, Hq))
    for r, n in enumerate(int(x) for x in kv_lens):
        a, b = int(q_off[r]), int(q_off[r + 1])
        if b <= a:
            continue
        out[a:b], lse[a:b] = 0.0, -np.inf
        pages = table[r, :-(-n // B)].astype(np.int64)
        seen = np.arange(n)[None, :] <= (n - (b - a) + np.arange(b - a))[:, None]
        rows = np.nonzero(seen.any(axis=1))[0]
        if not rows.size:
            continue
        for h in range(H):
            k = (ref.VALUES[k_cache[pages, h]] * k_scales[pages, h][:, None, None]).reshape(-1, dk)[:n]
            v = ref.VALUES[v_cache[pages, h]] * v_scales[pages, h][:, None, None]
            v = v.transpose(0, 2, 1).reshape(-1, dv)[:n]
            for j in range(h * G, h * G + G):
                x = q[a + rows, j]
                z = np.where(seen[rows], scale * (x @ k.T), -np.inf)
                m = z.max(axis=1, keepdims=True)
                p = np.exp(z - m)
                norm = p.sum(axis=1, keepdims=True)
                out[a + rows, j] = p @ v / norm
                lse[a + rows, j] = (m + np.log(norm))[:, 0]
                weight[a + rows, j] = p @ np.abs(v) / norm
                size = np.where(seen[rows], np.abs(x) @ np.abs(k).T, 0.0).max(axis=1)
                slack[a + rows, j] = abs(scale) * size * 2.0 ** -20
    return out, lse, weight, slack


def bound(want, weight, slack):
    """How far an output may be from `want`, with `weight` the mean of |v| under the same weights.

    2^-8 |want|     the output is rounded to bf16 once: eight significant bits, half a unit of the last
    2^-16 weight    p enters as its bf16 rounding and the bf16 rounding of what that leaves
    2^-16 weight    the exponent s c - m, below 128 where a weight counts, is rounded to 24 bits: p is off
                    by 2^-17.5 of itself, above and below the line of the mean
    2^-15 weight    fp32 sums: two products for 16 tokens at least, each rounded at 2^-24; 4096 tokens in
                    a row of one accumulator, or as many as 512 parts of shorter rows, stay below this
    2 slack weight  the logits' fp32 sums, above and below the line
    """
    return 2.0 ** -8 * np.abs(want) + (2.0 ** -14 + 2.0 * slack[..., None]) * weight * (1 + 2.0 ** -7) + 1e-30


def check(out, lse, q, arrays, table, q_off, kv_lens, scale, what=""):
    """float64 out [T, Hq, Dv] and lse [T, Hq] against the reference; returns the worst err / bound."""
    want, want_lse, weight, slack = attention(q, *arrays, table, q_off, kv_lens, scale)
    rows = ~np.isnan(want_lse)
    g, w = out[rows], want[rows]
    assert np.isfinite(g).all(), f"{what}: not finite"
    worst = float((np.abs(g - w) / bound(w, weight[rows], slack[rows])).max(initial=0.0))
    assert worst <= 1.0, f"{what}: worst err/bound {worst:.3f}"
    wl, gl = want_lse[rows], lse[rows]
    dead = np.isinf(wl)
    assert np.array_equal(dead, np.isneginf(gl)), f"{what}: rows that see nothing"
    l_err = np.abs(np.where(dead, 0, gl) - np.where(dead, 0, wl))
    # fp32: the statistic's own rounding, and its sum's
    l_bound = 2 * slack[rows] + 2.0 ** -20 * (1 + np.where(dead, 0, np.abs(wl)))
    assert (l_err <= l_bound).all(), f"{what}: lse off by {l_err.max():.3e}"
    return worst


class Cancelling:
    """One request of n tokens, one KV head: tokens at .. at + 63 have the unit vectors as keys, the
    others zero keys; values of tokens 2 u and 2 u + 1 of them are opposite.  Row (x, u) of the
    queries answers to that pair alone, with logits of about 15 that are 1/16 apart, so that the
    weighted values nearly cancel and the outputs are a 32nd of the values: what either weight
    lacks shows.  Everywhere else weights are e^-15 of those."""

    HOT, PAIRS = 64, 32

    def __init__(self, seed, at, n, B, dk, dv, draws):
        rng = np.random.default_rng(seed)
        assert at % 2 == 0 and at + self.HOT <= n and dk >= self.HOT
        P = -(-n // B) + 2
        order = rng.permutation(P)
        self.table = order[None, :-(-n // B)].astype(np.int32)
        keys, values = np.zeros((P * B, dk), np.uint8), rng.integers(0, 127, (P * B, dv), dtype=np.uint8)
        keys[at + np.arange(self.HOT), np.arange(self.HOT)] = ONE
        # sizes of 1 to 1.875, so that no row is another's rounding error
        values[at:at + self.HOT:2] = ONE + rng.integers(0, 8, (self.PAIRS, dv), dtype=np.uint8)
        values[at + 1:at + self.HOT:2] = values[at:at + self.HOT:2] | 0x80
        self.k, self.v = np.zeros((P, 1, B, dk), np.uint8), np.zeros((P, 1, dv, B), np.uint8)
        for i, p in enumerate(self.table[0]):
            self.k[p, 0] = keys[i * B:(i + 1) * B]
            self.v[p, 0] = values[i * B:(i + 1) * B].T
        self.ks = np.ones((P, 1), np.float32)
        self.vs = np.ones((P, 1), np.float32)
        self.arrays = (self.k, self.ks, self.v, self.vs)
        self.at, self.n = at, n
        # logits of 14 to 15.9375 in steps of 1/16, exact in bf16; the draws differ in all pairs
        base = 14 + rng.permuted(np.tile(np.arange(1, 31) / 16, (self.PAIRS, 1)), axis=1)[:, :draws]
        self.q = np.zeros((draws, self.PAIRS, dk))
        u = np.arange(self.PAIRS)
        swap = rng.integers(0, 2, (draws, self.PAIRS)) / 16
        self.q[:, u, 2 * u] = base.T + swap
        self.q[:, u, 2 * u + 1] = base.T + 1 / 16 - swap
