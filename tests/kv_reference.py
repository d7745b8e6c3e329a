"""Plain 64-bit implementations of the paged-cache operators, by loops over requests, pages and
heads, from the definitions in include/bfp8.h.  Nothing here is shared with the library."""
import numpy as np

FLOOR = np.float32(1e-4)


def e4m3_values():
    """The 256 values of OCP e4m3 (0x7F and 0xFF are NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if (c & 127) == 127 else s * v
    return out


VALUES = e4m3_values()


def encode(x):
    """Nearest e4m3 code, ties to the even code, saturating at 448; the sign of zero is kept."""
    x = np.asarray(x, np.float64)
    pos = VALUES[:127]                                   # ascending
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - pos[lo], pos[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return np.where(np.signbit(x), code | 128, code).astype(np.uint8)


def scale_of(amax):
    """max(amax, 1e-4f) / 448 in fp32, rounded up to a power of two."""
    y = float(np.float32(max(np.float32(amax), FLOOR)) / np.float32(448.0))
    m, e = np.frexp(y)
    return float(np.ldexp(1.0, int(e) - (1 if m == 0.5 else 0)))


def plan(ctx, new, free, head, table, B, T):
    """(q_offsets, kv_lens, tile_offsets, slot_map, positions, counts, table)."""
    R, W = table.shape
    table = table.copy()
    q_off, kv, tiles = np.zeros(R + 1, np.int64), np.zeros(R, np.int64), np.zeros(R + 1, np.int64)
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    start = wanted = taken = kept = 0
    left = max(len(free) - max(head, 0), 0)
    for r in range(R):
        c, n = int(ctx[r]), int(new[r])
        q_off[r] = min(start, T)
        first, start = start, start + max(n, 0)
        have, want = -(-c // B), -(-(c + n) // B)
        ok = c >= 0 and n >= 0 and want <= W
        need = want - have if ok else 0
        wanted += need
        ok = ok and start <= T and (need == 0 or wanted <= left)
        if ok:
            kept += 1
            for j in range(need):
                table[r, have + j] = free[max(head, 0) + taken + j]
            taken += need
            for i in range(n):
                p = c + i
                pos[first + i] = p
                slots[first + i] = int(table[r, p // B]) * B + p % B
            kv[r] = c + n if n else 0
        tiles[r + 1] = tiles[r] + -(-int(kv[r]) // 128)
    q_off[R] = min(start, T)
    counts = np.array([q_off[R], max(head, 0) + taken, kept, wanted])
    return q_off, kv, tiles, slots, pos, counts, table


def append(k, v, slots, k_cache, k_scales, v_cache, v_scales):
    """k, v float64 [T, H, D] (bf16 values); returns the four updated arrays."""
    k_cache, k_scales, v_cache, v_scales = (x.copy() for x in (k_cache, k_scales, v_cache, v_scales))
    P, H, B, _ = k_cache.shape
    touched = {}
    for t, s in enumerate(slots):
        if 0 <= s < P * B:
            touched.setdefault(int(s) // B, []).append((int(s) % B, t))
    for page, places in touched.items():
        first = min(o for o, _ in places)
        ts = [t for _, t in places]
        offs = [o for o, _ in places]
        for h in range(H):
            x, y = k[ts, h], v[ts, h]
            bad_value = ~np.isfinite(y).all(axis=1)
            for x_, cache, scales, keys in ((x, k_cache, k_scales, True), (y, v_cache, v_scales, False)):
                fin = np.isfinite(x_)
                amax = np.abs(x_[fin]).max() if fin.any() else 0.0
                s, old = scale_of(amax), float(scales[page, h])
                view = cache[page, h] if keys else cache[page, h].T
                if first > 0:
                    s = max(s, old)
                    if s > old:
                        held = VALUES[view[:first]]
                        nan = np.isnan(held)
                        view[:first] = np.where(nan, view[:first], encode(np.where(nan, 0, held) * (old / s)))
                codes = encode(np.where(fin, x_, 0.0) / s)
                if keys:
                    codes = np.where(fin, codes, 0x7F)
                    codes[bad_value] = 0x7F
                else:
                    codes = np.where(fin, codes, 0)
                view[offs] = codes
                scales[page, h] = s
    return k_cache, k_scales, v_cache, v_scales


def attention(q, k_cache, k_scales, v_cache, v_scales, table, q_off, kv_lens, scale):
    """q float64 [T, Hq, Dk].  Returns out, lse and, per output, the mean of |v| under the same
    weights; rows of no request are NaN."""
    T, Hq, dk = q.shape
    P, H, B, _ = k_cache.shape
    dv = v_cache.shape[2]
    G = Hq // H
    out, lse = np.full((T, Hq, dv), np.nan), np.full((T, Hq), np.nan)
    weight, slack = np.zeros((T, Hq, dv)), np.zeros((T, Hq))
    for r, n in enumerate(int(x) for x in kv_lens):
        a, b = int(q_off[r]), int(q_off[r + 1])
        if b <= a:
            continue
        pages = table[r, :-(-n // B)].astype(np.int64)
        for h in range(H):
            k = (VALUES[k_cache[pages, h]] * k_scales[pages, h][:, None, None]).reshape(-1, dk)[:n]
            v = VALUES[v_cache[pages, h]] * v_scales[pages, h][:, None, None]
            v = v.transpose(0, 2, 1).reshape(-1, dv)[:n]
            for t in range(a, b):
                seen = min(n, n - (b - a) + (t - a) + 1)
                for j in range(h * G, h * G + G):
                    if seen <= 0:
                        out[t, j], lse[t, j] = 0.0, -np.inf
                        continue
                    z = scale * (k[:seen] @ q[t, j])
                    m = z.max()
                    p = np.exp(z - m)
                    out[t, j] = p @ v[:seen] / p.sum()
                    lse[t, j] = m + np.log(p.sum())
                    weight[t, j] = p @ np.abs(v[:seen]) / p.sum()
                    # fp32 accumulation of the logits' terms, and the exponent's rounding
                    slack[t, j] = abs(scale) * (np.abs(k[:seen]) @ np.abs(q[t, j])).max() * 2.0 ** -20
    return out, lse, weight, slack
