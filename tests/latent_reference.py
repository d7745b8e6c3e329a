"""Plain 64-bit implementations of rotary positions and of the latent cache's operators, by loops over
tokens and requests, from the definitions in include/bfp8.h.  Nothing here is shared with the library."""
import numpy as np

from kv_reference import VALUES, encode, scale_of

LATENT, ROPE = 512, 64


def rotate(x, positions, inv_freq, interleaved, amplitude):
    """x float64 [T, H, D]; angles positions * inv_freq [D / 2]."""
    out = np.array(x, np.float64)
    half = x.shape[-1] // 2
    for t, p in enumerate(positions):
        if p < 0:
            continue
        w = float(p) * np.asarray(inv_freq, np.float64)
        a, b = (x[t, :, 0::2], x[t, :, 1::2]) if interleaved else (x[t, :, :half], x[t, :, half:])
        lo, hi = amplitude * (a * np.cos(w) - b * np.sin(w)), amplitude * (a * np.sin(w) + b * np.cos(w))
        if interleaved:
            out[t, :, 0::2], out[t, :, 1::2] = lo, hi
        else:
            out[t, :, :half], out[t, :, half:] = lo, hi
    return out


def norm(c, weight, eps):
    if weight is None:
        return c
    return c / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps) * weight


def append(kv, slots, positions, inv_freq, interleaved, amplitude, weight, eps, num_slots):
    """{slot: (y [512], scale, rotated [64])} of the tokens that are stored; scale is NaN for a poisoned one."""
    y = norm(kv[:, :LATENT], weight, eps)
    k = rotate(kv[:, None, LATENT:], np.maximum(positions, 0), inv_freq, interleaved, amplitude)[:, 0]
    held = {}
    for t, s in enumerate(slots):
        if not 0 <= s < num_slots:
            continue
        bad = not (np.isfinite(y[t]).all() and np.isfinite(k[t]).all()) or np.abs(y[t]).max() >= 2.0 ** 127
        held[int(s)] = (y[t], np.nan if bad else scale_of(np.abs(y[t]).max()), k[t])
    return held


def tokens(codes, scales, rope, table_row, n):
    """A request's first n tokens: values [n, 512], scales [n], rotated dims [n, 64]."""
    B = codes.shape[1]
    at = np.arange(n)
    page = np.clip(table_row[at // B].astype(np.int64), 0, codes.shape[0] - 1)
    s = scales[page, at % B].astype(np.float64)
    return VALUES[codes[page, at % B]] * s[:, None], s, rope[page, at % B].astype(np.float64)


def attention(ql, qr, cache, table, q_off, kv_lens, scale):
    """ql [T, H, 512], qr [T, H, 64] float64.  Returns out, lse, and the bounds of their errors but for the
    output's own rounding; rows of no request are NaN.

    Logits: a row's 576 products are summed in fp32 over 36 steps of 16, each off by 2^-24 of the sum of
    their sizes at most, 2^-24 more for each step's own sum: 2^-18 of it in all; the exponent x log2 e + e_t
    and its power are off by 2^-22 of their size (e_t is below 32 here) and 2^-22.  A weight's rounding to
    fp16 loses 2^-11 of it at most, or 2^-25 absolutely, where the largest is above 2^-1; the reference may
    be one step above the maximum: 2^-23 of the largest contribution p_t s_t, per unit of each code."""
    T, H, _ = ql.shape
    out, lse = np.full((T, H, LATENT), np.nan), np.full((T, H), np.nan)
    bound, lse_bound = np.zeros((T, H, LATENT)), np.zeros((T, H))
    for r, n in enumerate(int(x) for x in kv_lens):
        a, b = int(q_off[r]), int(q_off[r + 1])
        if b <= a:
            continue
        c, s, k = tokens(*cache, table[r], n) if n > 0 else (np.zeros((0, LATENT)), np.zeros(0), np.zeros((0, ROPE)))
        for t in range(a, b):
            seen = max(0, min(n, n - (b - a) + (t - a) + 1))
            if seen == 0:
                out[t], lse[t] = 0.0, -np.inf
                continue
            ct, kt, st = c[:seen], k[:seen], s[:seen]
            z = scale * (ql[t] @ ct.T + qr[t] @ kt.T)                                   # [H, seen]
            m = z.max(axis=1, keepdims=True)
            p = np.exp(z - m)
            norm_ = p.sum(axis=1, keepdims=True)
            out[t], lse[t] = p @ ct / norm_, (m + np.log(norm_))[:, 0]
            size = abs(scale) * (np.abs(ql[t]) @ np.abs(ct).T + np.abs(qr[t]) @ np.abs(kt).T).max(axis=1)
            slack = 2.0 ** -18 * size + 2.0 ** -22 * (np.abs(z).max(axis=1) * 1.5 + 33)
            big = (p * st).max(axis=1, keepdims=True)
            bound[t] = (2.0 ** -11 + 2 * slack)[:, None] * (p @ np.abs(ct) / norm_) + \
                2.0 ** -23 * big * (np.abs(ct) / st[:, None]).sum(axis=0)[None] / norm_
            lse_bound[t] = slack + 2.0 ** -21 * (1 + np.abs(lse[t]))
    return out, lse, bound, lse_bound
