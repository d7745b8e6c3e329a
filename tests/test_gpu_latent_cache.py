"""Rotary positions and the latent cache's append and read back, against plain 64-bit implementations;
and a run of them with the plan and the attention, as a serving step uses them."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import latent_reference as ref
from gpu_helpers import announce, canary_intact, dev, with_canary
from kv_helpers import bf16, f64, host, i32, offsets
from kv_reference import VALUES
from latent_helpers import LatentCache, check, queries

pytestmark = pytest.mark.gpu

FILL = -23131


# --------------------------------------------------------------------------------- rope

def rope_bound(x, want, amplitude):
    """The output's rounding, 2^-8 of it, and the fp32 arithmetic's: a cosine or sine off by 2^-22 (half
    a turn reduced in 64 bits and rounded to fp32: 2^-25 pi; the function: two units of 2^-24) and three
    roundings, of pairs of which the larger is at most the two together."""
    D, size = x.shape[-1], np.abs(x)
    pair = np.maximum(size, np.maximum(np.roll(size, 1, -1), np.roll(size, -1, -1)))
    pair = np.maximum(pair, np.maximum(np.roll(size, D // 2, -1), np.roll(size, -D // 2, -1)))
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * abs(amplitude) * 2 * pair


def run_rope(x, positions, inv_freq, interleaved, amplitude, out):
    bfp8.bfp8_rope(x, i32(positions), torch.from_numpy(inv_freq).to(dev()), out, interleaved, amplitude)
    torch.cuda.synchronize()


def check_rope(x, positions, inv_freq, interleaved, amplitude, out):
    want = ref.rotate(f64(x), positions, inv_freq, interleaved, amplitude)
    err = np.abs(f64(out) - want)
    live = np.asarray(positions) >= 0
    bound = rope_bound(f64(x), want, amplitude)[live] + 1e-38
    assert (err[live] <= bound).all(), f"worst err/bound {np.max(err[live] / bound):.3f}"


def freq(D, base=1e4):
    return (base ** (-2.0 * np.arange(D // 2) / D)).astype(np.float32)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,D", [(1, 1, 2), (1, 128, 64), (3, 5, 6), (64, 128, 64), (65, 1, 64), (7, 3, 96),
                                   (2, 2, 1024), (1030, 2, 128), (2050, 1, 64), (5, 300, 64), (33, 40, 128),
                                   (3000, 1, 24), (2, 2000, 16)])
def test_rope(T, H, D, interleaved):
    rng = np.random.default_rng(T + H + D)
    x = bf16(rng.standard_normal((T, H, D)) * 4)
    pos = rng.integers(0, 200000, T)
    pos[0] = 0
    raw, out, pad = with_canary((T, H, D), torch.bfloat16)
    announce(f"rope {T} {H} {D} interleaved={interleaved}")
    run_rope(x, pos, freq(D), interleaved, 1.0, out)
    assert canary_intact(raw, pad)
    check_rope(x, pos, freq(D), interleaved, 1.0, out)
    run_rope(x, pos, freq(D), interleaved, 1.0, x)          # in place
    assert torch.equal(x, out)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("first", [0, 64, 3])
def test_rope_of_a_part(interleaved, first):
    """The rest of the head, and rows between the strides, are left alone; unaligned parts as well."""
    rng = np.random.default_rng(first)
    wide = bf16(rng.standard_normal((40, 9, 200)))
    pos = rng.integers(0, 5000, 40)
    before = wide.clone()
    part = wide[..., first:first + 64]
    run_rope(part, pos, freq(64), interleaved, 1.25, part)
    check_rope(before[..., first:first + 64], pos, freq(64), interleaved, 1.25, part)
    assert torch.equal(wide[..., :first], before[..., :first])
    assert torch.equal(wide[..., first + 64:], before[..., first + 64:])


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_far_positions_and_skipped_tokens(interleaved):
    rng = np.random.default_rng(5)
    pos = np.array([2 ** 31 - 1, 2 ** 30 + 7, -1, 16777217, 0, -2 ** 31, 999999999])
    x = bf16(rng.standard_normal((7, 4, 64)))
    raw, out, pad = with_canary((7, 4, 64), torch.bfloat16)
    run_rope(x, pos, freq(64), interleaved, 0.7, out)
    assert canary_intact(raw, pad)
    check_rope(x, pos, freq(64), interleaved, 0.7, out)
    assert (out[[2, 5]].view(torch.int16) == FILL).all()
    got = bfp8.rope(x, i32(pos), torch.from_numpy(freq(64)).to(dev()), interleaved, 0.7)
    assert torch.equal(got[[0, 1, 3, 4, 6]], out[[0, 1, 3, 4, 6]]) and (got[[2, 5]] == 0).all()


def test_rope_keeps_infinities_and_nan_in_their_pairs():
    x = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=dev())
    x[0, 0, 4], x[0, 1, 9] = float("inf"), float("nan")
    out = bfp8.rope(x, i32([3]), torch.from_numpy(freq(64)).to(dev()), True)
    bad = ~torch.isfinite(out[0])
    want = torch.zeros(2, 64, dtype=torch.bool, device=dev())
    want[0, 4:6], want[1, 8:10] = True, True
    assert torch.equal(bad, want)


# ------------------------------------------------------------------------------- append

def run_append(kv, slots, pos, inv_freq, cache, **kw):
    bfp8.bfp8_latent_append(kv, i32(slots), i32(pos), torch.from_numpy(inv_freq).to(dev()), *cache, **kw)
    torch.cuda.synchronize()


def check_append(kv, slots, pos, inv_freq, before, cache, interleaved, amplitude, weight, eps):
    """Slots of the map hold their tokens, all others what they held."""
    codes, scales, rope = (host(x) if x.dtype != torch.bfloat16 else f64(x) for x in cache)
    P, B, _ = codes.shape
    w = f64(weight) if weight is not None else None
    held = ref.append(f64(kv), slots, pos, inv_freq, interleaved, amplitude, w, eps, P * B)
    old = [host(x) if x.dtype != torch.bfloat16 else f64(x) for x in before]
    rest = np.ones(P * B, bool)
    for s, (y, scale, k) in held.items():
        rest[s] = False
        at = s // B, s % B
        if np.isnan(scale):
            assert np.isnan(scales[at]) and (codes[at] == 0).all() and (rope[at] == 0).all()
            continue
        # a maximum within its fp32 rounding of a power of two may take either scale
        top = np.abs(y).max() / 448
        near = abs(np.log2(max(top, 1e-30)) - round(np.log2(max(top, 1e-30)))) < 2.0 ** -18
        assert scales[at] == scale or (near and scales[at] in (scale / 2, scale * 2)), (scales[at], scale)
        # half a step of e4m3, and y's fp32 arithmetic (a sum of 512 squares, a root, two products)
        bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * scales[at]) + 2.0 ** -18 * np.abs(y)
        assert (np.abs(VALUES[codes[at]] * scales[at] - y) <= bound).all()
        # as rope_bound, the pairs' sizes bounded by the rotated ones'
        assert (np.abs(rope[at] - k) <= 2.0 ** -8 * np.abs(k) + 2.0 ** -18 * np.abs(k).max() + 1e-38).all()
    for new, was in zip((codes, scales, rope), old):
        assert np.array_equal(new.reshape((P * B,) + new.shape[2:])[rest], was.reshape((P * B,) + was.shape[2:])[rest],
                              equal_nan=True)


def pool(P, B, rng):
    cache = bfp8.latent_cache_buffers(P, B, dev())
    cache[0].copy_(torch.from_numpy(rng.integers(0, 256, tuple(cache[0].shape), dtype=np.uint8)))
    cache[1].fill_(float("nan"))
    cache[2].fill_(float("nan"))
    return cache


@pytest.mark.parametrize("B", [32, 64, 128])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("T", [1, 3, 200])
def test_append(T, normed, interleaved, B):
    rng = np.random.default_rng(T + B)
    P = T // B + 3
    slots = rng.permutation(P * B)[:T]
    pos = rng.integers(0, 100000, T)
    sizes = 2.0 ** rng.integers(-20, 20, (T, 1))
    kv = bf16(rng.standard_normal((T, 576)) * np.concatenate([np.broadcast_to(sizes, (T, 512)), np.ones((T, 64))], 1))
    weight = bf16(1 + 0.2 * rng.standard_normal(512)) if normed else None
    cache = pool(P, B, rng)
    before = [x.clone() for x in cache]
    run_append(kv, slots, pos, freq(64), cache, norm_weight=weight, eps=1e-6, interleaved=interleaved, amplitude=1.1)
    check_append(kv, slots, pos, freq(64), before, cache, interleaved, 1.1, weight, 1e-6)


@pytest.mark.parametrize("lead", [64, 3])
def test_append_strided_rows_and_skipped_slots(lead):
    rng = np.random.default_rng(lead)
    T, P, B = 70, 4, 32
    wide = bf16(rng.standard_normal((T, lead + 576 + (24 if lead == 64 else 5))))
    kv = wide[:, lead:lead + 576]
    slots = rng.permutation(P * B)[:T].astype(np.int64)
    slots[[0, 7, 69]] = [-1, P * B, 2 ** 31 - 1]
    pos = np.where(slots < 0, -1, rng.integers(0, 4000, T))
    cache = pool(P, B, rng)
    before = [x.clone() for x in cache]
    weight = bf16(1 + 0.2 * rng.standard_normal(512))
    run_append(kv, slots, pos, freq(64), cache, norm_weight=weight)
    check_append(kv, slots, pos, freq(64), before, cache, True, 1.0, weight, 1e-6)


def test_append_extremes():
    """All zeros, the smallest and largest values, powers of two, infinities and NaN in either part."""
    rng = np.random.default_rng(9)
    kv = rng.standard_normal((12, 576))
    kv[0] = 0
    kv[1, :512] = 0
    kv[1, 5] = 2.0 ** -133                                 # subnormal
    kv[2, :512] *= 2.0 ** 124 / np.abs(kv[2, :512]).max()
    kv[3, :512] = 448.0 * 2.0 ** rng.integers(-12, 1, 512)
    kv[4, 17], kv[5, 511], kv[6, 520], kv[7, 575] = np.inf, np.nan, -np.inf, np.nan
    kv[8, 3] = 3.0e38                                      # finite, beyond 2^127
    kv[9, :512] = 2.0 ** -14
    kv[10, :512] = 1.0
    kv[11, 500] = -1e30
    kv = bf16(kv)
    for weight in (None, bf16(np.ones(512))):
        cache = pool(1, 32, rng)
        before = [x.clone() for x in cache]
        slots, pos = np.arange(12) * 2, np.arange(12) * 100
        run_append(kv, slots, pos, freq(64), cache, norm_weight=weight)
        scales = host(cache[1])[0]
        bad = np.isnan(scales[slots])
        # the norm's mean of squares passes fp32 where a value passes 2^64
        if weight is None:
            assert bad.tolist() == [False] * 4 + [True] * 5 + [False] * 3
            check_append(kv, slots, pos, freq(64), before, cache, True, 1.0, None, 1e-6)
        else:
            assert bad[[4, 5, 6, 7]].all() and not bad[[0, 1, 3, 9, 10]].any()


# ------------------------------------------------------------------------------- gather

def test_gather_is_exact():
    rng = np.random.default_rng(11)
    kv = [0, 1, 31, 0, 64, 200, 33, 0, 129]
    for B in (32, 64, 128):
        cache = LatentCache(rng, kv, B, spread=10)
        off = offsets(kv)
        N = int(off[-1]) + 3
        raw_l, latent, pad = with_canary((N, 512), torch.bfloat16)
        raw_r, rope, _ = with_canary((N, 64), torch.bfloat16)
        bfp8.bfp8_latent_gather(*cache.gpu(), i32(cache.table), i32(off), latent, rope)
        torch.cuda.synchronize()
        assert canary_intact(raw_l, pad) and canary_intact(raw_r, pad)
        for r, n in enumerate(kv):
            if n:
                c, _, k = ref.tokens(*cache.arrays, cache.table[r], n)
                assert np.array_equal(f64(latent[off[r]:off[r + 1]]), c) and np.array_equal(f64(rope[off[r]:off[r + 1]]), k)
        assert (latent[-3:].view(torch.int16) == FILL).all() and (rope[-3:].view(torch.int16) == FILL).all()


def test_gather_parts_and_strides():
    """Chunks from a start on, into one combined array; capacity below the rows; poisoned tokens."""
    rng = np.random.default_rng(12)
    kv, starts, count = [300, 90, 128, 5], [100, 0, 127, 2], [150, 90, 1, 0]
    cache = LatentCache(rng, kv, 64)
    at = cache.table[1, 0], 7
    cache.codes[at], cache.scales[at], cache.rope[at] = 0, np.nan, 0
    off = offsets(count)
    both = torch.full((int(off[-1]) - 10, 576 + 8), 7.0, dtype=torch.bfloat16, device=dev())
    bfp8.bfp8_latent_gather(*cache.gpu(), i32(cache.table), i32(off), both[:, :512], both[:, 512:576], i32(starts))
    torch.cuda.synchronize()
    got = f64(both)
    assert (got[:, 576:] == 7.0).all()
    for r, n in enumerate(count):
        c, _, k = ref.tokens(*cache.arrays, cache.table[r], kv[r])
        rows = got[off[r]:off[r + 1]]
        assert np.array_equal(rows[:, :512], c[starts[r]:starts[r] + n][:len(rows)], equal_nan=True)
        assert np.array_equal(rows[:, 512:576], k[starts[r]:starts[r] + n][:len(rows)])
    assert np.isnan(got[157, :512]).all()


@pytest.mark.parametrize("R", [65, 500, 4096])
def test_gather_many_requests(R):
    rng = np.random.default_rng(R)
    kv = [int(x) for x in rng.choice([0, 0, 0, 1, 2, 40], R)]
    kv[5:75] = [0] * min(70, R - 5)                        # more than 64 empty ones in a row
    kv = kv[:R]
    kv[-1] = 3
    cache = LatentCache(rng, kv, 32)
    off = offsets(kv)
    latent, rope = bfp8.latent_gather(cache.gpu(), i32(cache.table), i32(off), int(off[-1]))
    got, k_got = f64(latent), f64(rope)
    for r, n in enumerate(kv):
        if n:
            c, _, k = ref.tokens(*cache.arrays, cache.table[r], n)
            assert np.array_equal(got[off[r]:off[r + 1]], c) and np.array_equal(k_got[off[r]:off[r + 1]], k), r


def test_gather_any_offsets_stay_inside_the_buffers():
    rng = np.random.default_rng(13)
    cache = LatentCache(rng, [100, 100, 100], 64)
    for off in ([0, 2 ** 31 - 1, 5, 6], [7, 3, 1, 0], [-2 ** 31, 2, -4, 40], [0, 40, 40, 2 ** 31 - 1]):
        raw_l, latent, pad = with_canary((50, 512), torch.bfloat16)
        raw_r, rope, _ = with_canary((50, 64), torch.bfloat16)
        for starts in (None, i32([-2 ** 31, 2 ** 31 - 1, 60])):
            bfp8.bfp8_latent_gather(*cache.gpu(), i32(cache.table), i32(off), latent, rope, starts)
        torch.cuda.synchronize()
        assert canary_intact(raw_l, pad) and canary_intact(raw_r, pad)


# ---------------------------------------------------------------------------- the whole

@pytest.mark.parametrize("H", [16, 128])
def test_a_serving_run(H):
    """Plan, rotate, append and attend over several steps: prompts, single tokens, a draft that is taken
    back; the last two steps are one captured graph.  Against 64 bits over what the cache holds, and the
    cache against 64 bits over all tokens that were kept."""
    rng = np.random.default_rng(14)
    R, B, W = 5, 32, 10
    P = R * W
    cache = pool(P, B, rng)
    table = torch.zeros(R, W, dtype=torch.int32, device=dev())
    free, head = i32(rng.permutation(P)), i32([0])
    ctx = i32([0] * R)
    f, amplitude = bfp8.rope_frequencies(64, factor=40.0)
    weight = bf16(1 + 0.2 * rng.standard_normal(512))
    scale = 192 ** -0.5
    T = 160
    kv = bf16(rng.standard_normal((T, 576)))
    q = bf16(0.5 * rng.standard_normal((T, H, 576)))
    rotated = torch.empty(T, H, 64, dtype=torch.bfloat16, device=dev())
    out = torch.zeros(T, H, 512, dtype=torch.bfloat16, device=dev())
    lse = torch.zeros(T, H, dtype=torch.float32, device=dev())
    plan = bfp8.kv_plan_buffers(R, T, dev())
    ws = bfp8.attn_latent_workspace(R, 64, H, dev())
    new = i32([0] * R)

    def step():
        bfp8.bfp8_kv_plan(ctx, new, free, table, B, plan, head)
        bfp8.bfp8_rope(q[..., 512:], plan.positions, f, rotated, True, amplitude)
        bfp8.bfp8_latent_append(kv, plan.slot_map, plan.positions, f, *cache, norm_weight=weight, amplitude=amplitude)
        bfp8.bfp8_attn_latent(q[..., :512], rotated, *cache, table, plan.q_offsets, plan.kv_lens, 64, scale, out, lse, ws)
        ctx.copy_(torch.where(plan.kv_lens > 0, plan.kv_lens, ctx))
        head.copy_(plan.counts[1:2])

    kept = [[] for _ in range(R)]                          # (rows of 576) of each request

    def after(lens):
        torch.cuda.synchronize()
        off = offsets(lens)
        rows, pos = f64(kv), host(plan.positions)
        for r, n in enumerate(lens):
            kept[r] += [rows[off[r] + i] for i in range(n)]
        arrays = host(cache[0]), host(cache[1]), f64(cache[2])
        n = int(off[-1])
        assert pos[:n].tolist() == [len(kept[r]) - m + i for r, m in enumerate(lens) for i in range(m)]
        want = ref.rotate(f64(q)[:n, :, 512:], pos[:n], host(f), True, amplitude)
        assert (np.abs(f64(rotated)[:n] - want) <= rope_bound(f64(q)[:n, :, 512:], want, amplitude)).all()
        kv_lens = [len(k) if m else 0 for k, m in zip(kept, lens)]
        check(out[:n], lse[:n], q[:n, :, :512], rotated[:n], arrays, host(table), off, kv_lens, scale, f"step {lens}")
        for r in range(R):
            if not kept[r]:
                continue
            c, s, k = ref.tokens(*arrays, host(table)[r], len(kept[r]))
            y = ref.norm(np.array(kept[r])[:, :512], f64(weight), 1e-6)
            assert (np.abs(c - y) <= np.maximum((2.0 ** -4 + 2.0 ** -18) * np.abs(y), 2.0 ** -10 * s[:, None])).all()

    for lens in ([40, 1, 0, 64, 33], [1, 1, 5, 1, 1], [4, 0, 4, 4, 4]):
        new.copy_(i32(lens))
        kv.copy_(bf16(rng.standard_normal((T, 576))))
        step()
        after(lens)
    # two of the four drafted tokens of request 0, all of request 4's, are taken back
    kept[0], kept[4] = kept[0][:-2], kept[4][:-4]
    ctx.copy_(i32([len(k) for k in kept]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([1, 1, 1, 0, 1], [2, 1, 1, 1, 0], [1, 3, 1, 60, 1]):
        new.copy_(i32(lens))
        kv.copy_(bf16(rng.standard_normal((T, 576))))
        graph.replay()
        after(lens)


def test_expanded_form_gives_the_absorbed_result():
    """Latents read back and expanded to a head's keys and values, in 64 bits, against the absorbed form:
    the same attention to the absorbed queries' and outputs' rounding."""
    rng = np.random.default_rng(15)
    kv, H = [150], 16
    cache = LatentCache(rng, kv, 64)
    up_k, up_v = 0.05 * rng.standard_normal((H, 128, 512)), 0.05 * rng.standard_normal((H, 128, 512))
    q = rng.standard_normal((1, H, 128))
    qr = queries(rng, 1, H)[1]
    ql = bf16(np.einsum("thd,hdc->thc", q, up_k))
    latent, rope = bfp8.latent_gather(cache.gpu(), i32(cache.table), i32([0, 150]), 150)
    c, k = f64(latent), f64(rope)
    plan = type("Plan", (), {"q_offsets": i32([0, 1]), "kv_lens": i32(kv)})
    out = f64(bfp8.attn_latent(ql, qr, cache.gpu(), i32(cache.table), plan, 1, 192 ** -0.5))
    z = 192 ** -0.5 * (np.einsum("hd,hdc,nc->hn", q[0], up_k, c) + f64(qr)[0] @ k.T)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want = np.einsum("hn,nc,hdc->hd", p, c, up_v)
    got = np.einsum("hc,hdc->hd", out[0], up_v)
    # ql is off by 2^-8 of itself, so logits by 2^-8 sum |q c|; the output by 2^-8 of itself
    slip = 192 ** -0.5 * 2.0 ** -8 * (np.abs(f64(ql)[0]) @ np.abs(c).T).max()
    bound = np.einsum("hn,nc,hdc->hd", p, np.abs(c), np.abs(up_v)) * (np.exp(2 * slip) - 1 + 2.0 ** -8 + 2.0 ** -10)
    assert (np.abs(got - want) <= bound).all()
