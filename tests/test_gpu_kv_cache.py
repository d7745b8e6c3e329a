"""bfp8_kv_plan and bfp8_kv_append against plain implementations, exactly, and the chain plan ->
append -> attention over several steps, eagerly and from a captured graph."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import kv_reference as ref
from gpu_helpers import announce, canary_intact, dev, with_canary
from kv_helpers import Cache, attend, bf16, check_attention, f64, host, i32, offsets

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 128), (192, 128)]


# -------------------------------------------------------------------------------- plan

def run_plan(ctx, new, free, table, B, T, head=None):
    """The library's call with guard bands; the outputs and the table as numpy."""
    R = len(ctx)
    bufs, arrays = [], []
    for n in (R + 1, R, R + 1, T, T, 4):
        raw, view, pad = with_canary((n,), torch.int32)
        bufs.append(raw)
        arrays.append(view)
    raw_t, tab, pad = with_canary(table.shape, torch.int32)
    tab.copy_(i32(table))
    plan = bfp8.KVPlan(*arrays)
    bfp8.bfp8_kv_plan(i32(ctx), i32(new), i32(free), tab, B, plan, None if head is None else i32([head]))
    torch.cuda.synchronize()
    assert all(canary_intact(x, pad) for x in bufs + [raw_t]), "wrote outside an output"
    return [host(x) for x in arrays] + [host(tab)]


def check_plan(ctx, new, free, table, B, T, head=None, what=""):
    announce(f"plan {what} R={len(ctx)} T={T} B={B} W={table.shape[1]} free={len(free)} head={head}")
    got = run_plan(ctx, new, free, table, B, T, head)
    want = ref.plan(ctx, new, free, head or 0, table, B, T)
    names = ("q_offsets", "kv_lens", "tile_offsets", "slot_map", "positions", "counts", "block_table")
    for n, g, w in zip(names, got, want):
        assert np.array_equal(g, w), f"{what}: {n} differs"
    return got


def requests(rng, R, top_ctx, top_new, B, short=0):
    ctx = rng.integers(0, top_ctx + 1, R)
    new = rng.integers(0, top_new + 1, R)
    need = -(-(ctx + new) // B) - -(-ctx // B)
    W = int((-(-(ctx + new) // B)).max(initial=0)) + 1
    table = rng.integers(0, 1 << 20, (R, W)).astype(np.int32)
    free = rng.permutation(1 << 20)[:max(int(need.sum()) - short, 0)].astype(np.int32)
    return ctx, new, free, table, int(new.sum())


@pytest.mark.parametrize("R", [1, 2, 63, 64, 65, 511, 512, 513, 1000, 4096])
@pytest.mark.parametrize("B", [32, 64, 128])
def test_plan_sizes(R, B):
    rng = np.random.default_rng(R + B)
    ctx, new, free, table, T = requests(rng, R, 700, 40, B)
    check_plan(ctx, new, free, table, B, T + int(rng.integers(0, 5)), what="sizes")


@pytest.mark.parametrize("seed", range(6))
def test_plan_runs_out_of_pages(seed):
    rng = np.random.default_rng(seed)
    ctx, new, free, table, T = requests(rng, 200, 300, 60, 32, short=int(rng.integers(1, 60)))
    got = check_plan(ctx, new, free, table, 32, T, what="short")
    assert got[5][2] < 200 and (got[1] == 0).any()


def test_plan_prompts_and_decode():
    rng = np.random.default_rng(7)
    ctx = np.array([0, 1, 63, 64, 65, 128, 0, 5000, 127])
    new = np.array([1, 1, 1, 1, 1, 0, 3000, 1, 129])
    W = 90
    table = rng.integers(0, 999, (9, W)).astype(np.int32)
    check_plan(ctx, new, np.arange(500, 700), table, 64, int(new.sum()) + 100, what="mixed")
    check_plan(ctx, new, np.arange(500, 700), table, 64, int(new.sum()), head=37, what="head")


def test_plan_refusals():
    rng = np.random.default_rng(8)
    table = rng.integers(0, 99, (6, 4)).astype(np.int32)
    free = np.arange(100, 200)
    # negative lengths, a request past its table row, and the ones behind them
    ctx, new = [3, -1, 200, 100, 10, 0], [5, 2, 100, 28, -3, 64]
    check_plan(ctx, new, free, table, 64, 400, what="lengths")
    check_plan(ctx, new, free, table, 64, 100, what="token capacity")
    check_plan(ctx, new, free, table, 64, 0, what="no tokens")
    check_plan(ctx, new, free[:0], table, 64, 400, what="no pages")
    check_plan(ctx, new, free, table, 64, 400, head=100, what="all taken")
    check_plan(ctx, new, free, table, 64, 400, head=250, what="head past the list")
    check_plan([2 ** 31 - 1, 5, 5], [2 ** 31 - 1, 2 ** 31 - 1, 5], free, table[:3], 64, 400, what="large")


def test_plan_without_requests():
    got = check_plan(np.zeros(0, int), np.zeros(0, int), np.arange(4), np.zeros((0, 3), np.int32), 64, 70,
                     what="empty")
    assert (got[3] == -1).all()


def test_plan_continues_from_its_own_counts():
    """A free list consumed over steps by handing counts[1] back."""
    B, R = 32, 5
    rng = np.random.default_rng(9)
    free = rng.permutation(64).astype(np.int32)
    table = np.full((R, 12), -1, np.int32)
    tab, fr = i32(table), i32(free)
    ctx = np.zeros(R, int)
    head = None
    taken = []
    for step in range(6):
        new = rng.integers(0, 40, R)
        plan = bfp8.kv_plan(i32(ctx), i32(new), fr, tab, B, int(new.sum()) + 3, head)
        want = ref.plan(ctx, new, free, int(host(head)[0]) if head is not None else 0, table, B,
                        int(new.sum()) + 3)
        table = want[-1]
        assert np.array_equal(host(tab), table)
        for g, w in zip(plan, want):
            assert np.array_equal(host(g), w)
        head = plan.counts[1:2].clone()
        ctx = np.where(want[1] > 0, want[1], ctx)
        taken = table[table >= 0]
        assert len(set(taken)) == len(taken), "a page was handed out twice"


# ------------------------------------------------------------------------------ append

class Pool:
    """Cache arrays with guard bands, filled with random codes (NaN among them) and scales."""

    def __init__(self, rng, P, H, B, dk, dv):
        self.np = [rng.integers(0, 256, (P, H, B, dk), dtype=np.uint8),
                   (2.0 ** rng.integers(-12, 3, (P, H))).astype(np.float32),
                   rng.integers(0, 127, (P, H, dv, B), dtype=np.uint8),
                   (2.0 ** rng.integers(-12, 3, (P, H))).astype(np.float32)]
        self.raw, self.gpu = [], []
        for x in self.np:
            raw, view, self.pad = with_canary(x.shape, torch.uint8 if x.dtype == np.uint8 else torch.float32)
            view.copy_(torch.from_numpy(x))
            self.raw.append(raw)
            self.gpu.append(view)

    def append(self, k, v, slots, what=""):
        """Both sides, compared bit for bit."""
        want = ref.append(f64(k), f64(v), slots, *self.np)
        bfp8.bfp8_kv_append(k, v, i32(slots), *self.gpu)
        torch.cuda.synchronize()
        assert all(canary_intact(r, self.pad) for r in self.raw), f"{what}: wrote outside the cache"
        for name, g, w in zip(("k_cache", "k_scales", "v_cache", "v_scales"), self.gpu, want):
            g = host(g)
            assert np.array_equal(g, w), f"{what}: {name}: {(g != w).sum()} of {g.size} differ"
        self.np = list(want)


def rows(rng, T, H, d, size=1.0):
    return bf16(rng.standard_normal((T, H, d)) * size * 2.0 ** rng.integers(-6, 6, (T, 1, 1)))


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
def test_append_prompts_and_single_tokens(dk, dv, B):
    rng = np.random.default_rng(dk + B)
    H = 3
    pool = Pool(rng, 14, H, B, dk, dv)
    # runs: a whole page and more from its start, a tail in the middle, one token, a page's last token
    runs = [(0, 0, 2 * B + 5), (5, 3, 7), (6, B - 1, 1), (7, 0, 1), (8, B // 2, B // 2), (9, 1, B - 1)]
    slots = []
    for page, off, n in runs:
        for i in range(n):
            slots.append((page + (off + i) // B) * B + (off + i) % B)
    T = len(slots)
    announce(f"append {dk}/{dv} B={B} T={T}")
    pool.append(rows(rng, T, H, dk), rows(rng, T, H, dv), np.array(slots), "runs")
    # growing pages, token by token, with larger and smaller elements: scales only grow
    for step in range(6):
        slots = np.array([10 * B + step, 11 * B + 2 + step, 6 * B, 12 * B + B - 6 + step])
        size = [1e-3, 1.0, 1e-2, 300.0, 1e-5, 2e4][step]
        pool.append(rows(rng, 4, H, dk, size), rows(rng, 4, H, dv, size), slots, f"step {step}")


def test_append_skips_slots_outside_the_pool():
    rng = np.random.default_rng(1)
    pool = Pool(rng, 4, 2, 64, 128, 128)
    slots = np.array([-1, 0, 1, -1, 256, 100, 2 ** 31 - 1, -2 ** 31, 101, 255, -1])
    pool.append(rows(rng, 11, 2, 128), rows(rng, 11, 2, 128), slots, "outside")
    pool.append(rows(rng, 3, 2, 128), rows(rng, 3, 2, 128), np.array([-1, -1, 256]), "none")
    pool.append(rows(rng, 0, 2, 128), rows(rng, 0, 2, 128), np.zeros(0, int), "no tokens")


def test_append_small_and_extreme_elements():
    rng = np.random.default_rng(2)
    pool = Pool(rng, 8, 1, 32, 64, 64)
    k, v = rng.standard_normal((6, 1, 64)), rng.standard_normal((6, 1, 64))
    k[0], v[0] = 0.0, -0.0                                   # an all-zero page
    k[1] *= 1e-38
    v[1] *= 1e30
    k[2] = 448.0 * 2.0 ** -5                                 # exact quotients and halfway ones
    v[2] = 17.0 * 2.0 ** -3
    k[3, 0, 0] = 3.3e38
    v[3, 0, :32] = 2.0 ** -133                               # subnormal bf16
    pool.append(bf16(k), bf16(v), np.array([0, 32, 64, 96, 128, 160]), "extremes")


def test_append_every_bf16_pattern():
    """All finite bf16 patterns as keys and values, blocks of ordinary and of huge maxima."""
    bits = np.arange(65536, dtype=np.uint32)
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    x = x[np.isfinite(x)]
    x = np.concatenate([x, np.zeros((-len(x)) % (64 * 32), np.float32)]).reshape(-1, 1, 64)
    order = np.random.default_rng(3).permutation(len(x))
    x = x[order]
    T = len(x)
    pool = Pool(np.random.default_rng(4), T // 32, 1, 32, 64, 64)
    pool.append(bf16(x), bf16(x[::-1].copy()), np.arange(T), "patterns")


def test_append_elements_that_are_not_finite():
    rng = np.random.default_rng(5)
    H = 2
    pool = Pool(rng, 6, H, 32, 128, 128)
    k, v = rng.standard_normal((40, H, 128)), rng.standard_normal((40, H, 128))
    k[3, 0, 7], k[20, 1, 100], k[39, 0, 0] = np.nan, np.inf, -np.inf
    v[5, 1, 3], v[33, 0, 127] = np.inf, np.nan
    k[36] = np.nan                                           # a whole token
    pool.append(bf16(k), bf16(v), np.arange(40) + 64, "not finite")
    # the page goes on with a token that makes its scale grow
    pool.append(bf16(k[:1] * 1e4), bf16(v[:1] * 1e4), np.array([64 + 40]), "after")


@pytest.mark.parametrize("at", [0, 1, 8])
def test_append_strided_rows(at):
    """Slices of one projection: unaligned ones take the scalar loads."""
    rng = np.random.default_rng(6)
    H, B = 2, 64
    for T in (1, 3, 130):
        wide = bf16(rng.standard_normal((T, H * 256 + 24)))
        kv = wide[:, at:at + H * 256].unflatten(1, (H, 256))
        pool = Pool(rng, 5, H, B, 128, 128)
        pool.append(kv[:, :, :128], kv[:, :, 128:], np.arange(T) + 10, f"T={T}")
    k = bf16(rng.standard_normal((H, 70, 128))).transpose(0, 1)      # head-major
    pool = Pool(rng, 5, H, B, 128, 128)
    pool.append(k, rows(rng, 70, H, 128), np.arange(70) + 64, "head-major")
    one = bf16(rng.standard_normal((1, 1, 128))).expand(5, H, 128)   # stride 0
    pool.append(one, one, np.arange(5) + 192, "broadcast")


@pytest.mark.parametrize("H,T", [(1, 9000), (64, 300)])
def test_append_long_prompts(H, T):
    rng = np.random.default_rng(7)
    B = 128
    pool = Pool(rng, -(-T // B) + 1, H, B, 64, 64)
    k = bf16(rng.standard_normal((T, H, 64)).astype(np.float32))
    pool.append(k, k, np.arange(T) + 77, "long")


def test_append_past_32_bits():
    P, H, B = 70000, 4, 128                                  # 4.6 GB an array
    k = torch.zeros(P, H, B, 128, dtype=torch.uint8, device=dev())
    v = torch.zeros(P, H, 128, B, dtype=torch.uint8, device=dev())
    ks, vs = torch.ones(P, H, device=dev()), torch.ones(P, H, device=dev())
    rng = np.random.default_rng(8)
    x, y = rows(rng, 5, H, 128), rows(rng, 5, H, 128)
    slots = np.array([(P - 1) * B + 126, (P - 1) * B + 127, 0, 1, 65537 * B])
    bfp8.bfp8_kv_append(x, y, i32(slots), k, ks, v, vs)
    small = [np.zeros((3, H, B, 128), np.uint8), np.ones((3, H), np.float32),
             np.zeros((3, H, 128, B), np.uint8), np.ones((3, H), np.float32)]
    want = ref.append(f64(x), f64(y), np.array([2 * B + 126, 2 * B + 127, 0, 1, B]), *small)
    pages = torch.tensor([0, 65537, P - 1], device=dev())
    for g, w in zip((k, ks, v, vs), want):
        assert np.array_equal(host(g[pages]), w)
    assert int((k != 0).sum()) == int((want[0] != 0).sum())


def test_append_on_another_stream():
    rng = np.random.default_rng(9)
    pool = Pool(rng, 4, 2, 64, 128, 128)
    x, y = rows(rng, 70, 2, 128), rows(rng, 70, 2, 128)
    slots = np.arange(70) + 30
    want = ref.append(f64(x), f64(y), slots, *pool.np)
    s, sl = torch.cuda.Stream(), i32(slots)
    torch.cuda.synchronize()
    bfp8.bfp8_kv_append(x, y, sl, *pool.gpu, stream=s)
    s.synchronize()
    assert all(np.array_equal(host(g), w) for g, w in zip(pool.gpu, want))


# ------------------------------------------------------------------------------- chain

def _chain(dk, dv, B, H, G, steps, seed):
    """Plan, append and attend over `steps` (lists of new lengths); every step against the plain
    implementations on the same bf16 inputs."""
    rng = np.random.default_rng(seed)
    R = len(steps[0])
    total = np.sum(steps, axis=0)
    P = int((-(-total // B)).sum()) + 2
    free = rng.permutation(P).astype(np.int32)
    cache = bfp8.kv_cache_buffers(P, H, B, dk, dv, dev())
    for x in cache:
        x.fill_(0x7F if x.dtype == torch.uint8 else float("nan"))
    arrays = [host(x) for x in cache]
    table_np = np.zeros((R, int((-(-total // B)).max()) + 1), np.int32)
    table, fr, head = i32(table_np), i32(free), None
    ctx = np.zeros(R, int)
    for n, new in enumerate(steps):
        new = np.array(new)
        T = int(new.sum())
        plan = bfp8.kv_plan(i32(ctx), i32(new), fr, table, B, T, head)
        head_np = int(host(head)[0]) if head is not None else 0
        want = ref.plan(ctx, new, free, head_np, table_np, B, T)
        table_np = want[-1]
        head = plan.counts[1:2].clone()
        k, v = rows(rng, T, H, dk), rows(rng, T, H, dv)
        q = bf16(rng.standard_normal((T, H * G, dk)) * 0.05)
        bfp8.bfp8_kv_append(k, v, plan.slot_map, *cache)
        arrays = ref.append(f64(k), f64(v), want[3], *arrays)
        for g, w in zip(cache, arrays):
            assert np.array_equal(host(g), w, equal_nan=True), f"step {n}: cache differs"
        out = bfp8.attn_paged(q, cache, table, plan, max(1, int(new.max())))
        lse = torch.empty(T, H * G, device=dev())
        again = torch.empty_like(out)
        bfp8.bfp8_attn_paged(q, *cache, table, plan.q_offsets, plan.kv_lens, plan.tile_offsets,
                             max(1, int(new.max())), dk ** -0.5, again, lse)
        check_attention(out, lse, f64(q), arrays, table_np, want[0], want[1], dk ** -0.5, f"step {n}")
        ctx = ctx + new


@pytest.mark.parametrize("dk,dv", DIMS)
def test_chain(dk, dv):
    _chain(dk, dv, 32, 2, 2, [[70, 1, 0, 33], [1, 1, 5, 1], [1, 0, 1, 31], [1, 1, 1, 1], [40, 3, 1, 1]], dk)


def test_chain_larger_pages():
    _chain(128, 128, 128, 1, 8, [[130, 7], [1, 1], [2, 2], [1, 200]], 3)


def test_chain_replayed_from_a_graph():
    """A decode step (plan, append, attention) captured once; replays against eager calls on a copy
    of the cache, lengths advanced in place between the replays."""
    R, H, G, B, d = 5, 2, 4, 32, 128
    rng = np.random.default_rng(11)
    P = 40
    ctx = i32([0, 31, 64, 100, 7])
    new = i32([1, 1, 0, 1, 1])
    free = i32(rng.permutation(np.arange(20, P)))
    head, head_e = i32([0]), i32([0])
    table = i32(rng.permutation(20).reshape(5, 4).repeat(2, axis=1)[:, :6])
    cache = bfp8.kv_cache_buffers(P, H, B, d, d, dev())
    for x in cache:
        x.fill_(0x30 if x.dtype == torch.uint8 else 1.0)
    k, v, q = rows(rng, 4, H, d), rows(rng, 4, H, d), rows(rng, 4, H * G, d, 0.1)
    plan = bfp8.kv_plan_buffers(R, 4, dev())
    out = torch.zeros(4, H * G, d, dtype=torch.bfloat16, device=dev())
    ws = bfp8.attn_paged_workspace(R, 1, H * G, H, d, d, dev())
    table_e, cache_e = table.clone(), tuple(x.clone() for x in cache)
    state = (table.clone(), tuple(x.clone() for x in cache))

    def step(tab, c, hd, o):
        bfp8.bfp8_kv_plan(ctx, new, free, tab, B, plan, hd)
        bfp8.bfp8_kv_append(k, v, plan.slot_map, *c)
        bfp8.bfp8_attn_paged(q, *c, tab, plan.q_offsets, plan.kv_lens, plan.tile_offsets, 1, 0.1, o, None,
                             ws)

    step(table, cache, head, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(table, cache, head, out)
    table.copy_(state[0])
    for x, y in zip(cache, state[1]):
        x.copy_(y)
    out_e = torch.zeros_like(out)
    for r in range(5):
        step(table_e, cache_e, head_e, out_e)
        head_e.copy_(plan.counts[1:2])
        torch.cuda.synchronize()
        ws.fill_(0xFF)
        out.zero_()
        graph.replay()
        head.copy_(plan.counts[1:2])
        torch.cuda.synchronize()
        announce(f"chain replay {r}")
        assert torch.equal(out, out_e) and torch.equal(table, table_e)
        assert all(torch.equal(x, y) for x, y in zip(cache, cache_e))
        ctx += new
        k.mul_(1.5)                                          # eager work between the replays
        q.neg_()
