"""bfp8_attn_latent against a plain 64-bit implementation: head counts, page sizes, lengths from none to
many tiles, one and many new tokens, rows that see nothing, stale bytes that hold NaN, poisoned tokens."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import latent_reference as ref
from gpu_helpers import announce, dev
from kv_helpers import bf16, f64, i32, offsets
from latent_helpers import LatentCache, attend, check, queries

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
FILL = -23131                                              # the guard pattern as int16


def _case(seed, kv, new, H, B, scale=SCALE, max_new=None, workspace=True, size=0.05, spread=3):
    rng = np.random.default_rng(seed)
    cache = LatentCache(rng, kv, B, spread=spread)
    q_off = offsets(new)
    T = int(q_off[-1]) + 2                                  # two rows of no request
    ql, qr = queries(rng, T, H, size)
    max_new = max(max(new), 1) if max_new is None else max_new
    what = f"seed={seed} kv={list(kv)[:8]} new={list(new)[:8]} H={H} B={B} ws={workspace}"
    announce("latent attention " + what)
    out, lse = attend(ql, qr, cache.gpu(), cache.table, q_off, kv, max_new, scale, workspace)
    worst = check(out, lse, ql, qr, cache.arrays, cache.table, q_off, kv, scale, what)
    announce(f"worst err/bound {worst:.3f}")
    assert (out[-2:].view(torch.int16) == FILL).all(), "a row of no request was written"
    return ql, qr, cache, q_off, out, lse


@pytest.mark.parametrize("B", [32, 64, 128])
@pytest.mark.parametrize("H", [1, 16, 64])
@pytest.mark.parametrize("workspace", [True, False])
def test_single_tokens(H, B, workspace):
    kv = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 300, 517]
    _case(B + H, kv, [1] * len(kv), H, B, workspace=workspace)


@pytest.mark.parametrize("H", [2, 5, 31, 32, 33, 40, 63, 65, 96, 128, 129, 200])
def test_head_counts(H):
    _case(H, [140, 3, 260], [1, 1, 1], H, 64)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("H", [3, 16, 20, 48])
def test_several_new_tokens(H, workspace):
    # a draft of four, one token, a whole prompt, a chunk behind a cached prefix
    _case(7 * H, [100, 1, 50, 290, 4], [4, 1, 50, 37, 4], H, 32, workspace=workspace)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("H", [16, 128])
def test_idle_requests_and_rows_that_see_nothing(H, workspace):
    # idle slots, requests without tokens, more new tokens than cached ones
    _case(H, [0, 70, 0, 0, 3, 1, 200, 0], [0, 1, 2, 0, 5, 0, 3, 1], H, 64, workspace=workspace)


def test_nothing_at_all():
    for ws in (True, False):
        _, _, _, _, out, lse = _case(3, [0, 0], [2, 1], 16, 64, workspace=ws)
        assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()


def test_more_new_tokens_than_max_new():
    rng = np.random.default_rng(4)
    cache = LatentCache(rng, [90, 90], 64)
    ql, qr = queries(rng, 12, 16)
    out, lse = attend(ql, qr, cache.gpu(), cache.table, [0, 6, 12], [90, 90], 4, SCALE)
    rows = np.zeros((12, 1), bool)
    rows[[0, 1, 2, 3, 6, 7, 8, 9]] = True
    check(out, lse, ql, qr, cache.arrays, cache.table, [0, 6, 12], [90, 90], SCALE, "max_new", rows)
    assert (out[[4, 5, 10, 11]].view(torch.int16) == FILL).all()


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("B", [32, 128])
def test_long_ones_shared_by_many_workgroups(H, B):
    _case(H + B, [9000, 4097, 1], [1, 1, 1], H, B, size=0.1)


@pytest.mark.parametrize("H", [16, 64])
def test_more_requests_than_lanes(H):
    # every workgroup's share passes over idle requests and request boundaries
    rng = np.random.default_rng(40)
    new = [int(x) for x in rng.integers(0, 3, 150)]
    kv = [n + int(rng.choice([0, 1, 60, 63, 64, 300])) if n else 0 for n in new]
    _case(40, kv, new, H, 64)
    _case(41, kv, new, H, 64, workspace=False)


@pytest.mark.parametrize("R", [700, 1023, 1024])
def test_about_as_many_items_as_a_split_launch_takes(R):
    rng = np.random.default_rng(50)
    new = [int(x) for x in rng.integers(0, 2, R)]
    kv = [n + int(rng.integers(0, 90)) if n else 0 for n in new]
    assert (bfp8.bfp8_attn_latent_workspace_size(R, 1, 16) == 0) == (R >= 1024)
    _case(50, kv, new, 16, 32)


def test_most_requests():
    R = bfp8.KV_MAX_REQUESTS
    rng = np.random.default_rng(51)
    new = [int(x) for x in rng.integers(0, 2, R)]
    kv = [n + int(rng.integers(0, 3)) if n else 0 for n in new]
    _case(51, kv, new, 2, 32)


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    R = int(rng.integers(1, 20))
    H = int(rng.choice([1, 2, 7, 16, 24, 32, 64, 80, 128]))
    B = int(rng.choice([32, 64, 128]))
    top = int(rng.choice([1, 1, 3, 9, 40]))
    new = [int(x) for x in rng.integers(0, top + 1, R)]
    kv = [n + int(rng.integers(0, 600)) if n else 0 for n in new]
    _case(1000 + seed, kv, new, H, B, workspace=bool(seed % 4))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1.5])
def test_scales(H, scale):
    _case(22, [300, 70], [1, 3], H, 64, scale=scale)


@pytest.mark.parametrize("H", [16, 64])
def test_token_scales_far_apart(H):
    _case(23, [400, 129], [1, 2], H, 64, spread=14, size=0.4)


@pytest.mark.parametrize("H", [16, 64])
def test_growing_logits_move_the_reference(H):
    """Keys that grow along the request, by leaps in one half of a tile and then in the other."""
    rng = np.random.default_rng(24)
    n = 700
    cache = LatentCache(rng, [n], 64)
    for t in range(n):
        page, off = cache.table[0, t // 64], t % 64
        cache.rope[page, off] = f64(bf16(np.full(64, (t // 45) * (1.0 + 0.3 * (t % 64 >= 32)))))
    ql, qr = queries(rng, 1, H)
    qr = torch.ones_like(qr)
    qr[0, ::3] = -1
    scale = 0.1
    out, lse = attend(ql, qr, cache.gpu(), cache.table, [0, 1], [n], 1, scale)
    check(out, lse, ql, qr, cache.arrays, cache.table, [0, 1], [n], scale, "growing")


@pytest.mark.parametrize("H", [16, 64])
def test_far_logits(H):
    """Logits of +-2^30: one token takes all the weight."""
    rng = np.random.default_rng(25)
    cache = LatentCache(rng, [150], 64)
    ql, qr = queries(rng, 1, H, 2.0 ** 24)
    out, _ = attend(ql, qr, cache.gpu(), cache.table, [0, 1], [150], 1, 4.0)
    want = ref.attention(f64(ql), f64(qr), cache.arrays, cache.table, [0, 1], [150], 4.0)[0]
    assert np.allclose(f64(out), want, rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("H", [16, 64])
def test_poisoned_tokens(H, workspace):
    """A token stored as not finite makes the rows that see it NaN, and no others."""
    rng = np.random.default_rng(26)
    kv, new = [200, 130, 64], [4, 1, 1]
    cache = LatentCache(rng, kv, 64)
    at = cache.table[0, 3], 6                               # token 198: seen by the last two of four
    cache.codes[at], cache.scales[at], cache.rope[at] = 0, np.nan, 0
    ql, qr = queries(rng, 6, H)
    out, lse = attend(ql, qr, cache.gpu(), cache.table, offsets(new), kv, 4, SCALE, workspace)
    assert torch.isnan(out[2:4]).all() and torch.isnan(lse[2:4]).all()
    cache.scales[at] = 1.0                                  # (hidden from the other rows)
    rows = np.ones((6, 1), bool)
    rows[2:4] = False
    check(out, lse, ql, qr, cache.arrays, cache.table, offsets(new), kv, SCALE, "poison", rows)


@pytest.mark.parametrize("H", [16, 40])
def test_strides(H):
    """Queries as slices of wider rows, unaligned ones, outputs head-major."""
    rng = np.random.default_rng(27)
    kv, new = [90, 200], [2, 1]
    cache = LatentCache(rng, kv, 64)
    gpu = cache.gpu()
    ql, qr = queries(rng, 3, H)
    want, want_lse = attend(ql, qr, gpu, cache.table, offsets(new), kv, 2, SCALE)
    for lead in (8, 3):                                     # 16-byte aligned, and not
        wide = torch.zeros(3, H, lead + 512 + 64, dtype=torch.bfloat16, device=dev())
        wide[..., lead:lead + 512], wide[..., lead + 512:] = ql, qr
        out = torch.empty(H, 3, 512 + 8, dtype=torch.bfloat16, device=dev())
        view = out[..., :512].transpose(0, 1)
        out.fill_(7.0)
        bfp8.bfp8_attn_latent(wide[..., lead:lead + 512], wide[..., lead + 512:], *gpu, i32(cache.table),
                              i32(offsets(new)), i32(kv), 2, SCALE, view, None,
                              bfp8.attn_latent_workspace(2, 2, H, dev()))
        torch.cuda.synchronize()
        assert torch.equal(view, want) and (out[..., 512:] == 7.0).all()
        assert not torch.isnan(want_lse).any()


def test_head_major_queries():
    rng = np.random.default_rng(28)
    cache = LatentCache(rng, [100], 64)
    ql, qr = queries(rng, 2, 48)
    want, _ = attend(ql, qr, cache.gpu(), cache.table, [0, 2], [100], 2, SCALE)
    turned = ql.transpose(0, 1).contiguous().transpose(0, 1)
    got, _ = attend(turned, qr, cache.gpu(), cache.table, [0, 2], [100], 2, SCALE)
    assert torch.equal(got, want)


@pytest.mark.parametrize("H", [16, 128])
def test_same_bits_every_time(H):
    rng = np.random.default_rng(29)
    kv = [3000, 700, 50]
    cache = LatentCache(rng, kv, 64)
    ql, qr = queries(rng, 3, H)
    gpu = cache.gpu()
    first, lse = attend(ql, qr, gpu, cache.table, [0, 1, 2, 3], kv, 1, SCALE)
    for _ in range(4):
        again, lse2 = attend(ql, qr, gpu, cache.table, [0, 1, 2, 3], kv, 1, SCALE)
        assert torch.equal(again, first) and torch.equal(lse2, lse)


def test_table_entries_are_clamped_into_the_pool():
    rng = np.random.default_rng(30)
    cache = LatentCache(rng, [256], 64, spare=0)
    table = cache.table.copy()
    ql, qr = queries(rng, 1, 16)
    table[0, 1], table[0, 2] = -2 ** 31, 2 ** 31 - 1
    out, lse = attend(ql, qr, cache.gpu(), table, [0, 1], [256], 1, SCALE)
    check(out, lse, ql, qr, cache.arrays, np.clip(table, 0, cache.codes.shape[0] - 1), [0, 1], [256], SCALE, "clamped")


def test_any_lengths_stay_inside_the_buffers():
    """Offsets and lengths that no plan writes: no result, and no access out of range."""
    rng = np.random.default_rng(31)
    cache = LatentCache(rng, [100, 100, 100], 64)
    ql, qr = queries(rng, 6, 16)
    gpu = cache.gpu()
    for q_off, kv in (([0, 2 ** 31 - 1, -5, 6], [2 ** 31 - 1, -7, 50]), ([5, 3, 1, 0], [60, 60, 60]),
                      ([-2 ** 31, 2, 2, 4], [2 ** 31 - 1] * 3)):
        for ws in (True, False):
            attend(ql, qr, gpu, cache.table, q_off, kv, 4, SCALE, ws)


@pytest.mark.parametrize("H", [16, 128])
def test_replayed_from_a_graph(H):
    """A captured step, replayed as its lengths, queries and cache change; two graphs share a workspace."""
    rng = np.random.default_rng(32)
    R, B, W = 5, 64, 8
    cache = LatentCache(rng, [W * B] * R, B)
    gpu = cache.gpu()
    ql, qr = queries(rng, R, H)
    out = torch.zeros(2, R, H, 512, dtype=torch.bfloat16, device=dev())
    lse = torch.zeros(2, R, H, dtype=torch.float32, device=dev())
    ws = bfp8.attn_latent_workspace(R, 1, H, dev())
    kv, q_off, table = i32([1] * R), i32(range(R + 1)), i32(cache.table)

    def call(x):
        bfp8.bfp8_attn_latent(ql, qr, *gpu, table, q_off, kv, 1, SCALE, out[x], lse[x], ws)
    call(0)
    call(1)
    torch.cuda.synchronize()
    graphs = []
    for x in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(x)
    for lens in ([1, 2, 3, 4, 5], [500, 0, 64, 1, 300], [512] * 5, [0, 0, 0, 0, 1], [65, 129, 64, 63, 200]):
        kv.copy_(i32(lens))
        ql.copy_(queries(rng, R, H)[0])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x in range(2):
            check(out[x], lse[x], ql, qr, cache.arrays, cache.table, range(R + 1), lens, SCALE, f"replay {lens}")


def test_streams():
    """Calls on two streams at once, each with its own workspace, on tensors made on a third."""
    rng = np.random.default_rng(33)
    kv = [2500, 300]
    cache = LatentCache(rng, kv, 64)
    gpu = cache.gpu()
    ql, qr = queries(rng, 2, 64)
    table, q_off, lens = i32(cache.table), i32([0, 1, 2]), i32(kv)
    want = torch.empty(2, 64, 512, dtype=torch.bfloat16, device=dev())
    outs = [torch.zeros_like(want) for _ in range(2)]
    spaces = [bfp8.attn_latent_workspace(2, 1, 64, dev()) for _ in range(3)]
    bfp8.bfp8_attn_latent(ql, qr, *gpu, table, q_off, lens, 1, SCALE, want, None, spaces[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for out, ws, s in zip(outs, spaces, streams):
            bfp8.bfp8_attn_latent(ql, qr, *gpu, table, q_off, lens, 1, SCALE, out, None, ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
