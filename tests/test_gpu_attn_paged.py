"""bfp8_attn_paged against a plain 64-bit implementation: head layouts, page sizes, lengths from
none to several tiles, one and many new tokens, rows that see nothing, stale bytes that hold NaN."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import kv_reference as ref
from gpu_helpers import announce, dev
from kv_helpers import Cache, attend, bf16, check_attention, f64, i32, offsets

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 128), (192, 128)]


def _case(seed, kv_lens, new, H, G, B, dk, dv, scale=None, max_new=None, workspace=True):
    rng = np.random.default_rng(seed)
    cache = Cache(rng, kv_lens, H, B, dk, dv)
    q_off = offsets(new)
    T = int(q_off[-1]) + 2                                  # two rows of no request
    q = bf16(rng.standard_normal((T, H * G, dk)))
    scale = dk ** -0.5 if scale is None else scale
    max_new = max(max(new), 1) if max_new is None else max_new
    what = f"seed={seed} kv={list(kv_lens)[:8]} new={list(new)[:8]} H={H} G={G} B={B} {dk}/{dv}"
    announce("attention " + what)
    out, lse = attend(q, cache.gpu(), cache.table, q_off, kv_lens, max_new, scale, workspace)
    check_attention(out, lse, f64(q), cache.arrays, cache.table, q_off, kv_lens, scale, what)
    # rows of no request keep the fill pattern
    assert (out[-2:].view(torch.int16) == -23131).all(), "a row of no request was written"
    return q, cache, q_off, out, lse


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
@pytest.mark.parametrize("G", [1, 4])
def test_single_tokens(dk, dv, B, G):
    kv = [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 200, 300, 517]
    _case(dk + B + G, kv, [1] * len(kv), 2, G, B, dk, dv)


@pytest.mark.parametrize("G", [2, 3, 5, 7, 8, 16, 17, 32, 40])
def test_head_groups(G):
    _case(G, [140, 3, 260], [1, 1, 1], 2, G, 64, 128, 128)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("G", [1, 3, 8])
def test_several_new_tokens(dk, dv, G):
    # a draft of four, one token, a whole prompt, a chunk behind a cached prefix
    _case(7 * G + dk, [100, 1, 150, 290, 4], [4, 1, 150, 37, 4], 2, G, 32, dk, dv)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_prompts(dk, dv):
    _case(dk, [257, 1, 130, 64], [257, 1, 130, 64], 1, 2, 64, dk, dv)


@pytest.mark.parametrize("workspace", [True, False])
def test_long_and_ragged(workspace):
    kv = [5000, 1, 777, 2049, 64]
    q, cache, q_off, a, la = _case(11, kv, [1] * 5, 2, 4, 64, 128, 128, workspace=workspace)


def test_idle_and_empty_requests():
    # idle slots, requests whose cache is empty although they have queries, lengths below the
    # number of queries (the first rows then see nothing)
    kv, new = [0, 130, 0, 5, 0, 40, 2], [0, 1, 1, 9, 0, 3, 4]
    _case(3, kv, new, 2, 2, 64, 128, 128)
    _case(4, kv, new, 2, 16, 32, 64, 64)


def test_every_request_idle():
    rng = np.random.default_rng(0)
    cache = Cache(rng, [0, 0], 1, 64, 128, 128)
    q = bf16(rng.standard_normal((3, 2, 128)))
    out, lse = attend(q, cache.gpu(), cache.table, [0, 0, 0], [0, 0], 1, 1.0)
    assert (out.view(torch.int16) == -23131).all()


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales(scale):
    # 3.0: one token takes nearly all the weight
    _case(21, [300, 9], [1, 5], 2, 4, 64, 128, 128, scale=scale)


def test_far_logits():
    """Queries of 2^60 and 2^-60 next to ordinary ones: exponents of the split terms."""
    rng = np.random.default_rng(5)
    cache = Cache(rng, [200] * 3, 1, 64, 128, 128)
    q = rng.standard_normal((3, 4, 128))
    q[0] *= 2.0 ** 60
    q[1] *= 2.0 ** -60
    q[2, :, ::3] *= 2.0 ** -9                                # a wide spread within a block
    q = bf16(q)
    out, lse = attend(q, cache.gpu(), cache.table, [0, 1, 2, 3], [200] * 3, 1, 0.088)
    check_attention(out[1:], lse[1:], f64(q)[1:], cache.arrays, cache.table[1:], [0, 1, 2], [200] * 2,
                    0.088, "far")
    want = ref.attention(f64(q)[:1], *cache.arrays, cache.table[:1], [0, 1], [200], 0.088)
    assert np.allclose(f64(out)[:1], want[0], rtol=2.0 ** -8)       # one-hot weights


def test_identity_values():
    """Weights read back one by one: value t is the unit vector t, so out is p / sum p."""
    rng = np.random.default_rng(6)
    n = 128
    cache = Cache(rng, [n], 1, 64, 128, 128)
    pages = cache.table[0, :2]
    cache.v[pages] = 0
    for t in range(n):
        cache.v[pages[t // 64], 0, t, t % 64] = 0x38         # 1.0
    cache.vs[pages] = 1.0
    q = bf16(rng.standard_normal((1, 1, 128)))
    out, lse = attend(q, cache.gpu(), cache.table, [0, 1], [n], 1, 0.1)
    check_attention(out, lse, f64(q), cache.arrays, cache.table, [0, 1], [n], 0.1, "identity")


def test_one_hot_keys_pick_tokens():
    """A query that only token t answers returns v_t exactly (weights below 2^-100 elsewhere)."""
    rng = np.random.default_rng(8)
    n = 300
    cache = Cache(rng, [n], 1, 32, 128, 128)
    pages = cache.table[0, :10]
    cache.k[pages] = 0
    cache.ks[pages] = 1.0
    picks = [0, 31, 32, 127, 128, 299]
    for i, t in enumerate(picks):
        cache.k[pages[t // 32], 0, t % 32, i] = 0x7E         # 448
    q = np.zeros((1, len(picks), 128))
    for i in range(len(picks)):
        q[0, i, i] = 1.0
    out, _ = attend(bf16(q), cache.gpu(), cache.table, [0, 1], [n], 1, 1.0)
    for i, t in enumerate(picks):
        p = pages[t // 32]
        v = ref.VALUES[cache.v[p, 0, :, t % 32]] * cache.vs[p, 0]
        assert np.array_equal(f64(out)[0, i], v), f"token {t}"


def test_page_order_and_repeats_do_not_matter():
    """The same tokens behind other page numbers give the same bits, and so does a second call."""
    rng = np.random.default_rng(9)
    kv = [700, 90]
    cache = Cache(rng, kv, 2, 64, 128, 128)
    q = bf16(rng.standard_normal((2, 8, 128)))
    a, la = attend(q, cache.gpu(), cache.table, [0, 1, 2], kv, 1, 0.1)
    b, lb = attend(q, cache.gpu(), cache.table, [0, 1, 2], kv, 1, 0.1)
    P = cache.k.shape[0]
    perm = rng.permutation(P)
    inv = np.argsort(perm)
    moved = tuple(torch.from_numpy(x[perm]).to(dev()) for x in cache.arrays)
    table = inv[np.clip(cache.table, 0, P - 1)]
    c, lc = attend(q, moved, table, [0, 1, 2], kv, 1, 0.1)
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert torch.equal(a, c) and torch.equal(la, lc)


def test_strided_queries():
    rng = np.random.default_rng(10)
    kv, new = [150, 70], [2, 3]
    cache = Cache(rng, kv, 2, 64, 128, 128)
    wide = bf16(rng.standard_normal((5, 2 * 4 * 128 + 40)))
    for at in (0, 8, 3):                                     # aligned rows, and odd ones
        q = wide[:, at:at + 1024].unflatten(1, (8, 128))
        out, lse = attend(q, cache.gpu(), cache.table, [0, 2, 5], kv, 3, 0.1)
        check_attention(out, lse, f64(q), cache.arrays, cache.table, [0, 2, 5], kv, 0.1, f"at {at}")
    q = bf16(rng.standard_normal((8, 5, 128))).transpose(0, 1)       # head-major rows
    out, lse = attend(q, cache.gpu(), cache.table, [0, 2, 5], kv, 3, 0.1)
    check_attention(out, lse, f64(q), cache.arrays, cache.table, [0, 2, 5], kv, 0.1, "head-major")


def test_queries_that_are_not_finite_stay_in_their_row():
    rng = np.random.default_rng(12)
    cache = Cache(rng, [300], 1, 64, 128, 128)
    q = rng.standard_normal((2, 3, 128))
    q[0, 1, 5], q[1, 2, 100] = np.nan, np.inf
    clean = q.copy()
    clean[0, 1, 5] = clean[1, 2, 100] = 0
    out, _ = attend(bf16(q), cache.gpu(), cache.table, [0, 2], [300], 2, 0.1)
    good, _ = attend(bf16(clean), cache.gpu(), cache.table, [0, 2], [300], 2, 0.1)
    for t in range(2):
        for j in range(3):
            if (t, j) in ((0, 1), (1, 2)):
                assert torch.isnan(out[t, j].float()).all()
            else:
                assert torch.equal(out[t, j], good[t, j])


def test_a_nan_key_reaches_only_the_queries_that_see_it():
    rng = np.random.default_rng(13)
    n = 200
    cache = Cache(rng, [n], 1, 64, 128, 128)
    at = 150                                                 # position of the broken token
    cache.k[cache.table[0, at // 64], 0, at % 64] = 0x7F
    q = bf16(rng.standard_normal((n, 1, 128)))
    out, lse = attend(q, cache.gpu(), cache.table, [0, n], [n], n, 0.1)
    assert torch.isnan(out[at:].float()).all() and torch.isfinite(out[:at].float()).all()
    check_attention(out[:at], lse[:at], f64(q)[:at], cache.arrays, cache.table, [0, at], [at], 0.1, "before")


def test_more_queries_than_announced_are_left_alone():
    rng = np.random.default_rng(14)
    cache = Cache(rng, [90], 1, 64, 128, 128)
    q = bf16(rng.standard_normal((6, 2, 128)))
    out, _ = attend(q, cache.gpu(), cache.table, [0, 6], [90], 4, 0.1)
    full, _ = attend(q, cache.gpu(), cache.table, [0, 6], [90], 6, 0.1)
    assert (out[4:].view(torch.int16) == -23131).all()
    assert torch.allclose(out[:4].float(), full[:4].float(), rtol=2.0 ** -7, atol=1e-3)


def test_offsets_past_32_bits():
    """A pool of over 4 GiB per array, pages at both ends of it."""
    B, H, P = 128, 4, 70000                                  # 4.6 GB of keys
    k = torch.zeros(P, H, B, 128, dtype=torch.uint8, device=dev())
    v = torch.zeros(P, H, 128, B, dtype=torch.uint8, device=dev())
    ks = torch.ones(P, H, device=dev())
    vs = torch.ones(P, H, device=dev())
    rng = np.random.default_rng(15)
    small = Cache(rng, [300], H, B, 128, 128, spare=0)
    where = np.array([P - 1, 0, 65537])
    pages = small.table[0, :3]
    for x, y in zip((k, ks, v, vs), small.arrays):
        x[torch.from_numpy(where).to(dev())] = torch.from_numpy(y[pages]).to(dev())
    q = bf16(rng.standard_normal((1, 8, 128)))
    out, lse = attend(q, (k, ks, v, vs), where[None], [0, 1], [300], 1, 0.1)
    check_attention(out, lse, f64(q), small.arrays, small.table, [0, 1], [300], 0.1, "large pool")


def test_another_stream():
    rng = np.random.default_rng(16)
    cache = Cache(rng, [400], 2, 64, 128, 128)
    gpu = cache.gpu()
    q = bf16(rng.standard_normal((1, 8, 128)))
    ref_out, _ = attend(q, gpu, cache.table, [0, 1], [400], 1, 0.1)
    args = (i32(cache.table), i32([0, 1]), i32([400]), i32([0, 4]))
    out = torch.empty_like(ref_out)
    ws = bfp8.attn_paged_workspace(1, 1, 8, 2, 128, 128, dev())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    bfp8.bfp8_attn_paged(q, *gpu, *args, 1, 0.1, out, None, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref_out)


@pytest.mark.parametrize("seed", range(24))
def test_seeded_random_sizes(seed):
    rng = np.random.default_rng(1000 + seed)
    dk, dv = DIMS[seed % 3]
    R = int(rng.integers(1, 7))
    H = int(rng.choice([1, 2, 3]))
    G = int(rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 20]))
    B = int(rng.choice([32, 64, 128]))
    top = int(rng.choice([1, 1, 3, 9, 70, 200]))
    new = [int(x) for x in rng.integers(0, top + 1, R)]
    kv = [n + int(rng.integers(0, 600)) if n else 0 for n in new]
    _case(1000 + seed, kv, new, H, G, B, dk, dv, workspace=bool(seed % 4))


# ------------------------------------------------------------- many query columns

@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
def test_chunks_split_over_tokens(dk, dv, B):
    # few blocks: their tokens are shared by several workgroups where they are many
    _case(dk + B, [1500, 40, 513, 2100], [40, 40, 17, 1], 2, 4, B, dk, dv)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_chunks_of_many_heads(dk, dv):
    # enough blocks for the larger workgroups
    _case(dk + 1, [300, 700, 64, 90], [300, 150, 64, 33], 64, 1, 64, dk, dv)


@pytest.mark.parametrize("H", [1, 4])
def test_more_requests_than_lanes_with_a_chunk(H):
    rng = np.random.default_rng(H)
    new = [int(x) for x in rng.integers(0, 4, 150)]
    kv = [n + int(rng.integers(0, 90)) if n else 0 for n in new]
    new[3], kv[3], new[140], kv[140] = 130, 1300, 70, 70
    _case(30 + H, kv, new, H, 2, 32, 128, 128)


@pytest.mark.parametrize("G", [1, 3])
def test_more_requests_than_lanes(G):
    # every workgroup's range of tiles passes over idle requests and request boundaries
    rng = np.random.default_rng(40 + G)
    new = [int(x) for x in rng.integers(0, 3, 333)]
    kv = [n + int(rng.choice([0, 1, 60, 127, 128, 300])) if n else 0 for n in new]
    _case(40 + G, kv, new, 9, G, 64, 64, 64)


def test_most_requests():
    R = bfp8.KV_MAX_REQUESTS
    rng = np.random.default_rng(50)
    new = [int(x) for x in rng.integers(0, 2, R)]
    kv = [n + int(rng.integers(0, 5)) if n else 0 for n in new]
    _case(50, kv, new, 1, 2, 32, 64, 64)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales_of_chunks(scale):
    _case(22, [300, 600], [90, 30], 2, 4, 64, 128, 128, scale=scale)


@pytest.mark.parametrize("workspace", [True, False])
def test_chunks_with_and_without_a_workspace(workspace):
    _case(60, [1700, 1100], [60, 50], 2, 4, 64, 128, 128, workspace=workspace)


def test_padded_tokens_and_a_small_workspace():
    """T far above R * max_new: the workspace is sized for the latter."""
    rng = np.random.default_rng(62)
    cache = Cache(rng, [1300], 1, 64, 128, 128)
    q = bf16(rng.standard_normal((900, 4, 128)))
    out, lse = attend(q, cache.gpu(), cache.table, [0, 30], [1300], 30, 0.1)
    check_attention(out[:30], lse[:30], f64(q)[:30], cache.arrays, cache.table, [0, 30], [1300], 0.1, "padded")
    assert (out[30:].view(torch.int16) == -23131).all()


def test_far_logits_of_chunks():
    """Queries of 2^60, 2^-60 and a wide spread in one block, and value scales 2^20 apart."""
    rng = np.random.default_rng(61)
    n = 200
    cache = Cache(rng, [n], 1, 64, 128, 128, spread=20)
    q = rng.standard_normal((n, 1, 128))
    q[64:70] *= 2.0 ** 60
    q[70:80] *= 2.0 ** -60
    q[80:, :, ::3] *= 2.0 ** -9
    q = bf16(q)
    out, lse = attend(q, cache.gpu(), cache.table, [0, n], [n], n, 4.0)
    want, want_lse, weight, slack = ref.attention(f64(q), *cache.arrays, cache.table, [0, n], [n], 4.0)
    plain = np.r_[0:64, 70:n]
    err = np.abs(f64(out) - want)[plain]
    bound = 2.0 ** -9 * np.abs(want) + (2.0 ** -8 + 2 * slack[..., None]) * weight + 1e-30
    assert (err <= bound[plain]).all(), f"worst {np.max(err / bound[plain]):.3f}"
    assert np.allclose(f64(out)[64:70], want[64:70], rtol=2.0 ** -8)         # one-hot weights
