"""bfp8_attn_paged where its loops run long: workgroups that walk several requests and several tiles a
wave, blocks whose page numbers are fetched again and again, and weights whose last bits count."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import kv_terms
from gpu_helpers import announce, dev
from kv_helpers import Cache, attend, bf16, f64, i32, offsets

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 128), (192, 128)]


def run(rng, kv, new, H, G, B, dk, dv, what, workspaces=(True, False)):
    """With and without a workspace, each against the 64-bit reference and its bound."""
    cache = Cache(rng, kv, H, B, dk, dv)
    q_off = offsets(new)
    q = bf16(rng.standard_normal((int(q_off[-1]) + 1, H * G, dk)))          # a row of no request
    gpu, max_new = cache.gpu(), max(max(new), 1)
    for ws in workspaces:
        announce(f"attention {what} {dk}/{dv} B={B} H={H} G={G} R={len(kv)} workspace={ws}")
        out, lse = attend(q, gpu, cache.table, q_off, kv, max_new, dk ** -0.5, ws)
        worst = kv_terms.check(f64(out), f64(lse), f64(q), cache.arrays, cache.table, q_off, kv, dk ** -0.5, what)
        announce(f"worst err/bound {worst:.3f}")
        assert (out[-1].view(torch.int16) == -23131).all(), "a row of no request was written"


def per_workgroup(kv, H, max_new, G, dk, dv):
    """128-token tiles that a workgroup of the form for few columns walks."""
    groups = bfp8.bfp8_attn_paged_workspace_size(len(kv), max_new, H * G, H, dk, dv) // (2 * 16 * (dv + 2) * 4)
    units = sum(-(-n // 128) for n in kv) * H * -(-max_new * G // 16)
    return -(-units // groups)


# ------------------------------------------------------------------ few query columns

def ragged(rng, R, top):
    """Lengths of one token to `top`, many of them long; every ninth request is idle."""
    kv = np.where(rng.random(R) < 0.6, rng.integers(top // 2, top + 1, R), rng.integers(1, 300, R))
    kv[4::9] = 0
    return kv


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
def test_requests_handed_over_within_a_workgroup(dk, dv, B):
    rng = np.random.default_rng(dk + B)
    kv = ragged(rng, 170 if dv == 64 else 90, 1100)
    new = (kv > 0).astype(int)
    assert per_workgroup(kv, 4, 1, 2, dk, dv) >= 3
    run(rng, [int(x) for x in kv], [int(x) for x in new], 4, 2, B, dk, dv, "hand-over")


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
def test_column_tiles_that_are_skipped(dk, dv, B):
    # 24 columns at most: a request with one or two new tokens has none in the second tile of 16
    rng = np.random.default_rng(2 * dk + B)
    kv = ragged(rng, 150 if dv == 64 else 75, 1000)
    new = np.minimum(np.where(kv > 0, rng.integers(1, 4, len(kv)), 0), kv)
    assert per_workgroup(kv, 4, 3, 8, dk, dv) >= 4
    run(rng, [int(x) for x in kv], [int(x) for x in new], 4, 8, B, dk, dv, "skipped columns")


@pytest.mark.parametrize("dk,dv", DIMS)
def test_one_long_cache(dk, dv):
    # a wave walks several tiles of one request, workgroup after workgroup
    rng = np.random.default_rng(dk + 7)
    kv = [170001]
    assert per_workgroup(kv, 2, 1, 8, dk, dv) >= 3
    run(rng, kv, [1], 2, 8, 128, dk, dv, "long cache", workspaces=(True,))


# ------------------------------------------------------------------ many query columns

@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
@pytest.mark.parametrize("more", [0, 66])
def test_blocks_over_thousands_of_tokens(dk, dv, B, more):
    # without a workspace one workgroup walks them all; more: requests than lanes, blocks by number
    rng = np.random.default_rng(dk + B + more)
    kv = [2049, 2113, 4200, 6300] + [int(x) for x in rng.integers(0, 40, more)]
    new = [40, 33, 35, 40] + [min(n, 1) for n in kv[4:]]
    run(rng, kv, new, 1, 2, B, dk, dv, "long blocks")


@pytest.mark.parametrize("dk,dv", DIMS)
def test_parts_of_many_tiles(dk, dv):
    # sixteen parts of 39 tiles of 64 tokens, which start anywhere
    rng = np.random.default_rng(dk + 3)
    run(rng, [40000], [40], 1, 2, 64, dk, dv, "long parts", workspaces=(True,))


@pytest.mark.parametrize("dk,dv,B", [(64, 64, 128), (128, 128, 32), (192, 128, 64)])
def test_large_workgroups_over_thousands_of_tokens(dk, dv, B):
    rng = np.random.default_rng(dk + 5)
    run(rng, [4200, 66, 2111, 300], [66, 66, 1, 70], 64, 1, B, dk, dv, "large workgroups", workspaces=(True,))


# ------------------------------------------------------------------ the last bits of weights

@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("B", [32, 64, 128])
@pytest.mark.parametrize("at", [0, 70, 512])
def test_values_that_cancel(dk, dv, B, at):
    """Both forms; every token of a 64-token tile in turn has a weight that must keep its remainder."""
    c = kv_terms.Cancelling(dk + B + at, at, at + 130, B, dk, dv, draws=8)
    gpu = tuple(torch.from_numpy(x).to(dev()) for x in c.arrays)
    q = bf16(c.q.transpose(1, 0, 2))                                 # [pair, draw as head, dk]
    announce(f"cancelling values {dk}/{dv} B={B} at={at}")
    # one token a request: few columns
    table = np.repeat(c.table, c.PAIRS, 0)
    one = [c.n] * c.PAIRS
    for ws in (True, False):
        out, lse = attend(q, gpu, table, np.arange(c.PAIRS + 1), one, 1, 1.0, ws)
        kv_terms.check(f64(out), f64(lse), f64(q), c.arrays, table, np.arange(c.PAIRS + 1), one, 1.0, "few columns")
    # one request of 32 tokens, which all see the pairs: 256 columns
    off = np.array([0, c.PAIRS])
    for ws in (True, False):
        out, lse = attend(q, gpu, c.table, off, [c.n], c.PAIRS, 1.0, ws)
        kv_terms.check(f64(out), f64(lse), f64(q), c.arrays, c.table, off, [c.n], 1.0, "many columns")


@pytest.mark.parametrize("dk,dv", DIMS)
def test_values_that_cancel_in_large_workgroups(dk, dv):
    c = kv_terms.Cancelling(dk, 70, 200, 64, dk, dv, draws=8)
    R = 256                                                          # a block each: every CU is taken
    gpu = tuple(torch.from_numpy(x).to(dev()) for x in c.arrays)
    q = bf16(c.q.transpose(1, 0, 2))
    off = np.arange(R + 1) * c.PAIRS
    announce(f"cancelling values {dk}/{dv}, {R} requests")
    out, lse = attend(q.repeat(R, 1, 1), gpu, np.repeat(c.table, R, 0), off, [c.n] * R, c.PAIRS, 1.0)
    out, lse = out.view(R, *q.shape[:2], dv), lse.view(R, *q.shape[:2])
    kv_terms.check(f64(out[0]), f64(lse[0]), f64(q), c.arrays, c.table, off[:2], [c.n], 1.0, "large workgroups")
    assert (out == out[:1]).all() and (lse == lse[:1]).all()


# ------------------------------------------------------------------ chain

@pytest.mark.parametrize("dk,dv", DIMS)
def test_chain_without_a_workspace(dk, dv):
    """Plan, append and attention over several steps, attention with and without a workspace."""
    rng = np.random.default_rng(dk)
    H, G, B, R = 2, 3, 32, 4
    steps = np.array([[70, 1, 0, 33], [1, 1, 5, 1], [1, 0, 1, 31], [40, 3, 1, 1]])
    total = steps.sum(0)
    P = int((-(-total // B)).sum()) + 1
    cache = bfp8.kv_cache_buffers(P, H, B, dk, dv, dev())
    table = i32(np.zeros((R, int((-(-total // B)).max()))))
    free, head, ctx = i32(rng.permutation(P)), None, np.zeros(R, int)
    for x in cache:
        x.fill_(0x7F if x.dtype == torch.uint8 else float("nan"))
    for n, new in enumerate(steps):
        T, most = int(new.sum()), int(new.max())
        plan = bfp8.kv_plan(i32(ctx), i32(new), free, table, B, T, head)
        head = plan.counts[1:2].clone()
        k, v, q = (bf16(rng.standard_normal((T, h, d))) for h, d in ((H, dk), (H, dv), (H * G, dk)))
        bfp8.bfp8_kv_append(k, v, plan.slot_map, *cache)
        arrays = [x.cpu().numpy() for x in cache]
        q_off, kv, tab = (x.cpu().numpy() for x in (plan.q_offsets, plan.kv_lens, table))
        for ws in (bfp8.attn_paged_workspace(R, most, H * G, H, dk, dv, dev()), None):
            out = torch.empty(T, H * G, dv, dtype=torch.bfloat16, device=dev())
            lse = torch.empty(T, H * G, device=dev())
            announce(f"chain step {n} {dk}/{dv} workspace={ws is not None}")
            bfp8.bfp8_attn_paged(q, *cache, table, plan.q_offsets, plan.kv_lens, plan.tile_offsets, most,
                                 dk ** -0.5, out, lse, ws)
            torch.cuda.synchronize()
            kv_terms.check(f64(out), f64(lse), f64(q), arrays, tab, q_off, kv, dk ** -0.5, f"step {n}")
        ctx = ctx + new
