"""The latent cache's calls where offsets, sizes and launches reach their ends: pools past 4 GiB, queries
far apart, tables whose width forbids a split launch, both forms of the gather, captured calls."""
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


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_a_pool_past_four_gib():
    """Pages on both sides of the 2^32nd byte of codes and of the pool's end, by all three calls."""
    rng = np.random.default_rng(51)
    B, H, kv = 128, 40, [300, 1, 129]
    P = (1 << 32) // (B * 512) + 1500
    far = np.array([[P - 1, (1 << 32) // (B * 512), 0], [P - 700, 5, 5], [(1 << 32) // (B * 512) - 1, P - 2, 5]], np.int32)
    near = np.arange(9, dtype=np.int32).reshape(3, 3)
    announce(f"pool of {P} pages of {B}")
    big = bfp8.latent_cache_buffers(P, B, dev())
    small = bfp8.latent_cache_buffers(9, B, dev())
    q_off, T = offsets(kv), sum(kv)
    rows = bf16(rng.standard_normal((T, 576)))
    freq, amplitude = bfp8.rope_frequencies(64, device=dev())
    pos = i32(np.concatenate([np.arange(n) for n in kv]))
    for cache, table in ((big, far), (small, near)):
        slots = [int(table[r, p // B]) * B + p % B for r, n in enumerate(kv) for p in range(n)]
        bfp8.bfp8_latent_append(rows, i32(slots), pos, freq, *cache, amplitude=amplitude)
    gathered = [bfp8.latent_gather(cache, i32(table), i32(q_off), T) for cache, table in ((big, far), (small, near))]
    assert _same(gathered[0][0], gathered[1][0]) and _same(gathered[0][1], gathered[1][1])
    assert torch.isfinite(gathered[0][0].float()).all() and gathered[0][0].float().abs().sum() > 0
    ql, qr = queries(rng, 3, H)
    for workspace in (True, False):
        outs = [attend(ql, qr, cache, table, [0, 1, 2, 3], kv, 1, SCALE, workspace) for cache, table in ((big, far), (small, near))]
        assert _same(outs[0][0], outs[1][0]) and _same(outs[0][1], outs[1][1])
    arrays = small[0].cpu().numpy(), small[1].cpu().numpy(), f64(small[2])
    check(outs[1][0], outs[1][1], ql, qr, arrays, near, [0, 1, 2, 3], kv, SCALE)


@pytest.mark.parametrize("H", [16, 70])
@pytest.mark.parametrize("workspace", [True, False])
def test_queries_and_outputs_far_apart(H, workspace):
    """Token strides of 2^27 elements, which are more than 32 bits of offset allow for."""
    rng = np.random.default_rng(52)
    kv, far = [200, 70, 1], 1 << 27
    cache = LatentCache(rng, kv, 64)
    ql, qr = queries(rng, 3, H)
    wide = [torch.empty(2 * far + H * 576, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    fl = wide[0].as_strided((3, H, 512), (far, 576, 1))
    fr = wide[0].as_strided((3, H, 64), (far, 576, 1), 512)
    fo = wide[1].as_strided((3, H, 512), (far, 512, 1))
    fl.copy_(ql)
    fr.copy_(qr)
    gpu = cache.gpu()
    want, _ = attend(ql, qr, gpu, cache.table, [0, 1, 2, 3], kv, 1, SCALE, workspace)
    ws = bfp8.attn_latent_workspace(3, 1, H, dev()) if workspace else None
    bfp8.bfp8_attn_latent(fl, fr, *gpu, i32(cache.table), i32([0, 1, 2, 3]), i32(kv), 1, SCALE, fo, None, ws)
    torch.cuda.synchronize()
    assert _same(fo, want)


def test_a_table_too_wide_to_split():
    """A table that could hold 2^31 tiles and more takes the launch without parts, same rows."""
    rng = np.random.default_rng(53)
    R, B, H = 64, 128, 128
    kv = [int(n) for n in rng.integers(0, 200, R)]
    cache = LatentCache(rng, kv, B)
    gpu = cache.gpu()
    ql, qr = queries(rng, R, H)
    W = 1 << 23
    table = torch.zeros(R, W, dtype=torch.int32, device=dev())
    table[:, :cache.table.shape[1]] = i32(cache.table)
    out = torch.zeros(R, H, 512, dtype=torch.bfloat16, device=dev())
    lse = torch.zeros(R, H, dtype=torch.float32, device=dev())
    ws = bfp8.attn_latent_workspace(R, 1, H, dev())
    bfp8.bfp8_attn_latent(ql, qr, *gpu, table, i32(range(R + 1)), i32(kv), 1, SCALE, out, lse, ws)
    want, want_lse = attend(ql, qr, gpu, cache.table, range(R + 1), kv, 1, SCALE, workspace=False)
    assert _same(out, want) and _same(lse, want_lse)
    check(out, lse, ql, qr, cache.arrays, cache.table, range(R + 1), kv, SCALE)


@pytest.mark.parametrize("rows", [39999, 40000, 45001])
def test_gather_of_many_rows(rows):
    """Both sides of the size at which a wave takes fewer rows, against the codes widened by torch."""
    torch.manual_seed(rows)
    B, R = 64, 9
    cuts = [0] + sorted(torch.randint(0, rows - 7, (R - 1,)).tolist()) + [rows - 7]      # seven rows of no request
    lens = np.diff(cuts)
    W = -(-int(lens.max()) // B) + 1
    table = torch.randperm(R * W, device=dev()).to(torch.int32).view(R, W)
    codes = torch.randint(0, 127, (R * W, B, 512), dtype=torch.uint8, device=dev())
    scales = torch.randint(-9, 9, (R * W, B), device=dev()).float().exp2()
    rope = torch.randn(R * W, B, 64, device=dev()).bfloat16()
    latent = torch.full((rows, 512), -7.0, dtype=torch.bfloat16, device=dev())
    keys = torch.full((rows, 64), -7.0, dtype=torch.bfloat16, device=dev())
    bfp8.bfp8_latent_gather(codes, scales, rope, table, i32(cuts), latent, keys)
    for r in range(R):
        n = int(lens[r])
        pages = table[r, :-(-n // B)].long()
        wide = (codes[pages].view(torch.float8_e4m3fn).float() * scales[pages][..., None]).flatten(0, 1)[:n]
        assert torch.equal(latent[cuts[r]:cuts[r + 1]].float(), wide)                    # exact: four bits
        assert torch.equal(keys[cuts[r]:cuts[r + 1]], rope[pages].flatten(0, 1)[:n])
    assert (latent[-7:] == -7).all() and (keys[-7:] == -7).all()


def test_rope_append_and_gather_replayed():
    """A captured chain of the calls, replayed as rows, positions and slots change."""
    rng = np.random.default_rng(54)
    T, H, B, P = 37, 3, 32, 6
    x, rows = bf16(rng.standard_normal((T, H, 64))), bf16(rng.standard_normal((T, 576)))
    pos, slots = i32(range(T)), i32(range(T))
    freq, amplitude = bfp8.rope_frequencies(64, device=dev())
    table, ends = i32([list(range(P))]), i32([0, P * B])

    def buffers():
        cache = [t.zero_() for t in bfp8.latent_cache_buffers(P, B, dev())]
        return [torch.zeros(T, H, 64, dtype=torch.bfloat16, device=dev()), *cache,
                torch.zeros(P * B, 512, dtype=torch.bfloat16, device=dev()),
                torch.zeros(P * B, 64, dtype=torch.bfloat16, device=dev())]

    def call(b):
        bfp8.bfp8_rope(x, pos, freq, b[0], True, amplitude)
        bfp8.bfp8_latent_append(rows, slots, pos, freq, *b[1:4], amplitude=amplitude)
        bfp8.bfp8_latent_gather(*b[1:4], table, ends, b[4], b[5])
    got, want = buffers(), buffers()
    call(got)
    call(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(got)
    for k in range(4):
        x.copy_(bf16(rng.standard_normal((T, H, 64))))
        rows.copy_(bf16(rng.standard_normal((T, 576)) * 2.0 ** k))
        pos.copy_(i32(rng.integers(0, 100000, T)))
        slots.copy_(i32(rng.permutation(P * B)[:T]))
        graph.replay()
        call(want)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert _same(a, b), f"replay {k}"
