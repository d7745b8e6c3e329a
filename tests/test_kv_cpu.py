"""The paged cache's C ABI without a GPU (refusals, before any HIP call) and the plain
implementations the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_04_amd as bfp8
import kv_reference as ref
from block_scaled_fp8_04_amd import _lib

FAKE = ctypes.c_void_p(0x10000)            # aligned, never dereferenced: every call is rejected
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return _lib.library()


def plan(lib, **kw):
    a = dict(ctx=FAKE, new=FAKE, R=4, free=FAKE, n_free=8, head=None, table=FAKE, W=4, B=64, q=FAKE, kv=FAKE,
             tiles=FAKE, slots=FAKE, pos=FAKE, T=16, counts=FAKE)
    a.update(kw)
    return lib.bfp8_kv_plan(a["ctx"], a["new"], a["R"], a["free"], a["n_free"], a["head"], a["table"], a["W"],
                            a["B"], a["q"], a["kv"], a["tiles"], a["slots"], a["pos"], a["T"], a["counts"], None)


def test_plan_refusals(lib):
    for B in (0, 16, 48, 256, -64):
        assert plan(lib, B=B) == _lib.BFP8_ERR_ARG
    for kw in (dict(R=-1), dict(T=-1), dict(T=BIG), dict(n_free=-1), dict(n_free=BIG), dict(W=-1),
               dict(W=BIG // 64)):
        assert plan(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    assert plan(lib, R=bfp8.KV_MAX_REQUESTS + 1) == _lib.BFP8_ERR_GROUPS
    for name in ("ctx", "new", "free", "table", "q", "kv", "tiles", "slots", "pos", "counts"):
        assert plan(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
        assert plan(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    assert plan(lib, head=ODD) == _lib.BFP8_ERR_ALIGN
    assert plan(lib, R=0, q=None) == _lib.BFP8_ERR_NULL      # offsets are written all the same


def append(lib, **kw):
    a = dict(k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, slots=FAKE, T=4, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE,
             P=8, B=64, H=2, dk=128, dv=128)
    a.update(kw)
    return lib.bfp8_kv_append(a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["slots"], a["T"], a["kc"],
                              a["ks"], a["vc"], a["vs"], a["P"], a["B"], a["H"], a["dk"], a["dv"], None)


def test_append_refusals(lib):
    assert append(lib, B=16) == _lib.BFP8_ERR_ARG
    for kw in (dict(T=-1), dict(T=BIG), dict(H=0), dict(H=65536), dict(P=-1), dict(P=BIG // 64), dict(kt=-1),
               dict(kh=-1), dict(vt=-1), dict(vh=-1), dict(dk=64), dict(dv=64), dict(dk=192, dv=192),
               dict(dk=0, dv=0), dict(dk=256, dv=256)):
        assert append(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    for name in ("k", "v", "slots", "kc", "ks", "vc", "vs"):
        assert append(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
    for name in ("slots", "kc", "ks", "vc", "vs"):
        assert append(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    assert append(lib, k=ctypes.c_void_p(0x10001)) == _lib.BFP8_ERR_ALIGN
    assert append(lib, T=0, k=None) == _lib.BFP8_OK
    assert append(lib, P=0, kc=None) == _lib.BFP8_OK


def attn(lib, **kw):
    a = dict(q=FAKE, qt=512, qh=128, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, P=8, B=64, table=FAKE, W=4, off=FAKE,
             kv=FAKE, tiles=FAKE, R=2, T=2, max_new=1, hq=4, hkv=2, dk=128, dv=128, scale=0.1, out=FAKE,
             lse=None, ws=None, wsb=0)
    a.update(kw)
    return lib.bfp8_attn_paged(a["q"], a["qt"], a["qh"], a["kc"], a["ks"], a["vc"], a["vs"], a["P"], a["B"],
                               a["table"], a["W"], a["off"], a["kv"], a["tiles"], a["R"], a["T"], a["max_new"],
                               a["hq"], a["hkv"], a["dk"], a["dv"], a["scale"], a["out"], a["lse"], a["ws"],
                               a["wsb"], None)


def test_attention_refusals(lib):
    assert attn(lib, B=48) == _lib.BFP8_ERR_ARG
    for s in (math.nan, math.inf, -math.inf):
        assert attn(lib, scale=s) == _lib.BFP8_ERR_ARG
    for kw in (dict(R=-1), dict(T=-1), dict(T=BIG), dict(max_new=-1), dict(max_new=0), dict(max_new=BIG // 4),
               dict(hkv=0), dict(hq=0), dict(hq=3), dict(hq=1), dict(hq=65536), dict(dk=64), dict(dk=576, dv=512),
               dict(qt=-1), dict(qh=-1), dict(P=-1), dict(P=BIG // 64), dict(W=-1), dict(W=BIG // 64)):
        assert attn(lib, **kw) == _lib.BFP8_ERR_SHAPE, kw
    assert attn(lib, R=bfp8.KV_MAX_REQUESTS + 1) == _lib.BFP8_ERR_GROUPS
    for name in ("q", "kc", "ks", "vc", "vs", "table", "off", "kv", "tiles", "out"):
        assert attn(lib, **{name: None}) == _lib.BFP8_ERR_NULL, name
    for name in ("kc", "ks", "vc", "vs", "table", "off", "kv", "tiles", "out", "lse", "ws"):
        assert attn(lib, **{name: ODD}) == _lib.BFP8_ERR_ALIGN, name
    assert attn(lib, q=ctypes.c_void_p(0x10001)) == _lib.BFP8_ERR_ALIGN
    assert attn(lib, R=0, q=None) == _lib.BFP8_OK
    assert attn(lib, T=0, q=None) == _lib.BFP8_OK


def test_attention_workspace(lib):
    size = bfp8.bfp8_attn_paged_workspace_size
    for args in ((1, 1, 16, 4, 128, 128), (64, 1, 64, 8, 128, 128), (3, 4, 12, 4, 64, 64), (8, 500, 32, 32, 192, 128)):
        n = size(*args)
        assert n >= 0 and n % 16 == 0
        if n:
            R, mn, hq, hkv, dk, dv = args
            assert attn(lib, R=R, T=R * mn, max_new=mn, hq=hq, hkv=hkv, dk=dk, dv=dv, ws=FAKE,
                        wsb=n - 16) == _lib.BFP8_ERR_WORKSPACE
    assert size(0, 1, 4, 2, 128, 128) == size(1, 0, 4, 2, 128, 128) == size(1, 1, 4, 3, 128, 128) == 0
    assert size(1, 1, 4, 2, 576, 512) == size(5000, 1, 4, 2, 128, 128) == 0


def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        bfp8.bfp8_kv_plan(i, i, i, torch.zeros(4, 2, dtype=torch.int32), 64, bfp8.kv_plan_buffers(4, 4, "cpu"))
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cache = bfp8.kv_cache_buffers(3, 2, 64, 128, 128, "cpu")
    with pytest.raises(ValueError):
        bfp8.bfp8_kv_append(x, x, i, *cache)
    with pytest.raises(ValueError):
        bfp8.bfp8_attn_paged(x, *cache, torch.zeros(4, 2, dtype=torch.int32), i, i, i, 1, 1.0, x)


def test_reference_codes():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.VALUES, t, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * 2.0 ** np.arange(-10, 10).repeat(1000),
                        [0.0, 448.0, 460.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0]])
    x = x[np.abs(x) < 464].astype(np.float32)
    want = torch.from_numpy(np.concatenate([x, -x])).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(np.concatenate([x, -x])), want)
    assert ref.encode(np.array([1e9, -1e9])).tolist() == [0x7E, 0xFE]


def test_reference_scale():
    for a in (0.0, 1e-4, 1.0, 448.0, 449.0, 3.7, 1e30):
        s = ref.scale_of(a)
        y = max(a, float(np.float32(1e-4))) / 448
        assert math.log2(s) == int(math.log2(s)) and y <= s * (1 + 1e-7) and s < 2 * y * (1 + 1e-6)


def test_reference_attention_is_softmax():
    """Against torch's softmax in 64 bits on one dense request."""
    rng = np.random.default_rng(1)
    B, n, H, G, d = 32, 70, 2, 2, 64
    k, v = rng.standard_normal((n, H, d)), rng.standard_normal((n, H, d))
    cache = [np.zeros((4, H, B, d), np.uint8), np.ones((4, H), np.float32), np.zeros((4, H, d, B), np.uint8),
             np.ones((4, H), np.float32)]
    table = np.array([[2, 0, 3]])
    slots = [int(table[0, i // B]) * B + i % B for i in range(n)]
    cache = ref.append(k, v, slots, *cache)
    q = rng.standard_normal((5, H * G, d))
    out, lse, weight, _ = ref.attention(q, *cache, table, [0, 5], [n], 0.2)
    dk = np.stack([ref.VALUES[cache[0][table[0, i // B], :, i % B]] * cache[1][table[0, i // B]][:, None] for i in range(n)])
    dv = np.stack([ref.VALUES[cache[2][table[0, i // B], :, :, i % B]] * cache[3][table[0, i // B]][:, None] for i in range(n)])
    assert np.abs(dk - k).max() < 2.0 ** -3 and np.abs(dv - v).max() < 2.0 ** -3
    z = torch.einsum("thd,nhd->thn", torch.from_numpy(q), torch.from_numpy(dk).repeat_interleave(G, 1)) * 0.2
    z.masked_fill_(torch.arange(n)[None, None, :] > (n - 5 + torch.arange(5))[:, None, None], -math.inf)
    want = torch.einsum("thn,nhd->thd", z.softmax(2), torch.from_numpy(dv).repeat_interleave(G, 1))
    assert np.allclose(out, want.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(z, 2).numpy(), rtol=1e-12)
    assert (np.abs(out) <= weight + 1e-15).all()
